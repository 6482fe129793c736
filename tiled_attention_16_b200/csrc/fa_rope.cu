// fa_rope.cu — RMS norm of each query and key head with the position rotation
// in the same pass, forward and backward (include/fa_rope.h has the formulas).
//
// Bound by HBM: the forward reads and writes 2 bytes an element, the backward
// reads 4 and writes 2.  A row (one head of one token) is held by D / 8 lanes
// with 8 values each, chosen so that both values of every rotated pair are in
// one lane: lane c takes values [4c, 4c+4) and the four partners (or 8c .. 8c+7
// when pairs are neighbours), lanes past the rotated part take 8 neighbours
// with cos = 1, sin = 0.  A thread keeps one token for all the heads it walks,
// so its four angles are reduced (in fp64) and turned into cos / sin once, in
// registers; no shared memory and no table are read per row.  Four rows are
// loaded before the first is used.
#include "fa_internal.h"
#include "sm100.cuh"

#include <cuda_bf16.h>

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;

// The two groups of four consecutive values that lane c of a row holds, and
// the first of its four rotation indices (-1: not rotated).
struct LaneMap {
    int o0, o1, pair0;
};

template <bool kInter>
__device__ __forceinline__ LaneMap lane_map(int c, int rot) {
    LaneMap m;
    if (kInter) {
        m.o0 = 8 * c;
        m.o1 = 8 * c + 4;
        m.pair0 = 8 * c < rot ? 4 * c : -1;
    } else if (c < rot / 8) {
        m.o0 = 4 * c;
        m.o1 = rot / 2 + 4 * c;
        m.pair0 = 4 * c;
    } else {
        m.o0 = rot + (c - rot / 8) * 8;
        m.o1 = m.o0 + 4;
        m.pair0 = -1;
    }
    return m;
}

// cos and sin of the lane's four angles p * inv_freq.  The number of turns is
// formed and reduced to [-1/2, 1/2] in fp64 (its error, 2^-53 of up to 2^31
// turns, is 2e-7); fp32 sincospi does the rest.
__device__ __forceinline__ void lane_angles(const LaneMap& m, const float* inv_freq, int pos, float (&cs)[4],
                                            float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (m.pair0 >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double t = static_cast<double>(pos) * static_cast<double>(inv_freq[m.pair0 + i]) * 0.15915494309189535;
            sincospif(static_cast<float>(2.0 * (t - rint(t))), &sn[i], &cs[i]);
        }
    }
}

// Values 0..3 are the lane's first group, 4..7 its second.  Index pairs that
// rotate together: (i, i + 4), or (2i, 2i + 1) when interleaved.
template <bool kInter>
__device__ __forceinline__ void turn(float (&u)[8], const float (&cs)[4], const float (&sn)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = kInter ? 2 * i : i, b = kInter ? 2 * i + 1 : i + 4;
        const float x = u[a], y = u[b];
        u[a] = x * cs[i] - y * sn[i];
        u[b] = y * cs[i] + x * sn[i];
    }
}

struct Raw8 {
    uint2 a, b;
};

__device__ __forceinline__ Raw8 load8(const __nv_bfloat16* p, const LaneMap& m) {
    Raw8 r;
    r.a = __ldg(reinterpret_cast<const uint2*>(p + m.o0));
    r.b = __ldg(reinterpret_cast<const uint2*>(p + m.o1));
    return r;
}

__device__ __forceinline__ void unpack8(const Raw8& r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const LaneMap& m, const float (&v)[8]) {
    *reinterpret_cast<uint2*>(p + m.o0) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    *reinterpret_cast<uint2*>(p + m.o1) = make_uint2(pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void load_weights(const void* w, int bf16, const LaneMap& m, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = (i < 4 ? m.o0 : m.o1 - 4) + i;
        v[i] = bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[d])
                    : reinterpret_cast<const float*>(w)[d];
    }
}

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int k = kLanes / 2; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    return x;
}

// Where a thread stands: CTA item = (token group, head part); 256 / (D / 8)
// row slots a CTA, token_slots of them for different tokens, the rest for
// different heads of the same tokens (few tokens: all slots stay busy).
struct Place {
    bool live;        // the token exists
    int b, n, slot_h; // token and first head slot
    int h0, h1;       // heads [h0, h1) of q followed by k belong to this CTA
};

template <int D>
__device__ __forceinline__ Place place(const RopeParams& p, int item) {
    const int slot = threadIdx.x / (D / 8);
    const int group = item / p.head_parts, part = item - group * p.head_parts;
    const long long t = static_cast<long long>(group) * p.token_slots + (slot & (p.token_slots - 1));
    Place w;
    w.live = t < p.tokens;
    w.b = w.live ? static_cast<int>(t / p.N) : 0;
    w.n = w.live ? static_cast<int>(t - static_cast<long long>(w.b) * p.N) : 0;
    w.slot_h = slot / p.token_slots;
    const int H = p.Hq + p.Hkv;
    w.h0 = static_cast<int>(static_cast<long long>(H) * part / p.head_parts);
    w.h1 = static_cast<int>(static_cast<long long>(H) * (part + 1) / p.head_parts);
    return w;
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads)
fa_qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;
    const int step = kRopeThreads / kLanes / p.token_slots;   // head slots
    const Place w = place<D>(p, static_cast<int>(blockIdx.x));
    const LaneMap m = lane_map<kInter>(threadIdx.x & (kLanes - 1), p.rot);
    const int pos = p.positions ? (w.live ? __ldg(p.positions + static_cast<size_t>(w.b) * p.N + w.n) : 0) : w.n;
    float cs[4], sn[4];
    bool have_angles = false;

    // heads [lo, hi) of one of the two tensors; every lane of a warp runs the
    // same number of iterations (the shuffles are over whole warps)
    auto walk = [&](const RopeRows& x, __nv_bfloat16* out, int H, const void* weight, int lo, int hi) {
        if (lo >= hi) return;
        const __nv_bfloat16* src = x.data + w.b * x.stride_b + w.n * x.stride_n;
        float wt[8];
        load_weights(weight, p.weight_bf16, m, wt);
        for (int h = lo; h < hi; h += step * kRopeUnroll) {
            Raw8 raw[kRopeUnroll];
#pragma unroll
            for (int i = 0; i < kRopeUnroll; ++i) {
                const int hh = h + i * step + w.slot_h;
                raw[i] = Raw8{};
                if (w.live && hh < hi) raw[i] = load8(src + hh * x.stride_h, m);
            }
            if (!have_angles) {   // after the first loads have been issued
                lane_angles(m, p.inv_freq, pos, cs, sn);
                have_angles = true;
            }
#pragma unroll
            for (int i = 0; i < kRopeUnroll; ++i) {
                if (h + i * step >= hi) break;
                const int hh = h + i * step + w.slot_h;
                float u[8], ss = 0.f;
                unpack8(raw[i], u);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
                const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= r * wt[e];
                turn<kInter>(u, cs, sn);
                if (w.live && hh < hi)
                    store8(out + ((static_cast<size_t>(w.b) * H + hh) * p.N + w.n) * D, m, u);
            }
        }
    };
    walk(p.q, p.q_out, p.Hq, p.q_weight, min(w.h0, p.Hq), min(w.h1, p.Hq));
    walk(p.k, p.k_out, p.Hkv, p.k_weight, max(w.h0, p.Hq) - p.Hq, max(w.h1, p.Hq) - p.Hq);
}

// Backward.  The grid is fixed by the multiprocessor count; a CTA walks items
// item = blockIdx.x, + gridDim.x, ... and keeps the weight gradients of its
// rows in registers (8 columns a thread, q and k), adds them over its row
// slots in shared memory and writes one pair of rows to the workspace.  The
// second kernel adds those rows in order, so the sums repeat bit for bit.
template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads)
fa_qk_norm_rope_bwd_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kSlots = kRopeThreads / kLanes;
    constexpr int kUnroll = 2;
    __shared__ float part[kSlots][D + 4];
    const int step = kSlots / p.token_slots;
    const LaneMap m = lane_map<kInter>(threadIdx.x & (kLanes - 1), p.rot);
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

    for (int item = static_cast<int>(blockIdx.x); item < p.n_items; item += static_cast<int>(gridDim.x)) {
        const Place w = place<D>(p, item);
        const int pos = p.positions ? (w.live ? __ldg(p.positions + static_cast<size_t>(w.b) * p.N + w.n) : 0) : w.n;
        float cs[4], sn[4];
        bool have_angles = false;
        auto walk = [&](const RopeRows& x, const RopeRows& dx, const __nv_bfloat16* dy, int H, const void* weight,
                        float (&dw)[8], int lo, int hi) {
            if (lo >= hi) return;
            const __nv_bfloat16* src = x.data + w.b * x.stride_b + w.n * x.stride_n;
            __nv_bfloat16* dst = dx.data + w.b * dx.stride_b + w.n * dx.stride_n;
            const __nv_bfloat16* dsrc = dy + (static_cast<size_t>(w.b) * H * p.N + w.n) * D;
            float wt[8];
            load_weights(weight, p.weight_bf16, m, wt);
            for (int h = lo; h < hi; h += step * kUnroll) {
                Raw8 rx[kUnroll], rg[kUnroll];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    const int hh = h + i * step + w.slot_h;
                    rx[i] = rg[i] = Raw8{};
                    if (w.live && hh < hi) {
                        rx[i] = load8(src + hh * x.stride_h, m);
                        rg[i] = load8(dsrc + static_cast<size_t>(hh) * p.N * D, m);
                    }
                }
                if (!have_angles) {
                    lane_angles(m, p.inv_freq, pos, cs, sn);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sn[i] = -sn[i];   // R(a)^T = R(-a)
                    have_angles = true;
                }
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    if (h + i * step >= hi) break;
                    const int hh = h + i * step + w.slot_h;
                    float xv[8], g[8], ss = 0.f, hx = 0.f;
                    unpack8(rx[i], xv);
                    unpack8(rg[i], g);
                    turn<kInter>(g, cs, sn);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ss = fmaf(xv[e], xv[e], ss);
                        hx = fmaf(g[e] * wt[e], xv[e], hx);
                    }
                    const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + p.eps);
                    const float c = row_sum<kLanes>(hx) * r * r * (1.f / D);   // mean(h x r) r
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // rows that do not exist were loaded as zeros
                        dw[e] = fmaf(g[e], xv[e] * r, dw[e]);
                        g[e] = r * (g[e] * wt[e] - xv[e] * c);
                    }
                    if (w.live && hh < hi) store8(dst + hh * dx.stride_h, m, g);
                }
            }
        };
        walk(p.q, p.dq, p.dq_out, p.Hq, p.q_weight, dwq, min(w.h0, p.Hq), min(w.h1, p.Hq));
        walk(p.k, p.dk, p.dk_out, p.Hkv, p.k_weight, dwk, max(w.h0, p.Hq) - p.Hq, max(w.h1, p.Hq) - p.Hq);
    }

    const int slot = threadIdx.x / kLanes;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const float* dw = t ? dwk : dwq;
        __syncthreads();
        *reinterpret_cast<float4*>(&part[slot][m.o0]) = make_float4(dw[0], dw[1], dw[2], dw[3]);
        *reinterpret_cast<float4*>(&part[slot][m.o1]) = make_float4(dw[4], dw[5], dw[6], dw[7]);
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) s += part[k][threadIdx.x];
            p.dw_part[(static_cast<size_t>(blockIdx.x) * 2 + t) * D + threadIdx.x] = s;
        }
    }
}

// dw[t][d] = sum over the CTAs' rows, in order: 16 columns a CTA, 16 threads a
// column with every 16th row each, then over the 16 in shared memory.
template <int D>
__global__ void __launch_bounds__(256)
fa_rope_dw_kernel(const float* __restrict__ part, int n_parts, float* __restrict__ dqw, float* __restrict__ dkw) {
    __shared__ float sum[16][17];
    const int col = static_cast<int>(blockIdx.x) * 16 + (threadIdx.x & 15);   // of 2 D
    const int g = threadIdx.x >> 4;
    float s = 0.f;
    for (int i = g; i < n_parts; i += 16) s += part[static_cast<size_t>(i) * 2 * D + col];
    sum[g][threadIdx.x & 15] = s;
    __syncthreads();
    if (g == 0) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += sum[i][threadIdx.x];
        (col < D ? dqw : dkw)[col < D ? col : col - D] = a;
    }
}

// Splits `tokens` x `H` rows over CTAs: token slots a power of two (at most
// the CTA's row slots), and as many head parts as keep about eight CTAs an SM
// busy with at least one unrolled step of heads each.
void rope_plan(RopeParams& p, int D, int sms) {
    const int slots = kRopeThreads / (D / 8);
    int ts = 1;
    while (ts < slots && ts < p.tokens) ts *= 2;
    p.token_slots = ts;
    const long long groups = (p.tokens + ts - 1) / ts;
    const int H = p.Hq + p.Hkv;
    const int per = slots / ts * kRopeUnroll;                 // heads of one unrolled step
    long long parts = (8LL * sms + groups - 1) / groups;
    const long long most = (H + per - 1) / per;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    p.head_parts = static_cast<int>(parts);
    p.n_items = static_cast<int>(groups * parts);
}

template <class F>
cudaError_t rope_dispatch(int D, int inter, F&& go) {
    if (D == 128) return inter ? go(std::integral_constant<int, 128>{}, std::true_type{})
                               : go(std::integral_constant<int, 128>{}, std::false_type{});
    return inter ? go(std::integral_constant<int, 64>{}, std::true_type{})
                 : go(std::integral_constant<int, 64>{}, std::false_type{});
}

}  // namespace

// CTAs of the backward: what fits on the SMs twice over, so that the last
// items spread; the workspace holds one pair of rows for each.
int rope_bwd_ctas(int sms) { return 4 * sms; }

cudaError_t launch_qk_norm_rope(int D, int inter, RopeParams p, int sms, cudaStream_t stream) {
    rope_plan(p, D, sms);
    return rope_dispatch(D, inter, [&](auto d, auto pairs) {
        fa_qk_norm_rope_kernel<decltype(d)::value, decltype(pairs)::value><<<p.n_items, kRopeThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_qk_norm_rope_bwd(int D, int inter, RopeParams p, float* dqw, float* dkw, int sms,
                                    cudaStream_t stream) {
    rope_plan(p, D, sms);
    const int ctas = p.n_items < rope_bwd_ctas(sms) ? p.n_items : rope_bwd_ctas(sms);
    return rope_dispatch(D, inter, [&](auto d, auto pairs) {
        constexpr int kD = decltype(d)::value;
        fa_qk_norm_rope_bwd_kernel<kD, decltype(pairs)::value><<<ctas, kRopeThreads, 0, stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        fa_rope_dw_kernel<kD><<<2 * kD / 16, 256, 0, stream>>>(p.dw_part, ctas, dqw, dkw);
        return cudaGetLastError();
    });
}

}  // namespace fa
