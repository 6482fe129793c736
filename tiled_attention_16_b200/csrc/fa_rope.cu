// fa_rope.cu — RMS norm of each query and key head with the position rotation
// in the same pass, forward and backward (include/fa_rope.h has the formulas).
//
// Bound by HBM: the forward reads and writes 2 bytes an element, the backward
// reads 4 and writes 2.  A row (one head of one token) is held by D / 8 lanes
// with 8 values each, chosen so that both values of every rotated pair are in
// one lane: lane c takes values [4c, 4c+4) and the four partners (or 8c .. 8c+7
// when pairs are neighbours), lanes past the rotated part take 8 neighbours
// with cos = 1, sin = 0.  A thread keeps one token for all the heads it walks,
// so its four angles are reduced (in 64-bit integers) and turned into cos / sin
// once, in registers; no table is read per row.  At these rates instructions
// count as much as bytes (a row passes an SM every 20 cycles): pairs of values
// go through packed fp32 arithmetic, and the weights and the turn are one 2 x 2
// matrix a pair.  8 x 2048 tokens of 64 heads of 128: forward 91 us (5.9 TB/s),
// backward 144 us (5.6 TB/s).
#include "fa_serving.cuh"

#include <climits>

#include <cuda_bf16.h>

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

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

// Turns a position moves by, inv_freq / (2 pi) modulo 1, in units of 2^-64.
// 1 / (2 pi) is the sum of two fp64 numbers, and the product with the first one
// that of its rounding and its error (fma), so what is left modulo 1 is within
// 1.5 units and 2^-106 inv_freq: position 2^31 is off by 2^-32 of a turn, and
// large frequencies keep their fraction (one fp64 product alone loses 2^-53 of
// itself a position: 0.07 rad at 2^31 for 3e5, all of it from 1e17 on).
__device__ __forceinline__ unsigned long long turn_rate(float inv_freq) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18, kUnits = 18446744073709551616.0;   // 2^64
    const double f = inv_freq, t = f * kHi, e = fma(f, kLo, fma(f, kHi, -t));
    return static_cast<unsigned long long>(__double2ll_rn((t - rint(t)) * kUnits)) +
           static_cast<unsigned long long>(__double2ll_rn((e - rint(e)) * kUnits));
}

// cos and sin of the lane's four angles.  position x rate wraps modulo a turn
// by itself in integers; its upper 32 bits are the turn in [-1/2, 1/2), and
// fp32 sincospi does the rest.
__device__ __forceinline__ void lane_angles(const unsigned long long (&rate)[4], int pos, float2 (&cs)[2],
                                            float2 (&sn)[2]) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned long long t = rate[i] * static_cast<unsigned long long>(static_cast<long long>(pos));
        sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 4.656612873077393e-10f, &s[i], &c[i]);   // 2^-31
    }
    cs[0] = make_float2(c[0], c[1]);
    cs[1] = make_float2(c[2], c[3]);
    sn[0] = make_float2(s[0], s[1]);
    sn[1] = make_float2(s[2], s[3]);
}

// A lane's 8 values as float pairs that the packed fp32 instructions take.
// Half-split: lo[i], hi[i] hold the values (2i, 2i + 1) of the first and second
// group, partners in the same places.  Interleaved: the even (lo) and odd (hi)
// values of the neighbouring pairs, two pairs in each.
struct Vals {
    float2 lo[2], hi[2];
};

__device__ __forceinline__ float2 f2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The same as they lie in memory.
template <bool kInter>
struct Raw8 {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* row, const LaneMap& m) {
        if constexpr (kInter) {
            w = *reinterpret_cast<const uint4*>(row + m.o0);
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(row + m.o0), b = *reinterpret_cast<const uint2*>(row + m.o1);
            w = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    __device__ __forceinline__ Vals vals() const {
        const float2 a = f2(w.x), b = f2(w.y), c = f2(w.z), d = f2(w.w);
        Vals v;
        if constexpr (kInter) {
            v.lo[0] = make_float2(a.x, b.x);
            v.hi[0] = make_float2(a.y, b.y);
            v.lo[1] = make_float2(c.x, d.x);
            v.hi[1] = make_float2(c.y, d.y);
        } else {
            v.lo[0] = a;
            v.lo[1] = b;
            v.hi[0] = c;
            v.hi[1] = d;
        }
        return v;
    }
};

template <bool kInter>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const LaneMap& m, const Vals& v) {
    if constexpr (kInter) {
        *reinterpret_cast<uint4*>(p + m.o0) =
            make_uint4(pack_bf16x2(v.lo[0].x, v.hi[0].x), pack_bf16x2(v.lo[0].y, v.hi[0].y),
                       pack_bf16x2(v.lo[1].x, v.hi[1].x), pack_bf16x2(v.lo[1].y, v.hi[1].y));
    } else {
        *reinterpret_cast<uint2*>(p + m.o0) = make_uint2(pack_bf16x2(v.lo[0].x, v.lo[0].y), pack_bf16x2(v.lo[1].x, v.lo[1].y));
        *reinterpret_cast<uint2*>(p + m.o1) = make_uint2(pack_bf16x2(v.hi[0].x, v.hi[0].y), pack_bf16x2(v.hi[1].x, v.hi[1].y));
    }
}

// The column of value e (lo, then hi) of the lane.
template <bool kInter>
__device__ __forceinline__ int column(const LaneMap& m, int e) {
    if (kInter) return m.o0 + 2 * (e & 3) + (e >> 2);
    return (e < 4 ? m.o0 : m.o1 - 4) + e;
}

__device__ __forceinline__ float2 neg(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <bool kInter>
__device__ __forceinline__ Vals load_weights(const void* w, int bf16, const LaneMap& m) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = column<kInter>(m, e);
        v[e] = bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[d])
                    : reinterpret_cast<const float*>(w)[d];
    }
    Vals r;
    r.lo[0] = make_float2(v[0], v[1]);
    r.lo[1] = make_float2(v[2], v[3]);
    r.hi[0] = make_float2(v[4], v[5]);
    r.hi[1] = make_float2(v[6], v[7]);
    return r;
}

// Copy of `bytes` (4 or 16) to shared memory, zeros where `real` is false.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool real) {
    const uint32_t n = real ? kBytes : 0u;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int k = kLanes / 2; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    return x;
}

// Where a thread stands in the CTA's walk over items blockIdx.x, + gridDim.x,
// ... An item is a group of token_slots tokens and a part of q's heads (items
// below items_q) or k's; the CTA has 256 / (D / 8) row slots, token_slots of
// them for different tokens and the rest for different heads of the same
// tokens, so that few tokens still fill a CTA.  A step is kHeads heads of every
// head slot.
template <int D, int kHeads>
struct Cursor {
    int item, h, h1;     // CTA-uniform: item (INT_MAX: past the end), first head of the step, end of the part
    int head, end;       // this thread's first head of the step and its end (none where its token does not exist)
    unsigned b, n;       // its token
    bool is_k;

    __device__ __forceinline__ void enter(const RopeParams& p, int it) {
        if (it >= p.n_items) {
            item = INT_MAX;
            return;
        }
        item = it;
        is_k = it >= p.items_q;
        const unsigned j = static_cast<unsigned>(is_k ? it - p.items_q : it);
        const unsigned parts = static_cast<unsigned>(is_k ? p.parts_k : p.parts_q);
        const unsigned group = j / parts, part = j - group * parts;
        const unsigned H = static_cast<unsigned>(is_k ? p.Hkv : p.Hq);
        h = static_cast<int>(H * part / parts);
        h1 = static_cast<int>(H * (part + 1) / parts);
        const unsigned slot = threadIdx.x / (D / 8);
        const unsigned t = group * static_cast<unsigned>(p.token_slots) + (slot & (p.token_slots - 1));
        const bool live = t < static_cast<unsigned>(p.tokens);
        b = live ? t / static_cast<unsigned>(p.N) : 0u;
        n = live ? t - b * static_cast<unsigned>(p.N) : 0u;
        head = h + static_cast<int>(slot / static_cast<unsigned>(p.token_slots));
        end = live ? h1 : 0;
    }
    // past this step; true when that entered another item
    __device__ __forceinline__ bool advance(const RopeParams& p, int hs) {
        h += kHeads * hs;
        head += kHeads * hs;
        if (h < h1) return false;
        enter(p, item + static_cast<int>(gridDim.x));
        return true;
    }
    // this thread's row of head `head` in a view, and in a contiguous [B, H, N, D]
    __device__ __forceinline__ __nv_bfloat16* in_view(const RopeRows& x) const {
        return x.data + b * x.stride_b + n * x.stride_n + head * x.stride_h;
    }
    __device__ __forceinline__ size_t in_heads(const RopeParams& p) const {
        return ((static_cast<size_t>(b) * static_cast<unsigned>(is_k ? p.Hkv : p.Hq) + static_cast<unsigned>(head)) *
                    static_cast<unsigned>(p.N) + n) * D;
    }
};

__device__ __forceinline__ float2 square_sum(const Vals& x) {
    float2 s = __fmul2_rn(x.lo[0], x.lo[0]);
    s = __ffma2_rn(x.lo[1], x.lo[1], s);
    s = __ffma2_rn(x.hi[0], x.hi[0], s);
    return __ffma2_rn(x.hi[1], x.hi[1], s);
}

// Rows of a forward step a thread loads before it uses the first.
constexpr int kFwdHeads = 4;
constexpr int kFwdCtas = 4;

template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kFwdCtas)
fa_qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;
    const int hs = kRopeThreads / kLanes / p.token_slots;        // head slots
    const LaneMap m = lane_map<kInter>(threadIdx.x & (kLanes - 1), p.rot);
    unsigned long long rate[4] = {0ull, 0ull, 0ull, 0ull};
    if (m.pair0 >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rate[i] = turn_rate(__ldg(p.inv_freq + m.pair0 + i));
    }
    Cursor<D, kFwdHeads> at{};
    at.enter(p, static_cast<int>(blockIdx.x));
    while (at.item != INT_MAX) {
        const RopeRows& x = at.is_k ? p.k : p.q;
        const long long x_head = x.stride_h * hs, y_head = static_cast<long long>(p.N) * D * hs;
        const __nv_bfloat16* src = at.in_view(x);
        __nv_bfloat16* dst = (at.is_k ? p.k_out : p.q_out) + at.in_heads(p);
        const int pos = p.positions ? __ldg(p.positions + static_cast<size_t>(at.b) * p.N + at.n) : static_cast<int>(at.n);
        const int item = at.item;
        Raw8<kInter> raw[kFwdHeads];
        auto load = [&] {
#pragma unroll
            for (int k = 0; k < kFwdHeads; ++k) {
                raw[k].zero();
                if (at.head + k * hs < at.end) raw[k].load(src + k * x_head, m);
            }
        };
        load();
        // the turn and the weight as one 2 x 2 matrix a pair:
        // (y_lo, y_hi) = r (x_lo wc_lo + x_hi ws_hi, x_hi wc_hi + x_lo ws_lo)
        float2 wc_lo[2], wc_hi[2], ws_lo[2], ws_hi[2];
        {
            const Vals wt = load_weights<kInter>(at.is_k ? p.k_weight : p.q_weight, p.weight_bf16, m);
            float2 cs[2], sn[2];
            lane_angles(rate, pos, cs, sn);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                wc_lo[i] = __fmul2_rn(wt.lo[i], cs[i]);
                wc_hi[i] = __fmul2_rn(wt.hi[i], cs[i]);
                ws_lo[i] = __fmul2_rn(wt.lo[i], sn[i]);
                ws_hi[i] = neg(__fmul2_rn(wt.hi[i], sn[i]));
            }
        }
        for (;;) {
#pragma unroll
            for (int k = 0; k < kFwdHeads; ++k) {
                if (at.h + k * hs >= at.h1) break;   // CTA-uniform
                const Vals x8 = raw[k].vals();
                const float2 ss = square_sum(x8);
                const float2 r = both(rsqrtf(row_sum<kLanes>(ss.x + ss.y) * (1.f / D) + p.eps));
                Vals y;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y.lo[i] = __fmul2_rn(__ffma2_rn(x8.hi[i], ws_hi[i], __fmul2_rn(x8.lo[i], wc_lo[i])), r);
                    y.hi[i] = __fmul2_rn(__ffma2_rn(x8.lo[i], ws_lo[i], __fmul2_rn(x8.hi[i], wc_hi[i])), r);
                }
                if (at.head + k * hs < at.end) store8<kInter>(dst + k * y_head, m, y);
            }
            at.advance(p, hs);
            if (at.item != item) break;
            src += kFwdHeads * x_head;
            dst += kFwdHeads * y_head;
            load();
        }
    }
}

// Backward.  Its rows (x and dy) come through shared memory: every warp has a
// ring of its own that asynchronous copies keep kStages - 1 steps ahead, across
// the CTA's items, so that the loads in flight cost no registers (loaded
// straight into registers: 3.9 TB/s).
//
// A CTA keeps the weight gradients of its rows in registers (8 columns a
// thread; q's first, then k's, since items are walked in order), adds them over
// its row slots in shared memory and writes one pair of rows to the workspace.
// The grid is fixed by the multiprocessor count and a second kernel adds those
// rows in order, so the sums repeat bit for bit.
constexpr int kBwdHeads = 2;
constexpr int kBwdCtas = 3;

template <int D>
struct RopeRing {
    static constexpr int kRows = 256 / D;                          // rows of a warp at a time
    static constexpr int kStages = 3;
    static constexpr int kTensor = kRows * D * 2;                  // their bytes of x (or of dy): 512
    static constexpr int kStage = kTensor * 2 * kBwdHeads + 16;    // a step's, and the rows' positions
    static constexpr int kPart = kRopeWarps * kStages * kStage;    // [row slots][D + 4] fp32
    static constexpr int kBytes = kPart + kRopeThreads / (D / 8) * (D + 4) * 4;
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kBwdCtas)
fa_qk_norm_rope_bwd_kernel(const RopeParams p) {
    using Ring = RopeRing<D>;
    constexpr int kLanes = D / 8;
    constexpr int kSlots = kRopeThreads / kLanes;
    constexpr int kStages = Ring::kStages;
    extern __shared__ __align__(16) uint8_t ring[];
    const int hs = kSlots / p.token_slots;                       // head slots
    const int c = threadIdx.x & (kLanes - 1);
    const int row = (threadIdx.x & 31) / kLanes;                 // row of the warp
    const LaneMap m = lane_map<kInter>(c, p.rot);
    uint8_t* mine = ring + (threadIdx.x >> 5) * kStages * Ring::kStage;
    const int copy_at = row * (D * 2) + c * 16;

    // loads: this thread's 16 bytes of each row of the next step
    Cursor<D, kBwdHeads> ld{}, at;
    const __nv_bfloat16 *lx = nullptr, *ldy = nullptr;
    long long lx_head = 0;
    const long long n_head = static_cast<long long>(p.N) * D * hs;
    bool ld_first = true;
    auto point_loads = [&] {
        if (ld.item == INT_MAX) return;
        const RopeRows& x = ld.is_k ? p.k : p.q;
        lx_head = x.stride_h * hs;
        lx = ld.in_view(x) + c * 8;
        ldy = (ld.is_k ? p.dk_out : p.dq_out) + ld.in_heads(p) + c * 8;
    };
    auto issue = [&](int st) {
        if (ld.item != INT_MAX) {
            uint8_t* dst = mine + st * Ring::kStage + copy_at;
#pragma unroll
            for (int k = 0; k < kBwdHeads; ++k) {
                const bool real = ld.head + k * hs < ld.end;
                copy_async<16>(dst + k * Ring::kTensor, lx, real);
                copy_async<16>(dst + (kBwdHeads + k) * Ring::kTensor, ldy, real);
                lx += lx_head;
                ldy += n_head;
            }
            if (ld_first && c == 0 && p.positions)
                copy_async<4>(mine + st * Ring::kStage + Ring::kStage - 16 + row * 4,
                              p.positions + static_cast<size_t>(ld.b) * p.N + ld.n, true);
            ld_first = ld.advance(p, hs);
            if (ld_first) point_loads();
        }
        copy_commit();
    };
    ld.enter(p, static_cast<int>(blockIdx.x));
    at = ld;
    point_loads();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s);

    unsigned long long rate[4] = {0ull, 0ull, 0ull, 0ull};
    if (m.pair0 >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rate[i] = turn_rate(__ldg(p.inv_freq + m.pair0 + i));
    }
    bool in_k = at.is_k;
    Vals wt = load_weights<kInter>(in_k ? p.k_weight : p.q_weight, p.weight_bf16, m);
    Vals dw;
    dw.lo[0] = dw.lo[1] = dw.hi[0] = dw.hi[1] = make_float2(0.f, 0.f);

    float(*part)[D + 4] = reinterpret_cast<float(*)[D + 4]>(ring + Ring::kPart);
    auto flush = [&](int t) {
        const float v[8] = {dw.lo[0].x, dw.lo[0].y, dw.lo[1].x, dw.lo[1].y, dw.hi[0].x, dw.hi[0].y, dw.hi[1].x, dw.hi[1].y};
#pragma unroll
        for (int e = 0; e < 8; ++e) part[threadIdx.x / kLanes][column<kInter>(m, e)] = v[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) s += part[k][threadIdx.x];
            p.dw_part[(static_cast<size_t>(blockIdx.x) * 2 + t) * D + threadIdx.x] = s;
        }
        __syncthreads();
        dw.lo[0] = dw.lo[1] = dw.hi[0] = dw.hi[1] = make_float2(0.f, 0.f);
    };

    __nv_bfloat16* out = nullptr;   // this thread's rows of the step in dx
    long long out_head = 0;
    float2 cs[2], sn[2];
    bool entered = true;
    int st = 0;
    while (at.item != INT_MAX) {
        copy_wait<kStages - 2>();
        __syncwarp();   // every lane's copies of this step; and the stage before it has been read
        issue(st == 0 ? kStages - 1 : st - 1);
        const uint8_t* stage = mine + st * Ring::kStage;
        if (entered) {  // CTA-uniform
            if (at.is_k != in_k) {
                flush(0);
                in_k = true;
                wt = load_weights<kInter>(p.k_weight, p.weight_bf16, m);
            }
            const int pos = p.positions ? *reinterpret_cast<const int*>(stage + Ring::kStage - 16 + row * 4)
                                        : static_cast<int>(at.n);
            lane_angles(rate, pos, cs, sn);
            const RopeRows& dx = in_k ? p.dk : p.dq;
            out_head = dx.stride_h * hs;
            out = at.in_view(dx);
        }
#pragma unroll
        for (int k = 0; k < kBwdHeads; ++k) {
            if (k > 0 && at.h + k * hs >= at.h1) break;   // CTA-uniform
            Raw8<kInter> raw;
            raw.load(reinterpret_cast<const __nv_bfloat16*>(stage + k * Ring::kTensor + row * (D * 2)), m);
            const Vals x = raw.vals();
            raw.load(reinterpret_cast<const __nv_bfloat16*>(stage + (kBwdHeads + k) * Ring::kTensor + row * (D * 2)), m);
            const Vals dy = raw.vals();
            const float2 ss = square_sum(x);
            Vals g, t, y;      // R^T dy; g x; dx
            float2 hx = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                g.lo[i] = __ffma2_rn(dy.hi[i], sn[i], __fmul2_rn(dy.lo[i], cs[i]));
                g.hi[i] = __ffma2_rn(dy.lo[i], neg(sn[i]), __fmul2_rn(dy.hi[i], cs[i]));
                t.lo[i] = __fmul2_rn(g.lo[i], x.lo[i]);
                t.hi[i] = __fmul2_rn(g.hi[i], x.hi[i]);
                hx = __ffma2_rn(t.lo[i], wt.lo[i], hx);
                hx = __ffma2_rn(t.hi[i], wt.hi[i], hx);
            }
            const float r = rsqrtf(row_sum<kLanes>(ss.x + ss.y) * (1.f / D) + p.eps);
            const float2 r2 = both(r), mk = both(-(row_sum<kLanes>(hx.x + hx.y) * r * r * (1.f / D)));   // -mean(h x r) r
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // a row that does not exist was copied as zeros
                dw.lo[i] = __ffma2_rn(t.lo[i], r2, dw.lo[i]);
                dw.hi[i] = __ffma2_rn(t.hi[i], r2, dw.hi[i]);
                y.lo[i] = __fmul2_rn(__ffma2_rn(x.lo[i], mk, __fmul2_rn(g.lo[i], wt.lo[i])), r2);
                y.hi[i] = __fmul2_rn(__ffma2_rn(x.hi[i], mk, __fmul2_rn(g.hi[i], wt.hi[i])), r2);
            }
            if (at.head + k * hs < at.end) store8<kInter>(out, m, y);
            out += out_head;
        }
        if (++st == kStages) st = 0;
        entered = at.advance(p, hs);
    }
    // a CTA without items of one kind leaves zeros for it
    if (in_k) {
        flush(1);
        if (static_cast<int>(blockIdx.x) >= p.items_q) flush(0);
    } else {
        flush(0);
        flush(1);
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

// Items: token slots a power of two (at most the CTA's row slots), each
// tensor's heads in parts of up to `s` steps.  Short parts spread evenly over
// the CTAs, but entering an item (angles, addresses) costs about as much as
// three rows a thread; s is the one whose busiest CTA has least to do.
// Returns the CTAs to launch.
int rope_plan(RopeParams& p, int D, int heads, int resident) {
    const int slots = kRopeThreads / (D / 8);
    int ts = 1;
    while (ts < slots && ts < p.tokens) ts *= 2;
    p.token_slots = ts;
    const long long groups = (p.tokens + ts - 1) / ts;
    const int per = heads * (slots / ts);
    const long long steps_q = (p.Hq + per - 1) / per, steps_k = (p.Hkv + per - 1) / per;
    long long best = -1;
    for (long long s = 1; s <= (steps_q > steps_k ? steps_q : steps_k); ++s) {
        const long long pq = (steps_q + s - 1) / s, pk = (steps_k + s - 1) / s;
        const long long rounds_q = (groups * pq + resident - 1) / resident;
        const long long rounds = (groups * (pq + pk) + resident - 1) / resident;
        const long long cost = rounds_q * (heads * ((steps_q + pq - 1) / pq) + 3) +
                               (rounds - rounds_q) * (heads * ((steps_k + pk - 1) / pk) + 3);
        if (best < 0 || cost <= best) {
            best = cost;
            p.parts_q = static_cast<int>(pq);
            p.parts_k = static_cast<int>(pk);
        }
    }
    p.items_q = static_cast<int>(groups * p.parts_q);
    p.n_items = p.items_q + static_cast<int>(groups * p.parts_k);
    return p.n_items < resident ? p.n_items : resident;
}

template <class F>
cudaError_t rope_dispatch(int D, int inter, F&& go) {
    if (D == 128) return inter ? go(std::integral_constant<int, 128>{}, std::true_type{})
                               : go(std::integral_constant<int, 128>{}, std::false_type{});
    return inter ? go(std::integral_constant<int, 64>{}, std::true_type{})
                 : go(std::integral_constant<int, 64>{}, std::false_type{});
}

}  // namespace

// CTAs of the backward: those resident at once, one pair of rows of the
// workspace each.
int rope_bwd_ctas(int sms) { return kBwdCtas * sms; }

cudaError_t launch_qk_norm_rope(int D, int inter, RopeParams p, int sms, cudaStream_t stream) {
    const int ctas = rope_plan(p, D, kFwdHeads, kFwdCtas * sms);
    return rope_dispatch(D, inter, [&](auto d, auto pairs) {
        fa_qk_norm_rope_kernel<decltype(d)::value, decltype(pairs)::value><<<ctas, kRopeThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_qk_norm_rope_bwd(int D, int inter, RopeParams p, float* dqw, float* dkw, int sms,
                                    cudaStream_t stream) {
    const int ctas = rope_plan(p, D, kBwdHeads, rope_bwd_ctas(sms));
    return rope_dispatch(D, inter, [&](auto d, auto pairs) {
        constexpr int kD = decltype(d)::value;
        auto kern = fa_qk_norm_rope_bwd_kernel<kD, decltype(pairs)::value>;
        static SmemOptIn opt_in;
        cudaError_t e = opt_in.set(reinterpret_cast<const void*>(kern), RopeRing<kD>::kBytes);
        if (e != cudaSuccess) return e;
        kern<<<ctas, kRopeThreads, RopeRing<kD>::kBytes, stream>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        fa_rope_dw_kernel<kD><<<2 * kD / 16, 256, 0, stream>>>(p.dw_part, ctas, dqw, dkw);
        return cudaGetLastError();
    });
}

}  // namespace fa
