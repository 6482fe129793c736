// fa_prefix.cu — attention of a whole batch over one shared prefix
// (include/fa_cache.h, n_prefix > 0).
//
// All B * (Hq / Hkv) * Nq query rows of a K/V head meet the prefix's keys as
// one matrix, so K and V are read once for the batch and the products run on
// tcgen05 with the rows as the M axis.  Every key is visible to every row.
// The key tiles (128 keys) of all (K/V head, block of rows) units are laid end
// to end and each CTA, one an SM, takes an equal run of them; a run may begin
// and end inside a unit, and each part of a unit leaves fp32 O / l and the LSE
// for the combine kernel, in slot (CTA + unit).
//
// Two 128 x 128 score blocks are in flight in a CTA, one per softmax
// warpgroup, so that the tensor core works on one while the other's
// exponentials are taken:
//   kRows2    a unit is 256 rows and both blocks use the same key tile (three
//             quarters of the shared-memory fill per product)
//   otherwise a unit is 128 rows, the blocks take alternate key tiles, and their
//             two accumulators are joined as they leave tensor memory
// Up to 128 rows the work is bound by HBM whichever rows are real: a 64 KB
// key tile costs about 1000 tensor cycles and, at the copy rate, 2800 cycles
// (8 K/V heads, 128 rows: 32768 keys more take 19.4 us, 6.9 TB/s; the first 32768
// 29 us, 4.6 TB/s with the start and the results).  512 rows of the same take
// 67 us: 2.15 us a key tile in the main loop, 70% of the burst rate of a library
// product, with the SM clock at 1.6 to 1.75 GHz under it.
//
// Warp roles (320 threads) and tensor memory as in fa_fwd.cu:
//   warps 0-3, 4-7  Q rows to shared memory, softmax, epilogue of block 0, 1
//   warp  8         MMA issuer     warp 9  TMA producer of the K/V ring
//   S0 | S1 | O0 | O1, 128 columns each; P over S as packed bf16 (2^-8 of each
//   weight, as in the forward: V is bf16, and P in two bf16 parts would be half
//   as many products again)
#include "fa_serving.cuh"

#include <cuda_bf16.h>

namespace fa {

namespace {

constexpr int kPfThreads = 320;
constexpr float kPfRescale = 8.0f;   // the O rescale is skipped while the row max grows by less (log2 units)

enum PfSite { kPfQ = 24, kPfK = 25, kPfEmpty = 26, kPfS = 27, kPfP = 28, kPfO = 29, kPfDrain = 30 };

template <int D, bool kRows2>
struct PfLayout {
    static constexpr int kTileBytes = kTileM * D * 2;
    static constexpr int kAtomBytes = kTileM * 128;
    static constexpr int kQTiles = kRows2 ? 2 : 1;
    static constexpr int kStages = D == 64 ? 4 : (kRows2 ? 2 : 3);
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kQTiles * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kMl = kV + kStages * kTileBytes;              // two floats a row
    static constexpr int kBar = kMl + (kRows2 ? 0 : kTileM * 8);
    static constexpr int kMisc = kBar + (1 + 2 * kStages + 2 + 2 + 1 + 1 + 3) * 8;
    static constexpr int kBytes = kMisc + 16;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "one CTA must fit");
};

__device__ __forceinline__ float pf_lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void pf_drain(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return;
        if ((it & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(&g_status, 1u << kPfDrain);
            return;
        }
    }
}

// A part of a unit: key tiles [t0, t0 + n) of unit u.
struct Part {
    int u, t0, n;
};

__device__ __forceinline__ bool next_part(const PrefixParams& p, int& x, int x1, Part& w) {
    if (x >= x1) return false;
    w.u = x / p.n_tiles;
    w.t0 = x - w.u * p.n_tiles;
    w.n = min(x1 - x, p.n_tiles - w.t0);
    x += w.n;
    return true;
}

template <int D, bool kRows2>
__global__ void __launch_bounds__(kPfThreads, 1)
fa_prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const PrefixParams p) {
    using L = PfLayout<D, kRows2>;
    constexpr int kStages = L::kStages;
    constexpr int kTileSteps = kRows2 ? 2 : 1;   // score blocks that use one key tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* kv_full = q_full + 1;
    uint64_t* kv_empty = kv_full + kStages;
    uint64_t* s_full = kv_empty + kStages;   // [2]
    uint64_t* p_full = s_full + 2;           // [2]
    uint64_t* part_done = p_full + 2;        // every MMA of the part has completed
    uint64_t* drain = part_done + 1;
    uint64_t* ml_full = drain + 1;           // alternate key tiles: (m, l) of block 1 are in place,
    uint64_t* f_full = ml_full + 1;          // the factors of both accumulators are,
    uint64_t* o_read = f_full + 1;           // both accumulators have been read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 2 * kTileM);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], kTileM);
        }
        mbar_init(part_done, 1);
        mbar_init(drain, 1);
        mbar_init(ml_full, kTileM);
        mbar_init(f_full, kTileM);
        mbar_init(o_read, 2 * kTileM);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_launch_dependents();   // the cache part needs nothing from here and may take SMs as they come free

    const int total = p.Hkv * p.n_rowtiles * p.n_tiles;
    const int x0 = static_cast<int>(static_cast<long long>(total) * blockIdx.x / gridDim.x);
    const int x1 = static_cast<int>(static_cast<long long>(total) * (blockIdx.x + 1) / gridDim.x);

    if (warp == 9) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            int gk = 0, issued = 0;
            bool ok = true;
            Part w;
            for (int x = x0; ok && next_part(p, x, x1, w);) {
                const int hkv = w.u / p.n_rowtiles;
                for (int j = 0; j < w.n; ++j, ++gk) {
                    const int st = gk % kStages;
                    if (gk >= kStages && !(ok = mbar_wait(&kv_empty[st], ((gk / kStages) - 1) & 1, abort_flag, kPfEmpty)))
                        break;
                    mbar_arrive_expect_tx(&kv_full[st], 2 * L::kTileBytes);
                    for (int a = 0; a < D / 64; ++a)
                        tma_load_3d(smem + L::kK + st * L::kTileBytes + a * L::kAtomBytes, &tmK, &kv_full[st], a * 64,
                                    (w.t0 + j) * kTileN, hkv);
                    for (int a = 0; a < D / 64; ++a)
                        tma_load_3d(smem + L::kV + st * L::kTileBytes + a * L::kAtomBytes, &tmV, &kv_full[st], a * 64,
                                    (w.t0 + j) * kTileN, hkv);
                    issued = gk + 1;
                }
            }
            for (int t = (issued > kStages ? issued - kStages : 0); t < issued; ++t)
                pf_drain(&kv_full[t % kStages], (t / kStages) & 1);
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA issuer
        // Step i of a part is one score block: block i & 1 over key tile i, or,
        // with two row tiles, key tile i / 2.
        if (lane == 0) {
            constexpr uint32_t kIdS = idesc_bf16_f32(kTileM, kTileN, 0, 0);
            constexpr uint32_t kIdPV = idesc_bf16_f32(kTileM, D, 0, 1);
            // Descriptors of the first k-step; the others are a constant number of
            // 16-byte units on, added to the address field (this thread shares its
            // scheduler with softmax warps, so every instruction between two MMAs
            // counts).
            const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::kQ), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::kK), 16, 1024);
            const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::kV), L::kAtomBytes, 1024);
            constexpr uint32_t kTileUnits = L::kTileBytes / 16;
            bool ok = true;
            int gk = 0;         // key tiles of earlier parts
            int waited = 0;     // key tiles whose arrival has been waited for
            int np[2] = {0, 0}; // P blocks consumed
            int parts = 0;
            Part w;
            auto issue_s = [&](int i) -> bool {
                const int s = i & 1, G = gk + i / kTileSteps, st = G % kStages;
                if (G >= waited) {
                    if (!mbar_wait(&kv_full[st], (G / kStages) & 1, abort_flag, kPfK)) return false;
                    waited = G + 1;
                }
                tc_fence_after();
                const uint64_t qa = q_desc + (kRows2 ? s * kTileUnits : 0), ka = k_desc + st * kTileUnits;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * L::kAtomBytes + (kk & 3) * 32) / 16;
                    mma_ss(tmem + s * 128, qa + off, ka + off, kIdS, kk > 0);
                }
                tc_commit(&s_full[s]);
                return true;
            };
            for (int x = x0; ok && next_part(p, x, x1, w);) {
                const int n_steps = w.n * kTileSteps;
                if (!(ok = mbar_wait(q_full, parts & 1, abort_flag, kPfQ))) break;
                tc_fence_after();
                ok = issue_s(0) && (n_steps < 2 || issue_s(1));
                for (int i = 0; ok && i < n_steps; ++i) {
                    const int s = i & 1, G = gk + i / kTileSteps, st = G % kStages;
                    if (!(ok = mbar_wait(&p_full[s], np[s] & 1, abort_flag, kPfP))) break;
                    ++np[s];
                    tc_fence_after();
                    const uint64_t va = v_desc + st * kTileUnits;
#pragma unroll
                    for (int kk = 0; kk < kTileN / 16; ++kk)
                        mma_ts(tmem + 256 + s * 128, tmem + s * 128 + kk * 8, va + kk * (2048 / 16), kIdPV, (i > 1 || kk > 0));
                    if (i % kTileSteps == kTileSteps - 1) tc_commit(&kv_empty[st]);
                    if (i + 2 < n_steps) ok = issue_s(i + 2);
                }
                if (!ok) break;
                tc_commit(part_done);
                gk += w.n;
                ++parts;
            }
            tc_commit(drain);
            pf_drain(drain, 0);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int s = warp >> 2;
        const int r = ((warp & 3) << 5) + lane;        // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
        const uint32_t tS = tmem + lane_off + s * 128;
        const uint32_t tO = tmem + lane_off + 256 + s * 128;
        const float c = p.scale_log2;
        const int R = p.G * p.Nq;                      // rows of one sequence
        const int n_rows = p.B * R;                    // rows of one K/V head
        // Q rows to shared memory, D / 8 lanes a row: a warp loads the 32 rows of its
        // lane quarter of its own tile (kRows2), or 16 of them (both warpgroups load
        // the one tile)
        auto load_q = [&](int u) {
            const int hkv = u / p.n_rowtiles;
            constexpr int kLanes = D / 8, kStep = 32 / kLanes;
            const int rw = (kRows2 ? (warp & 3) * 32 : warp * 16) + lane / kLanes, ch = lane % kLanes;
            const int first = (u - hkv * p.n_rowtiles) * p.rows_unit + (kRows2 ? s * kTileM : 0) + rw;
            uint8_t* dst = smem + L::kQ + (kRows2 ? s * L::kTileBytes : 0);
            constexpr int kLoads = (kRows2 ? 32 : 16) / kStep;
            uint4 v[kLoads];   // all in flight at once
            int b = first / R, in = first - b * R;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (first + k * kStep < n_rows)
                    v[k] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                                (static_cast<size_t>(b * p.Hkv + hkv) * R + in) * D) +
                                 ch);
                for (in += kStep; in >= R; in -= R) ++b;
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                *reinterpret_cast<uint4*>(dst + sw128_offset(rw + k * kStep, ch * 8, kTileM)) = v[k];
            fence_proxy_async_smem();
            mbar_arrive(q_full);
        };
        bool ok = true;
        int cs = 0;       // score blocks of this warpgroup so far
        int parts = 0;
        int x = x0;
        Part w;
        bool more = next_part(p, x, x1, w);
        if (more) load_q(w.u);
        while (more) {
            const int n_here = kRows2 ? w.n : (w.n + 1 - s) / 2;   // this block's key tiles of the part
            float m_used = -INFINITY;
            float l = 0.f;
            for (int j = 0; j < n_here; ++j, ++cs) {
                ok = mbar_wait(&s_full[s], cs & 1, abort_flag, kPfS);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t sr[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sr[q]);
                tmem_ld_wait();
                float* sv = reinterpret_cast<float*>(&sr[0][0]);
                const int kv0 = (w.t0 + (kRows2 ? j : 2 * j + s)) * kTileN;
                if (kv0 + kTileN > p.Np) {
                    const int hi = p.Np - kv0;
#pragma unroll
                    for (int cix = 0; cix < 128; ++cix) sv[cix] = (cix < hi) ? sv[cix] : -INFINITY;
                }
                float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                for (int cix = 4; cix < 124; cix += 8) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) mx4[t] = fmax3(mx4[t], sv[cix + t], sv[cix + 4 + t]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) mx4[t] = fmaxf(mx4[t], sv[124 + t]);
                const float mx = fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                const float m_new = fmaxf(m_used, mx * c);
                const bool rescale = __any_sync(0xffffffffu, m_new > m_used + kPfRescale);
                float alpha = 1.f;
                if (rescale) {
                    alpha = (m_new == -INFINITY) ? 1.f : ex2(m_used - m_new);
                    l *= alpha;
                    m_used = m_new;
                }
                const float msub = (m_used == -INFINITY) ? 0.f : m_used;
                const float2 c2 = make_float2(c, c);
                const float2 nm2 = make_float2(-msub, -msub);
                float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                static_for<0, 4>([&](auto qq) {
                    constexpr int qtr = decltype(qq)::value;
                    uint32_t pk[16];
                    static_for<0, 16>([&](auto tt) {
                        constexpr int t = decltype(tt)::value;
                        constexpr int cix = qtr * 32 + 2 * t;
                        const float2 y = __ffma2_rn(make_float2(sv[cix], sv[cix + 1]), c2, nm2);
                        const float p0 = ex2(y.x);
                        const float p1 = ex2(y.y);
                        ls2[t & 1] = __fadd2_rn(ls2[t & 1], make_float2(p0, p1));
                        pk[t] = pack_bf16x2(p0, p1);
                    });
                    tmem_st16(tS + qtr * 16, pk);
                });
                l += (ls2[0].x + ls2[0].y) + (ls2[1].x + ls2[1].y);
                if (rescale && j > 0) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t orow[32];
                        tmem_ld32(tO + q * 32, orow);
                        tmem_ld_wait();
#pragma unroll
                        for (int t = 0; t < 32; ++t) orow[t] = __float_as_uint(__uint_as_float(orow[t]) * alpha);
                        tmem_st32(tO + q * 32, orow);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[s]);
            }
            if (!ok) break;
            ok = mbar_wait(part_done, parts & 1, abort_flag, kPfO);
            ++parts;
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            // the next part's Q goes out before this part's results: nothing
            // reads the old one any more, and the issuer can start on it
            const Part done = w;
            more = next_part(p, x, x1, w);
            if (more) load_q(w.u);
            const int hkv = done.u / p.n_rowtiles;
            const int row = (done.u - hkv * p.n_rowtiles) * p.rows_unit + (kRows2 ? s * kTileM : 0) + r;
            const size_t prow = static_cast<size_t>(blockIdx.x + done.u) * p.rows_unit + (kRows2 ? s * kTileM : 0) + r;
            const bool valid = row < n_rows;
            // Factors of this row's accumulators.  With alternate key tiles both blocks
            // hold part of the same rows (the second nothing, when the part is one key
            // tile); a warp reaches the other block's accumulator of its rows too, so
            // each warpgroup joins half of the columns.
            float f0 = 1.f / l, f1 = 0.f, lse;
            const bool join = !kRows2 && done.n > 1;
            if constexpr (kRows2) {
                lse = (m_used + pf_lg2(l)) * 0.69314718055994531f;
            } else {
                // block 1 hands (m, l) over and gets the factors back
                float2* ml = reinterpret_cast<float2*>(smem + L::kMl) + r;
                const uint32_t parity = (parts - 1) & 1;
                if (s == 1) {
                    *ml = make_float2(m_used, l);
                    mbar_arrive(ml_full);
                    ok = mbar_wait(f_full, parity, abort_flag, kPfO);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    const float2 f = *ml;
                    f0 = f.x;
                    f1 = f.y;
                    lse = 0.f;
                } else {
                    ok = mbar_wait(ml_full, parity, abort_flag, kPfO);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    const float2 o1 = *ml;
                    const float M = join ? fmaxf(m_used, o1.x) : m_used;
                    // no key in either block (all scores -inf): weights and sum 0; NaN stays NaN
                    const bool none = M == -INFINITY;
                    const float w0 = none ? 0.f : ex2(m_used - M), w1 = none || !join ? 0.f : ex2(o1.x - M);
                    const float ls = join ? w0 * l + w1 * o1.y : l;
                    f0 = w0 / ls;
                    f1 = w1 / ls;
                    lse = (M + pf_lg2(ls)) * 0.69314718055994531f;
                    *ml = make_float2(f0, f1);
                    mbar_arrive(f_full);
                }
            }
            // 8 columns of 8 rows a store, whole 32-byte sectors
            const int row_w = row - lane;                          // the warp's first row
            float* out = p.o_part + (prow - lane) * D;
            const uint32_t t0 = kRows2 ? tO : tmem + lane_off + 256;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int ra = half * 16 + (lane >> 2), rb = ra + 8;
                const float a0 = __shfl_sync(0xffffffffu, f0, ra), b0 = __shfl_sync(0xffffffffu, f0, rb);
                const float a1 = __shfl_sync(0xffffffffu, f1, ra), b1 = __shfl_sync(0xffffffffu, f1, rb);
                const bool va = row_w + ra < n_rows, vb = row_w + rb < n_rows;
                constexpr int kQ = kRows2 ? D / 32 : D / 64;       // blocks of 32 columns
#pragma unroll 1
                for (int q = 0; q < kQ; ++q) {
                    const int col = (kRows2 ? 0 : s * (D / 2)) + q * 32;
                    uint32_t ov[16], pv[16];
                    tmem_ld_16x32(t0 + (static_cast<uint32_t>(half * 16) << 16) + col, ov);
                    if (join) tmem_ld_16x32(t0 + 128 + (static_cast<uint32_t>(half * 16) << 16) + col, pv);
                    tmem_ld_wait();
#pragma unroll
                    for (int c8 = 0; c8 < 4; ++c8) {
                        const int d = col + c8 * 8 + (lane & 3) * 2;
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = __uint_as_float(ov[4 * c8 + e]) * (e < 2 ? a0 : b0);
                            if (join) v[e] = fmaf(__uint_as_float(pv[4 * c8 + e]), e < 2 ? a1 : b1, v[e]);
                        }
                        if (va) *reinterpret_cast<float2*>(out + static_cast<size_t>(ra) * D + d) = make_float2(v[0], v[1]);
                        if (vb) *reinterpret_cast<float2*>(out + static_cast<size_t>(rb) * D + d) = make_float2(v[2], v[3]);
                    }
                }
            }
            if (valid && (kRows2 || s == 0)) p.lse_part[prow] = lse;
            tc_fence_before();
            if constexpr (!kRows2) {
                // the next part overwrites both accumulators
                mbar_arrive(o_read);
                ok = mbar_wait(o_read, (parts - 1) & 1, abort_flag, kPfO);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kRows2>
cudaError_t go(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixParams& p, cudaStream_t stream) {
    auto kern = fa_prefix_kernel<D, kRows2>;
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void*>(kern), PfLayout<D, kRows2>::kAlloc);
    if (e != cudaSuccess) return e;
    kern<<<p.n_cta, kPfThreads, PfLayout<D, kRows2>::kAlloc, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix(int D, const CUtensorMap& tk, const CUtensorMap& tv, const PrefixParams& p,
                          cudaStream_t stream) {
    if (p.rows_unit == 2 * kTileM) return D == 128 ? go<128, true>(tk, tv, p, stream) : go<64, true>(tk, tv, p, stream);
    return D == 128 ? go<128, false>(tk, tv, p, stream) : go<64, false>(tk, tv, p, stream);
}

}  // namespace fa
