// fa_cache_decode.cu — decoding over a cache of sequences of different lengths
// at 16 or 8 bits, and the merge with a shared prefix (include/fa_cache.h).
//
// Bound by HBM: each cached row is read once for the Hq / Hkv * Nq query rows
// of its K/V head.  The lengths are in device memory, so the split is made
// there too: all (sequence, K/V head, row block) units' 64-key tiles are laid
// end to end and every resident CTA takes an equal run of them, whatever the
// lengths; a run may begin and end inside a unit.  A CTA reads the lengths
// (one warp's scan) to find its run.
//
//   warp 4      producer: K and V tiles (TMA) and their scales (bulk copies)
//               through a ring that keeps running across units
//   warps 0-3   16 keys of every tile each, with the keys as the M axis of
//               warp-level m16n8k16 MMAs:
//                 S^T [16 keys, rows]  = K [16, D] Q^T
//                 O^T [D, rows]       += V^T [D, 16] P^T
//               so that 8 query rows (one K/V head's group, usually) fill the
//               N axis; P^T is turned by movmatrix between the two.
// 8-bit codes are exact in fp16 and so are the products' operands: q is scaled
// by a power of two for each row (its largest value in [2^14, 2^15), values
// below 2^-29 of that lose bits), the K scale multiplies S in fp32, and the V
// scale goes into P.  P, times the V scale over a power of two that bounds the
// scales seen so far, is rounded to fp16 with its row maximum between 2^6 and
// 2^14 (a value of 2^-20 of the maximum is still a normal number: relative
// error 2^-11; below, the absolute one is 2^-31 of it); the row sum l is taken
// before that.  With bf16 caches P is rounded to bf16 (2^-8).  The maximum in
// use is replaced only when a score exceeds it by more than 8 (log2 units), and
// the bound on the V scales when one exceeds it, so most tiles need one vote
// and no shuffles or rescaling.
//
// The order of the contraction is free, so a lane reads 16 consecutive codes
// of a key with one shared-memory load and uses them as its four k-steps; for
// V, ldmatrix.trans moves pairs of codes and a byte permute makes the two
// rows d, d + 1 of V^T from them.
#include "fa_internal.h"
#include "sm100.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kCdThreads = 160;   // 4 compute warps + 1 producer warp
constexpr int kCdKeys = 64;       // keys per tile
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kCdRescale = 8.f; // growth of a row's maximum (log2 units) up to which the old one stays in use

enum CdSite { kCdSiteFull = 20, kCdSiteEmpty = 21, kCdSiteDrain = 22 };

template <int D, int kFmt>
struct CdLayout {
    static constexpr int kElem = kFmt == 0 ? 2 : 1;
    static constexpr int kTileBytes = kCdKeys * D * kElem;              // one K or V tile
    static constexpr int kScaleBytes = kFmt == 0 ? 0 : kCdKeys * 4;
    static constexpr int kStages = kFmt == 0 ? (D == 128 ? 3 : 4) : (D == 128 ? 3 : 6);
    // CTAs an SM holds at once, by shared memory and by registers (five warps
    // of at most 128 registers three times, of 168 twice)
    static constexpr int kCtas(int nt) { return kFmt == 0 && D == 128 ? 2 : (nt == 1 ? 3 : 2); }
    static constexpr int kK = 0;
    static constexpr int kV = kStages * kTileBytes;
    static constexpr int kScales = 2 * kStages * kTileBytes;            // K then V scales of each stage
    static constexpr int kMerge = kScales + 2 * kStages * kScaleBytes;  // [4 warps][8 rows][kCols + 4] fp32
    static constexpr int kCols = 64;
    static constexpr int kMl = kMerge + 4 * 8 * (kCols + 4) * 4;        // m, l and V exponent of the warps
    static constexpr int kBar = kMl + 4 * 40 * 4;
    static constexpr int kBytes = kBar + 2 * kStages * 8 + 48;
    static constexpr int kAlloc = kBytes + 1024;
};

// Byte offset of the 16-byte chunk `c` of key row `row` in a tile as TMA
// leaves it: rows of 128 bytes (bf16 at D = 128: two blocks of 64 values) with
// the chunk index XOR row % 8, or rows of 64 bytes with it XOR row / 2 % 4.
template <int D, int kFmt>
__device__ __forceinline__ uint32_t chunk_off(int row, int c) {
    if constexpr (kFmt != 0 && D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (kCdKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// C (16 x 8 fp32) += A (16 x 16) B (16 x 8), fp16 or bf16 operands.
template <bool kHalf>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes to fp16: lo = codes 0, 1, hi = codes 2, 3.  int8: code + 128 put
// under the exponent of 1024 is 1024 + 128 + code, exactly.
template <int kFmt>
__device__ __forceinline__ void unpack4(uint32_t c, uint32_t& lo, uint32_t& hi) {
    if constexpr (kFmt == 1) {
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(c));
    } else {
        const uint32_t u = c ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        __half2 ah = __hsub2(*reinterpret_cast<__half2*>(&a), off), bh = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        lo = *reinterpret_cast<uint32_t*>(&ah);
        hi = *reinterpret_cast<uint32_t*>(&bh);
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Power of two >= x as a float (x >= 0; the exponent kept within the normal
// range), and the inverse of a power of two.
__device__ __forceinline__ float pow2_at_least(float x) {
    const int e = (__float_as_int(x) + 0x7fffff) & 0x7f800000;
    return __int_as_float(min(max(e, 1 << 23), 253 << 23));
}
__device__ __forceinline__ float pow2_inverse(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }

__device__ __forceinline__ int seq_len(const CacheDecodeParams& p, int b) {
    return min(max(__ldg(p.lens + b), 0), p.capacity);
}
// Tiles of one unit of sequence b; a sequence without keys has one (all of it
// masked), so every unit is visited and gets its output.
__device__ __forceinline__ int seq_tiles(const CacheDecodeParams& p, int b) {
    return max(1, (seq_len(p, b) + kCdKeys - 1) / kCdKeys);
}

// A CTA's place in the run of tiles: tile `tile` of unit (b, hr), hr = K/V
// head * row blocks + row block.
struct Walk {
    int b, hr, tile, tiles, len;
    __device__ __forceinline__ void enter(const CacheDecodeParams& p) {
        len = seq_len(p, b);
        tiles = max(1, (len + kCdKeys - 1) / kCdKeys);
    }
    __device__ __forceinline__ void next_unit(const CacheDecodeParams& p) {
        tile = 0;
        if (++hr == p.HR) {
            hr = 0;
            ++b;
            if (b < p.B) enter(p);
        }
    }
};

struct RunStart {
    long long x0, x1, unit_at, total;   // the CTA's tiles, where its first unit starts, all tiles
    int n;                              // CTAs with a run: no more than there are tiles
    Walk w;
};

// Warp-wide: the run of CTA c of n (none for those past the number of tiles,
// so that the CTAs that share a unit are consecutive).
__device__ __forceinline__ RunStart find_run(const CacheDecodeParams& p, int c, int n, int lane) {
    RunStart s;
    long long total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long v = b0 + lane < p.B ? static_cast<long long>(seq_tiles(p, b0 + lane)) * p.HR : 0;
        for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        total += v;
    }
    if (n > total) n = static_cast<int>(total);
    s.n = n;
    s.total = total;
    s.x0 = c < n ? total * c / n : 0;
    s.x1 = c < n ? total * (c + 1) / n : 0;
    s.w = Walk{0, 0, 0, 1, 0};
    s.unit_at = 0;
    long long at = 0;
    for (int b0 = 0; b0 < p.B && s.x0 < s.x1; b0 += 32) {
        const long long v = b0 + lane < p.B ? static_cast<long long>(seq_tiles(p, b0 + lane)) * p.HR : 0;
        long long incl = v;
        for (int k = 1; k < 32; k <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, k);
            if (lane >= k) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + incl > s.x0);
        if (past) {
            const int src = __ffs(past) - 1;
            const long long seq_at = __shfl_sync(0xffffffffu, at + incl - v, src);
            s.w.b = b0 + src;
            s.w.enter(p);
            const long long off = s.x0 - seq_at;
            s.w.hr = static_cast<int>(off / s.w.tiles);
            s.w.tile = static_cast<int>(off - static_cast<long long>(s.w.hr) * s.w.tiles);
            s.unit_at = s.x0 - s.w.tile;
            break;
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
    }
    return s;
}

__device__ __forceinline__ void cd_drain(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return;
        if ((it & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(&g_status, 1u << kCdSiteDrain);
            return;
        }
    }
}

// NT: blocks of 8 query rows a CTA holds.
template <int D, int kFmt, int NT>
__global__ void __launch_bounds__(kCdThreads, CdLayout<D, kFmt>::kCtas(NT))
fa_cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const CacheDecodeParams p) {
    using L = CdLayout<D, kFmt>;
    constexpr bool kHalf = kFmt != 0;
    constexpr int kStages = L::kStages;
    constexpr int kSteps = D / 16;
    constexpr float kShift = kHalf ? 6.f : 0.f;   // P is 2^kShift where the score is the row's (stale) maximum
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kBar + 2 * kStages * 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    const RunStart run = find_run(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), lane);
    __syncthreads();
    const int n_run = static_cast<int>(run.x1 - run.x0);
    if (n_run == 0) return;   // the whole CTA

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            Walk w = run.w;
            int issued = 0;
            for (int t = 0; t < n_run; ++t) {
                const int st = t % kStages;
                if (t >= kStages && !mbar_wait(&empty[st], ((t / kStages) - 1) & 1, abort_flag, kCdSiteEmpty)) break;
                const int key0 = w.tile * kCdKeys;
                const int bkv = w.b * p.Hkv + w.hr / p.RB;
                // the scales' rows end at the capacity, a multiple of 4
                const uint32_t sbytes = kHalf ? static_cast<uint32_t>(min(kCdKeys, p.capacity - key0)) * 4u : 0u;
                mbar_arrive_expect_tx(&full[st], 2 * L::kTileBytes + 2 * sbytes);
                constexpr int kBox = D * L::kElem > 128 ? 2 : 1;
#pragma unroll
                for (int a = 0; a < kBox; ++a) {
                    tma_load_3d(smem + L::kK + st * L::kTileBytes + a * (L::kTileBytes / kBox), &tmK, &full[st], a * 64,
                                key0, bkv);
                    tma_load_3d(smem + L::kV + st * L::kTileBytes + a * (L::kTileBytes / kBox), &tmV, &full[st], a * 64,
                                key0, bkv);
                }
                if constexpr (kHalf) {
                    const size_t at = static_cast<size_t>(bkv) * p.capacity + key0;
                    bulk_load(smem + L::kScales + st * 2 * L::kScaleBytes, p.k_scale + at, sbytes, &full[st]);
                    bulk_load(smem + L::kScales + st * 2 * L::kScaleBytes + L::kScaleBytes, p.v_scale + at, sbytes,
                              &full[st]);
                }
                issued = t + 1;
                if (++w.tile == w.tiles) w.next_unit(p);
            }
            // nothing may still be landing in shared memory when the CTA leaves
            for (int t = (issued > kStages ? issued - kStages : 0); t < issued; ++t)
                cd_drain(&full[t % kStages], (t / kStages) & 1);
        }
        return;
    }

    // ---------------------------------------------------------------- compute
    const int g8 = lane >> 2, t4 = lane & 3;
    const int kw = warp * 16;                       // this warp's 16 keys in a tile
    const uint32_t sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV), sS = smem_u32(smem + L::kScales);
    float* merge = reinterpret_cast<float*>(smem + L::kMerge);
    float* ml = reinterpret_cast<float*>(smem + L::kMl);   // [warp]: m [16], l [16], V exponent
    const int R = p.G * p.Nq;
    Walk w = run.w;
    long long unit_at = run.unit_at;
    bool ok = true;
    int st = 0;            // ring stage and its parity
    uint32_t phase = 0u;

    // After a wait that gave up, the remaining units are walked without loads
    // or outputs, so that the barriers below stay matched.
    for (int t = 0; t < n_run;) {
        // ---- one unit, or the part of it in this CTA's run
        const int n_here = min(w.tiles - w.tile, n_run - t);
        const int hkv = w.hr / p.RB;
        const int row0 = (w.hr - hkv * p.RB) * (8 * NT);
        const size_t rows_at = static_cast<size_t>(w.b * p.Hkv + hkv) * R;   // first query row of the K/V head
        // Q^T fragments: query row n * 8 + g8; zero on rows past R
        uint32_t qb[NT][kSteps][2];
        float qc[NT][2];      // softmax scale (log2 units) over q's power of two, rows 2 t4, 2 t4 + 1
        int pos[NT][2];       // last visible slot of rows 2 t4, 2 t4 + 1
        int pos_min = w.len - 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + n * 8 + g8;
            const __nv_bfloat16* qrow =
                reinterpret_cast<const __nv_bfloat16*>(p.q) + (rows_at + (r < R ? r : 0)) * D;
            if constexpr (kHalf) {
                uint2 raw[kSteps];
                uint32_t am = 0u;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    // step s = 4 hh + w4: values (chunk of 16) * 16 + 4 w4 .. + 3
                    const int d = (D == 128 ? (2 * t4 + (s >> 2)) : t4) * 16 + (s & 3) * 4;
                    raw[s] = r < R ? __ldg(reinterpret_cast<const uint2*>(qrow + d)) : make_uint2(0u, 0u);
                    am = __vmaxu2(am, __vmaxu2(raw[s].x & 0x7fff7fffu, raw[s].y & 0x7fff7fffu));
                }
                am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, 2));
                // 2^(14 - exponent of the row's largest value); q = 0: any
                const int ex = static_cast<int>(max(am & 0xffffu, am >> 16) >> 7) - 127;
                const int f = min(max(14 - ex, -113), 126);
                const float up = __int_as_float((127 + f) << 23);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    qb[n][s][0] = pack_half2(__uint_as_float(raw[s].x << 16) * up,
                                             __uint_as_float(raw[s].x & 0xffff0000u) * up);
                    qb[n][s][1] = pack_half2(__uint_as_float(raw[s].y << 16) * up,
                                             __uint_as_float(raw[s].y & 0xffff0000u) * up);
                }
                const float back = pow2_inverse(up);
                qc[n][0] = __shfl_sync(0xffffffffu, back, 8 * t4) * p.scale_log2;
                qc[n][1] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4) * p.scale_log2;
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qb[n][s][e] = r < R ? __ldg(reinterpret_cast<const uint32_t*>(qrow + s * 16 + e * 8 + 2 * t4))
                                            : 0u;
                qc[n][0] = qc[n][1] = p.scale_log2;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rr = row0 + n * 8 + 2 * t4 + h;
                pos[n][h] = p.causal ? w.len - p.Nq + (rr < R ? rr % p.Nq : 0) : w.len - 1;
            }
        }
        if (p.causal) pos_min = w.len - p.Nq;

        float o[NT][kSteps][4];
        // stale row maximum, kShift less it (infinite before the first key), partial row sum
        float m_run[NT][2], nm[NT][2], l_run[NT][2];
        float v_top = __int_as_float(1 << 23);   // power of two that bounds the V scales so far
        float v_inv = pow2_inverse(v_top);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
            m_run[n][0] = m_run[n][1] = -INFINITY;
            nm[n][0] = nm[n][1] = INFINITY;
            l_run[n][0] = l_run[n][1] = 0.f;
        }

        for (int i = 0; i < n_here; ++i, ++t) {
            ok = ok && mbar_wait(&full[st], phase, abort_flag, kCdSiteFull);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            const uint32_t kb = sK + st * L::kTileBytes, vb = sV + st * L::kTileBytes;
            const int key0 = (w.tile + i) * kCdKeys + kw;    // slot of the warp's first key
            const int kA = key0 + g8, kB = kA + 8;           // this lane's two keys in S^T
            const bool edge = key0 + 15 > pos_min;           // some key is hidden from some row (warp-uniform)
            const bool clear = key0 + 15 >= w.len;           // some key is behind the length
            if (clear) {
                // V rows behind the length may hold NaN, and 0 x NaN is NaN
                constexpr int kChunks = D * L::kElem / 16;
                for (int e = lane; e < 16 * kChunks; e += 32) {
                    const int row = kw + e / kChunks;
                    if (key0 + e / kChunks >= w.len)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                     ::"r"(vb + chunk_off<D, kFmt>(row, e % kChunks)), "r"(0u) : "memory");
                }
                __syncwarp();
            }
            // ---- S^T (16 keys x rows) = K Q^T
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            float ksA = 1.f, ksB = 1.f, vsA = 1.f, vsB = 1.f;
            const int mi = lane >> 3;
            if constexpr (kHalf) {
                const uint32_t sc = sS + st * 2 * L::kScaleBytes + (kw + g8) * 4;
                ksA = lds32(sc);
                ksB = lds32(sc + 32);
                vsA = lds32(sc + L::kScaleBytes);
                vsB = lds32(sc + L::kScaleBytes + 32);
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh) {
                    const int c = D == 128 ? 2 * t4 + hh : t4;
                    const uint4 ca = lds128(kb + chunk_off<D, kFmt>(kw + g8, c));
                    const uint4 cb = lds128(kb + chunk_off<D, kFmt>(kw + g8 + 8, c));
                    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
                    for (int w4 = 0; w4 < 4; ++w4) {
                        uint32_t a0, a1, a2, a3;
                        unpack4<kFmt>(wa[w4], a0, a2);
                        unpack4<kFmt>(wb[w4], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16<true>(s[n], a0, a1, a2, a3, qb[n][4 * hh + w4][0], qb[n][4 * hh + w4][1]);
                    }
                }
            } else {
                const int krow = kw + (mi & 1) * 8 + (lane & 7);   // matrices: (keys lo, hi) x (d lo, hi)
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk) {
                    uint32_t a[4];
                    ldsm4(kb + chunk_off<D, kFmt>(krow, 2 * kk + (mi >> 1)), a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16<false>(s[n], a[0], a[1], a[2], a[3], qb[n][kk][0], qb[n][kk][1]);
                }
            }
            // ---- mask, online softmax (rows 2 t4, 2 t4 + 1; keys kA, kB).  Element e is
            // (key e / 2, row e % 2); y = score + kShift - stale maximum, in log2 units.
            float y[NT][4];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[n][e] = fmaf(s[n][e], ((e >> 1) ? ksB : ksA) * qc[n][e & 1], nm[n][e & 1]);
                    if (edge && ((e >> 1) ? kB : kA) > pos[n][e & 1]) y[n][e] = -INFINITY;
                    grow |= y[n][e] > kShift + kCdRescale;
                }
            if constexpr (kHalf) grow |= (vsA > v_top && kA < w.len) || (vsB > v_top && kB < w.len);
            if (__any_sync(0xffffffffu, grow)) {
                // a maximum grew by more than kCdRescale, or a V scale past the
                // bound: take the new ones and bring the sums so far to them
                float vfac = 1.f;
                if constexpr (kHalf) {
                    float vm = fmaxf(kA < w.len ? vsA : 0.f, kB < w.len ? vsB : 0.f);
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, k));
                    const float top = fmaxf(v_top, pow2_at_least(vm));
                    v_inv = pow2_inverse(top);
                    vfac = v_top * v_inv;
                    v_top = top;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float alpha[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float xa = y[n][h] == -INFINITY ? -INFINITY : s[n][h] * (ksA * qc[n][h]);
                        const float xb = y[n][2 + h] == -INFINITY ? -INFINITY : s[n][2 + h] * (ksB * qc[n][h]);
                        float mx = fmaxf(xa, xb);
#pragma unroll
                        for (int k = 4; k <= 16; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                        const float m_new = fmaxf(m_run[n][h], mx);
                        alpha[h] = m_new == -INFINITY ? 1.f : ex2(m_run[n][h] - m_new);
                        m_run[n][h] = m_new;
                        nm[n][h] = kShift - m_new;
                        l_run[n][h] *= alpha[h];
                        alpha[h] *= vfac;
                        y[n][h] = xa + nm[n][h];            // -inf + inf, where no key was seen yet:
                        y[n][2 + h] = xb + nm[n][h];        // put right below
                        if (xa == -INFINITY) y[n][h] = -INFINITY;
                        if (xb == -INFINITY) y[n][2 + h] = -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        o[n][j][0] *= alpha[0];
                        o[n][j][1] *= alpha[1];
                        o[n][j][2] *= alpha[0];
                        o[n][j][3] *= alpha[1];
                    }
                }
            }
            vsA *= v_inv;
            vsB *= v_inv;
            uint32_t pb[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pw[e] = ex2(y[n][e]);
                l_run[n][0] += pw[0] + pw[2];
                l_run[n][1] += pw[1] + pw[3];
                if constexpr (kHalf) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pw[e] *= (e >> 1) ? vsB : vsA;
                        // a hidden key's scale may be anything
                        if (edge && y[n][e] == -INFINITY) pw[e] = 0.f;
                    }
                    pb[n][0] = turn8x8(pack_half2(pw[0], pw[1]));
                    pb[n][1] = turn8x8(pack_half2(pw[2], pw[3]));
                } else {
                    pb[n][0] = turn8x8(pack_bf16x2(pw[0], pw[1]));
                    pb[n][1] = turn8x8(pack_bf16x2(pw[2], pw[3]));
                }
            }
            // ---- O^T (D x rows) += V^T P^T
            if constexpr (kHalf) {
                // matrices: (keys lo, hi) x (chunk of 16 values j, j + 1)
                const int vrow = kw + (mi & 1) * 8 + (lane & 7);
#pragma unroll
                for (int j = 0; j < kSteps; j += 2) {
                    uint32_t r[4];
                    ldsm4_t(vb + chunk_off<D, kFmt>(vrow, j + (mi >> 1)), r);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a0, a1, a2, a3;   // rows d = 16 j + 2 g8 (a0, a2) and + 1 (a1, a3)
                        unpack4<kFmt>(__byte_perm(r[2 * u], 0u, 0x3120), a0, a1);
                        unpack4<kFmt>(__byte_perm(r[2 * u + 1], 0u, 0x3120), a2, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16<true>(o[n][j + u], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    }
                }
            } else {
                // matrices: (d lo, hi) x (keys lo, hi)
                const int vrow = kw + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    uint32_t r[4];
                    ldsm4_t(vb + chunk_off<D, kFmt>(vrow, 2 * j + (mi & 1)), r);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16<false>(o[n][j], r[0], r[1], r[2], r[3], pb[n][0], pb[n][1]);
                }
            }
            if (clear) fence_proxy_async_smem();   // the zeros before the next copy into this stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }

        // ---- the four warps' parts of the unit, joined in shared memory
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) l_run[n][h] += __shfl_xor_sync(0xffffffffu, l_run[n][h], k);
        if (g8 == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ml[warp * 40 + n * 8 + 2 * t4 + h] = m_run[n][h];
                    ml[warp * 40 + 16 + n * 8 + 2 * t4 + h] = l_run[n][h];
                }
            if (t4 == 0) ml[warp * 40 + 32] = v_top;
        }
        const long long unit_end = unit_at + w.tiles;
        const bool whole = n_here == w.tiles;
        // a part at the start of the run goes to slot 2 c, one that begins in it to 2 c + 1
        const bool at_start = unit_at + w.tile == run.x0;
        const int slot = 2 * static_cast<int>(blockIdx.x) + (at_start ? 0 : 1);
        if (w.tile == 0 && threadIdx.x == 0) {
            const int unit = w.b * p.HR + w.hr;
            const int last = static_cast<int>((unit_end * run.n - 1) / run.total);   // CTA of the last tile
            p.meta[unit] = make_int2(whole ? -1 : slot, last);
        }
        constexpr int kPitch = L::kCols + 4;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int dh = 0; dh < D / L::kCols; ++dh) {
                asm volatile("bar.sync 1, 128;" ::: "memory");   // the previous block has been read
#pragma unroll
                for (int jj = 0; jj < L::kCols / 16; ++jj) {
                    const int j = dh * (L::kCols / 16) + jj;
                    float* at = merge + (warp * 8 + 2 * t4) * kPitch + jj * 16;
                    if constexpr (kHalf) {   // o: (d, row 0), (d, row 1), (d + 1, row 0), (d + 1, row 1), d = 2 g8
                        *reinterpret_cast<float2*>(at + 2 * g8) = make_float2(o[n][j][0], o[n][j][2]);
                        *reinterpret_cast<float2*>(at + kPitch + 2 * g8) = make_float2(o[n][j][1], o[n][j][3]);
                    } else {                 // d = g8 and g8 + 8
                        at[g8] = o[n][j][0];
                        at[kPitch + g8] = o[n][j][1];
                        at[g8 + 8] = o[n][j][2];
                        at[kPitch + g8 + 8] = o[n][j][3];
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                // thread -> (row, 4 columns)
                const int r = threadIdx.x >> 4, c4 = (threadIdx.x & 15) * 4;
                const int row = row0 + n * 8 + r;
                float M = -INFINITY, wgt[4], Lsum = 0.f, top = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    M = fmaxf(M, ml[q * 40 + n * 8 + r]);
                    if (kHalf) top = fmaxf(top, ml[q * 40 + 32]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float mq = ml[q * 40 + n * 8 + r];
                    wgt[q] = mq == -INFINITY ? 0.f : ex2(mq - M);
                    Lsum += wgt[q] * ml[q * 40 + 16 + n * 8 + r];
                    if (kHalf) wgt[q] *= ml[q * 40 + 32] * pow2_inverse(top);
                }
                // rows without a key: 0; a NaN sum stays NaN
                const float inv = Lsum == 0.f ? 0.f : (kHalf ? top : 1.f) / Lsum;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(merge + (q * 8 + r) * kPitch + c4);
                    acc.x += wgt[q] * v.x;
                    acc.y += wgt[q] * v.y;
                    acc.z += wgt[q] * v.z;
                    acc.w += wgt[q] * v.w;
                }
                acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                const float lse = Lsum == 0.f ? -INFINITY : (M + log2f(Lsum) - kShift) * kLn2;
                const int d = dh * L::kCols + c4;
                if (row < R && ok) {
                    if (whole && p.o_unit == nullptr) {
                        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.o) + (rows_at + row) * D + d;
                        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
                        if (d == 0) p.lse[rows_at + row] = lse;
                    } else if (whole) {
                        *reinterpret_cast<float4*>(p.o_unit + (rows_at + row) * D + d) = acc;
                        if (d == 0) p.lse_unit[rows_at + row] = lse;
                    } else {
                        const size_t prow = static_cast<size_t>(slot) * (8 * NT) + n * 8 + r;
                        *reinterpret_cast<float4*>(p.o_part + prow * D + d) = acc;
                        if (d == 0) p.lse_part[prow] = lse;
                    }
                }
            }
        }
        w.tile += n_here;
        if (w.tile == w.tiles) {
            unit_at = unit_end;
            w.next_unit(p);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");   // ml is free again
    }
}

// Joins the parts of a query row: those of the CTAs that share its unit, and
// the prefix's.  One CTA a row, a warp for every fourth part.
//   LSE = log sum_s exp(LSE_s),   O = sum_s exp(LSE_s - LSE) O_s
template <int D>
__global__ void __launch_bounds__(128)
fa_cache_combine_kernel(const CacheDecodeParams p, const PrefixParams f) {
    constexpr int kPer = D / 32;
    __shared__ float sh_m[4], sh_z[4];
    __shared__ float sh_o[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = p.G * p.Nq;
    const int gr = static_cast<int>(blockIdx.x);      // row of [B, Hq, Nq]
    const int bkv = gr / R, r = gr - bkv * R;
    const int b = bkv / p.Hkv, hkv = bkv - b * p.Hkv;
    const int rb = r / p.rows_cta, in = r - rb * p.rows_cta;
    const int2 meta = p.meta[b * p.HR + hkv * p.RB + rb];
    const bool whole = meta.x < 0;
    if (whole && f.n_cta == 0) return;                // written by the main kernel
    const int own = whole ? 1 : meta.y - (meta.x >> 1) + 1;
    // the prefix unit that holds the row, and the CTAs that share it
    int pfirst = 0, np = 0, psub = 0, pin = 0, pu = 0;
    if (f.n_cta > 0) {
        const int prow = b * R + r;
        pu = hkv * f.n_rowtiles + prow / f.rows_unit;
        pin = prow % f.rows_unit;
        psub = f.subs;
        const long long total = static_cast<long long>(f.Hkv) * f.n_rowtiles * f.n_tiles;
        const long long ts = static_cast<long long>(pu) * f.n_tiles;
        pfirst = static_cast<int>(((ts + 1) * f.n_cta - 1) / total);
        np = (static_cast<int>(((ts + f.n_tiles) * f.n_cta - 1) / total) - pfirst + 1) * psub;
    }
    const int n = own + np;
    auto part = [&](int i, const float*& o, float& lse) {
        if (i < own) {
            if (whole) {
                o = p.o_unit + static_cast<size_t>(gr) * D;
                lse = p.lse_unit[gr];
            } else {
                const int slot = i == 0 ? meta.x : 2 * ((meta.x >> 1) + i);
                const size_t prow = static_cast<size_t>(slot) * p.rows_cta + in;
                o = p.o_part + prow * D;
                lse = p.lse_part[prow];
            }
        } else {
            const int k = i - own;
            const size_t prow = (static_cast<size_t>(pfirst + k / psub + pu) * psub + k % psub) * f.rows_unit + pin;
            o = f.o_part + prow * D;
            lse = f.lse_part[prow];
        }
    };
    float M = -INFINITY, Z = 0.f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int s = warp; s < n; s += 4) {
        const float* o;
        float lse;
        part(s, o, lse);
        if (lse == -INFINITY) continue;               // no key in this part; its o may be unwritten
        const float m_new = fmaxf(M, lse);
        const float a = __expf(M - m_new), e = expf(lse - m_new);
        M = m_new;
        Z = Z * a + e;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * a + e * o[lane * kPer + i];
    }
    if (lane == 0) {
        sh_m[warp] = M;
        sh_z[warp] = Z;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) sh_o[warp][lane * kPer + i] = acc[i];
    __syncthreads();
    if (warp != 0) return;
    float Mt = -INFINITY, Zt = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) Mt = fmaxf(Mt, sh_m[q]);
    float out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[i] = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float e = sh_m[q] == -INFINITY && sh_z[q] == 0.f ? 0.f : expf(sh_m[q] - Mt);
        Zt += e * sh_z[q];
#pragma unroll
        for (int i = 0; i < kPer; ++i) out[i] += e * sh_o[q][lane * kPer + i];
    }
    const float inv = Zt == 0.f ? 0.f : 1.f / Zt;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + static_cast<size_t>(gr) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(out[i] * inv, out[i + 1] * inv);
    if (lane == 0) p.lse[gr] = Zt == 0.f ? -INFINITY : Mt + logf(Zt);
}

template <int D, int kFmt, int NT>
cudaError_t go(const CUtensorMap& tk, const CUtensorMap& tv, const CacheDecodeParams& p, cudaStream_t stream) {
    auto kern = fa_cache_decode_kernel<D, kFmt, NT>;
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void*>(kern), CdLayout<D, kFmt>::kAlloc);
    if (e != cudaSuccess) return e;
    kern<<<p.n_cta, kCdThreads, CdLayout<D, kFmt>::kAlloc, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t go_fmt(int fmt, const CUtensorMap& tk, const CUtensorMap& tv, const CacheDecodeParams& p,
                   cudaStream_t stream) {
    const bool one = p.rows_cta == 8;
    if (fmt == 0) return one ? go<D, 0, 1>(tk, tv, p, stream) : go<D, 0, 2>(tk, tv, p, stream);
    if (fmt == 1) return one ? go<D, 1, 1>(tk, tv, p, stream) : go<D, 1, 2>(tk, tv, p, stream);
    return one ? go<D, 2, 1>(tk, tv, p, stream) : go<D, 2, 2>(tk, tv, p, stream);
}

}  // namespace

int cache_decode_ctas_per_sm(int D, int fmt, int rows_cta) {
    const int nt = rows_cta / 8;
    if (D == 128) return fmt == 0 ? CdLayout<128, 0>::kCtas(nt) : CdLayout<128, 1>::kCtas(nt);
    return fmt == 0 ? CdLayout<64, 0>::kCtas(nt) : CdLayout<64, 1>::kCtas(nt);
}

cudaError_t launch_cache_decode(int D, int fmt, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, cudaStream_t stream) {
    return D == 128 ? go_fmt<128>(fmt, tk, tv, p, stream) : go_fmt<64>(fmt, tk, tv, p, stream);
}

cudaError_t launch_cache_combine(int D, const CacheDecodeParams& p, const PrefixParams& f, cudaStream_t stream) {
    const unsigned rows = static_cast<unsigned>(p.B) * p.Hkv * p.G * p.Nq;
    if (D == 128)
        fa_cache_combine_kernel<128><<<rows, 128, 0, stream>>>(p, f);
    else
        fa_cache_combine_kernel<64><<<rows, 128, 0, stream>>>(p, f);
    return cudaGetLastError();
}

}  // namespace fa
