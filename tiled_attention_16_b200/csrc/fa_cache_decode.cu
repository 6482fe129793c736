// fa_cache_decode.cu — decoding over a cache of sequences of different lengths
// at 16 or 8 bits, and the merge with a shared prefix (include/fa_cache.h).
//
// Bound by HBM: each cached row is read once for the Hq / Hkv * Nq query rows
// of its K/V head (8 sequences of 32K slots, 64 query over 8 K/V heads of 128:
// e4m3 88 us, 6.1 TB/s; int8 88; bf16 157, 6.8).  The lengths are in device
// memory, so the split is made there too: all (sequence, K/V head) units'
// 64-key tiles are laid end to end and every resident CTA takes an equal run of
// them, whatever the lengths; a run may begin and end inside a unit.  A CTA
// reads the lengths (one warp's scan) to find its run.  Many short sequences
// are bound by what a unit costs besides its tiles (48 of up to 8100 int8
// slots, 12 query rows: 46 us, 4.6 TB/s).
//
//   warp 4      producer: K and V tiles (TMA) and their scales (bulk copies)
//               through a ring that keeps running across units
//   warps 0-3   warp-level m16n8k16 MMAs with keys, then columns, as the M axis,
//               so that 8 query rows (one K/V head's group, usually) fill the N
//               axis.  A warp takes 16 keys of every tile for the scores and a
//               quarter of the columns for the output:
//                 S^T [16 keys, rows]    = K [16, D] Q^T
//                 O^T [D / 4, rows]     += V^T [D / 4, 64 keys] P^T
//               P^T is turned by movmatrix and handed round in shared memory
//               (two buffers, so one barrier a tile).  A warp that kept its keys
//               for both products would need no barrier, but all D columns of
//               O: then a unit's end joins four accumulators (51 us instead of
//               46 in the case above) and 32 rows do not fit a CTA.
// 8-bit codes are exact in fp16 and so are the products' operands: q is scaled
// by a power of two for each row (its largest value in [2^14, 2^15), values
// below 2^-29 of that lose bits), the K scale multiplies S in fp32, and the V
// scale goes into P.  P, times the V scale over a power of two that bounds the
// scales seen so far, is rounded to fp16 with its row maximum between 2^6 and
// 2^14 (a value of 2^-20 of the maximum is still a normal number: relative
// error 2^-11; below, the absolute one is 2^-31 of it); the row sum l is taken
// before that.  With bf16 caches P is rounded to bf16 (2^-8): a product has one
// operand type, and V's range does not fit fp16.  The maximum in
// use is replaced only when a score exceeds it by more than 8 (log2 units), and
// the bound on the V scales when one exceeds it, so most tiles need one vote
// (which is the barrier) and no shuffles or rescaling.  All four warps use the
// same maxima and bound.
//
// The order of the contraction is free, so a lane reads 16 consecutive codes
// of a key with one shared-memory load and uses them as its four k-steps; for
// V, ldmatrix.trans moves pairs of codes and a byte permute makes the two
// rows d, d + 1 of V^T from them.
#include "fa_serving.cuh"

#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace fa {

namespace {

constexpr int kCdThreads = 160;   // 4 compute warps + 1 producer warp
constexpr int kCdKeys = 64;       // keys per tile
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kCdRescale = 8.f; // growth of a row's maximum (log2 units) up to which the old one stays in use

enum CdSite { kCdSiteFull = 20, kCdSiteEmpty = 21, kCdSiteDrain = 22 };

template <int D, int kFmt, int NT>
struct CdLayout {
    static constexpr int kElem = kFmt == 0 ? 2 : 1;
    static constexpr bool kWide = kFmt == 0 && D == 128;                // 32 KB a stage
    // CTAs an SM holds at once, by shared memory and by registers (five warps
    // of at most 128 registers three times, of 168 twice)
    static constexpr int kCtas = kWide || NT == 4 ? 2 : 3;
    static constexpr int kTileBytes = kCdKeys * D * kElem;              // one K or V tile
    static constexpr int kScaleBytes = kFmt == 0 ? 0 : kCdKeys * 4;
    static constexpr int kQFrag = NT * (D / 16) * 32 * 8;               // Q^T fragments of a unit
    static constexpr int kPFrag = 4 * NT * 32 * 8;                      // P^T fragments of a tile
    // Enough bytes under way for the copy rate, and no more: HBM serves fewer at
    // once better (8 sequences of 32K slots of 8 heads, stages: e4m3 at 128
    // 2: 89.9 us, 3: 88.1, 4: 92.3; bf16 at 128 2: 156.5, 3: 161; 16 sequences at
    // 64, e4m3 3: 98.0, 4: 94.5, 5: 99.2; bf16 2: 83.9, 3: 84.3, 4: 88.5).
    static constexpr int kStages = D == 128 ? (kFmt == 0 ? 2 : 3) : kFmt == 0 ? 2 : 4;
    static constexpr int kK = 0;
    static constexpr int kV = kStages * kTileBytes;
    static constexpr int kScales = 2 * kStages * kTileBytes;            // K then V scales of each stage
    static constexpr int kQ = kScales + 2 * kStages * kScaleBytes;      // two units' fragments,
    static constexpr int kQScale = kQ + 2 * kQFrag;                     // and their rows' factors
    static constexpr int kP = kQScale + 2 * NT * 8 * 4;                 // two tiles' fragments
    static constexpr int kMx = kP + 2 * kPFrag;                         // the warps' row maxima, V scales' maxima
    static constexpr int kMl = kMx + 4 * NT * 8 * 4 + 16;               // and row sums
    static constexpr int kBad = kMl + 4 * NT * 8 * 4;                   // two tiles' masks of poisoned V rows, one a warp
    static constexpr int kBar = kBad + 32;
    static constexpr int kAlloc = kBar + (2 * kStages + 4) * 8 + 16;
    static_assert((kAlloc + 1024) * kCtas <= 228 * 1024, "CTAs must fit");
};

// Byte offset of the 16-byte chunk `c` of key row `row` in a tile as TMA
// leaves it: rows of 128 bytes (bf16 at D = 128: two blocks of 64 values) with
// the chunk index XOR row % 8, or rows of 64 bytes with it XOR row / 2 % 4.
template <int D, int kFmt>
__device__ __forceinline__ uint32_t chunk_off(int row, int c) {
    if constexpr (kFmt != 0 && D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (kCdKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// The address `c` chunks on (c even, or the first chunk even) from an address
// that chunk_off() gave.
__device__ __forceinline__ uint32_t chunk_at(uint32_t addr, int c) {
    return (addr ^ ((c & 7) << 4)) + (c >> 3) * (kCdKeys * 128);
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
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
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

// Four codes (d, d + 1 of a first key, then of a second) to fp16, by d.
template <int kFmt>
__device__ __forceinline__ void unpack4_pairs(uint32_t c, uint32_t& d0, uint32_t& d1) {
    if constexpr (kFmt == 1) {
        unpack4<1>(__byte_perm(c, 0u, 0x3120), d0, d1);
    } else {
        const uint32_t u = c ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
        __half2 ah = __hsub2(*reinterpret_cast<__half2*>(&a), off), bh = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        d0 = *reinterpret_cast<uint32_t*>(&ah);
        d1 = *reinterpret_cast<uint32_t*>(&bh);
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

// Work is dealt out by position: a unit (sequence b, K/V head h) covers
// unit_cost positions for what it costs besides its tiles, then one for each
// tile.  All units lie end to end and run c of n takes positions
// [total c / n, total (c + 1) / n).  With more query rows a K/V head than a CTA
// holds, RB CTAs take a run, one a block of rows, at the same time: the tiles
// come from HBM once and from L2 for the others (8 sequences of 32K slots, two
// blocks of 16 rows: 163 us, 174 with the row blocks as units of their own).
struct Walk {
    int x0, x1, total, n;       // the run's positions, all positions, runs with any
    int b, h, at, tiles, len;   // unit, its first position, its tiles, its sequence's length
    int t0, t1;                 // the run's tiles of it

    __device__ __forceinline__ void enter(const CacheDecodeParams& p) {
        len = seq_len(p, b);
        tiles = max(1, (len + kCdKeys - 1) / kCdKeys);
    }
    __device__ __forceinline__ void clip(const CacheDecodeParams& p) {
        t0 = max(0, x0 - at - p.unit_cost);
        t1 = min(tiles, x1 - at - p.unit_cost);
    }
    // to the first unit from here on that the run has tiles of; false: none
    __device__ __forceinline__ bool settle(const CacheDecodeParams& p) {
        while (at < x1) {
            clip(p);
            if (t0 < t1) return true;
            step(p);
        }
        return false;
    }
    __device__ __forceinline__ void step(const CacheDecodeParams& p) {
        at += tiles + p.unit_cost;
        if (++h == p.Hkv) {
            h = 0;
            ++b;
            if (b < p.B) enter(p);
        }
    }
};

// Warp-wide: run c of n, at the unit its positions begin in; or, where units
// are not divided, unit c.
__device__ __forceinline__ Walk find_run(const CacheDecodeParams& p, int c, int n, int lane) {
    Walk w;
    auto weight = [&](int b) { return b < p.B ? (seq_tiles(p, b) + p.unit_cost) * p.Hkv : 0; };
    if (p.undivided) {
        w.b = c / p.Hkv;
        w.h = c - w.b * p.Hkv;
        w.enter(p);
        w.at = w.x0 = 0;
        w.x1 = w.total = w.tiles + p.unit_cost;
        w.n = 1;
        w.t0 = w.t1 = 0;
        return w;
    }
    const int first = weight(lane);
    int total = first;
#pragma unroll 4
    for (int b = lane + 32; b < p.B; b += 32) total += weight(b);
    total = __reduce_add_sync(0xffffffffu, total);
    n = min(n, total);          // every run has a position, so those that share a unit are consecutive
    w.n = n;
    w.total = total;
    w.x0 = c < n ? static_cast<int>(static_cast<long long>(total) * c / n) : 0;
    w.x1 = c < n ? static_cast<int>(static_cast<long long>(total) * (c + 1) / n) : 0;
    w.b = w.h = w.at = w.len = w.t0 = w.t1 = 0;
    w.tiles = 1;
    int at = 0;
    for (int b0 = 0; b0 < p.B && w.x0 < w.x1; b0 += 32) {
        const int v = b0 == 0 ? first : weight(b0 + lane);
        int incl = v;
        for (int k = 1; k < 32; k <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, k);
            if (lane >= k) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + incl > w.x0);
        if (past) {
            const int src = __ffs(past) - 1;
            w.at = __shfl_sync(0xffffffffu, at + incl - v, src);
            w.b = b0 + src;
            w.enter(p);
            w.h = (w.x0 - w.at) / (w.tiles + p.unit_cost);
            w.at += w.h * (w.tiles + p.unit_cost);
            break;
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
    }
    return w;
}

// Whether any thread of the four compute warps says so; also their barrier.
__device__ __forceinline__ bool any_of_warps(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\t"
                 "setp.ne.u32 a, %1, 0;\n\t"
                 "bar.red.or.pred b, 1, 128, a;\n\t"
                 "selp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)) : "memory");
    return r != 0u;
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

// bf16 V rows that only some of a CTA's query rows see: those that hold an
// infinity or a NaN among the warp's 16 rows of a tile, `slot0` the first's slot,
// first <= slot < len.  They are zeroed in the tile, since a hidden key's weight
// of 0 times them would be NaN, and returned as a mask: the query rows that do see
// them get them added behind the tile's products.
template <int D>
__device__ __forceinline__ uint32_t take_poisoned(uint32_t vb, int kw, int slot0, int first, int len, int lane) {
    constexpr int kChunks = D * 2 / 16, kRowsAtOnce = 32 / kChunks;
    uint32_t mask = 0u;
#pragma unroll
    for (int r = 0; r < 16; r += kRowsAtOnce) {
        const int row = r + lane / kChunks;
        const uint32_t at = vb + chunk_off<D, 0>(kw + row, lane % kChunks);
        uint32_t top = 0u;
        if (slot0 + row >= first && slot0 + row < len) {
            const uint4 w = lds128(at);
            constexpr uint32_t kAbs = 0x7fff7fffu;
            top = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
        }
        const unsigned lanes = __ballot_sync(0xffffffffu, (top >> 16) >= 0x7f80u || (top & 0xffffu) >= 0x7f80u);
        const unsigned mine = (lanes >> (lane / kChunks * kChunks)) & ((1u << kChunks) - 1u);
        if (mine)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k)
            if ((lanes >> (k * kChunks)) & ((1u << kChunks) - 1u)) mask |= 1u << (r + k);
    }
    if (mask) fence_proxy_async_smem();   // the zeros before the next copy into this stage
    return mask;
}

// One warp: the B fragments of Q^T for rows row0 .. row0 + 8 NT - 1 of the K/V
// head whose rows start at rows_at, in the order the MMAs take them (fragment
// (n, step): 8 bytes a lane), and the rows' factors from the products to
// log2-unit scores.  Rows past the head's are zero.
template <int D, int kFmt, int NT>
__device__ __forceinline__ void q_fragments(const CacheDecodeParams& p, uint8_t* smem, int buf, size_t rows_at, int row0,
                                            int lane) {
    using L = CdLayout<D, kFmt, NT>;
    constexpr int kSteps = D / 16;
    const int g8 = lane >> 2, t4 = lane & 3, R = p.G * p.Nq;
    uint2* frag = reinterpret_cast<uint2*>(smem + L::kQ + buf * L::kQFrag) + lane;
    float* factor = reinterpret_cast<float*>(smem + L::kQScale) + buf * NT * 8;
    uint2 raw[NT][kSteps];   // all loads before the first use
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = row0 + n * 8 + g8;
        const __nv_bfloat16* qrow = reinterpret_cast<const __nv_bfloat16*>(p.q) + (rows_at + (r < R ? r : 0)) * D;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            raw[n][s] = make_uint2(0u, 0u);
            if (r < R) {
                if constexpr (kFmt != 0) {
                    // step s = 4 hh + w4: values (chunk of 16) * 16 + 4 w4 .. + 3
                    const int d = (D == 128 ? (2 * t4 + (s >> 2)) : t4) * 16 + (s & 3) * 4;
                    raw[n][s] = __ldg(reinterpret_cast<const uint2*>(qrow + d));
                } else {
                    const uint32_t* at = reinterpret_cast<const uint32_t*>(qrow + s * 16 + 2 * t4);
                    raw[n][s] = make_uint2(__ldg(at), __ldg(at + 4));
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if constexpr (kFmt != 0) {
            uint32_t am = 0u;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                am = __vmaxu2(am, __vmaxu2(raw[n][s].x & 0x7fff7fffu, raw[n][s].y & 0x7fff7fffu));
            am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, 2));
            // 2^(14 - exponent of the row's largest value); q = 0: any
            const int ex = static_cast<int>(max(am & 0xffffu, am >> 16) >> 7) - 127;
            const int f = min(max(14 - ex, -113), 126);
            const float up = __int_as_float((127 + f) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint2 w = raw[n][s];
                frag[(n * kSteps + s) * 32] =
                    make_uint2(pack_half2(__uint_as_float(w.x << 16) * up, __uint_as_float(w.x & 0xffff0000u) * up),
                               pack_half2(__uint_as_float(w.y << 16) * up, __uint_as_float(w.y & 0xffff0000u) * up));
            }
            if (t4 == 0) factor[n * 8 + g8] = pow2_inverse(up) * p.scale_log2;
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) frag[(n * kSteps + s) * 32] = raw[n][s];
            if (t4 == 0) factor[n * 8 + g8] = p.scale_log2;
        }
    }
}

// NT: blocks of 8 query rows a CTA holds.  kMixed: bf16 V rows that only some
// query rows see are looked at for infinities and NaNs (single queries, all keys
// visible and 8 bits have none; it is kept out of their code: 4 sequences of up to
// 130 slots of 8 heads of 128 take 5.4 us, with it 5.7).
template <int D, int kFmt, int NT, bool kMixed>
__global__ void __launch_bounds__(kCdThreads, CdLayout<D, kFmt, NT>::kCtas)
fa_cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const CacheDecodeParams p) {
    using L = CdLayout<D, kFmt, NT>;
    constexpr bool kHalf = kFmt != 0;
    constexpr int kStages = L::kStages;
    constexpr int kSteps = D / 16;
    constexpr float kShift = kHalf ? 6.f : 0.f;   // P is 2^kShift where the score is the row's (stale) maximum
    // Stands for kShift less the maximum of a row that has none yet: any finite
    // score plus it asks for a maximum, and -inf (a hidden key) stays -inf, no NaN.
    constexpr float kFar = FLT_MAX;
    extern __shared__ __align__(1024) uint8_t smem[];   // the swizzle's alignment
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint64_t* empty = full + kStages;
    uint64_t* q_full = empty + kStages;    // [2]
    uint64_t* q_empty = q_full + 2;        // [2]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kBar + (2 * kStages + 4) * 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    grid_launch_dependents();
    const int run = static_cast<int>(blockIdx.x) / p.RB, rb = static_cast<int>(blockIdx.x) - run * p.RB;
    const int row0 = rb * (8 * NT);                 // the CTA's first query row of every K/V head
    Walk w = find_run(p, run, static_cast<int>(gridDim.x) / p.RB, lane);
    bool more = w.settle(p);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 32);
            mbar_init(&q_empty[s], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        int issued = 0, unit = 0, st = 0;
        uint32_t phase = 1u;               // the first pass over the ring waits for nothing
        bool ok = true;
        for (; more && ok; w.step(p), more = w.settle(p), ++unit) {
            const int bkv = w.b * p.Hkv + w.h;
            for (int i = w.t0; i < w.t1; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], phase, abort_flag, kCdSiteEmpty));
                if (!ok) break;
                if (lane == 0) {
                    const int key0 = i * kCdKeys;
                    // the scales' rows end at the capacity, a multiple of 4
                    const uint32_t sbytes = kHalf ? static_cast<uint32_t>(min(kCdKeys, p.capacity - key0)) * 4u : 0u;
                    mbar_arrive_expect_tx(&full[st], 2 * L::kTileBytes + 2 * sbytes);
                    constexpr int kBox = D * L::kElem > 128 ? 2 : 1;
#pragma unroll
                    for (int a = 0; a < kBox; ++a)
                        tma_load_3d(smem + L::kK + st * L::kTileBytes + a * (L::kTileBytes / kBox), &tmK, &full[st],
                                    a * 64, key0, bkv);
#pragma unroll
                    for (int a = 0; a < kBox; ++a)
                        tma_load_3d(smem + L::kV + st * L::kTileBytes + a * (L::kTileBytes / kBox), &tmV, &full[st],
                                    a * 64, key0, bkv);
                    if constexpr (kHalf) {
                        const size_t at = static_cast<size_t>(bkv) * p.capacity + key0;
                        bulk_load(smem + L::kScales + st * 2 * L::kScaleBytes, p.k_scale + at, sbytes, &full[st]);
                        bulk_load(smem + L::kScales + st * 2 * L::kScaleBytes + L::kScaleBytes, p.v_scale + at, sbytes,
                                  &full[st]);
                    }
                }
                __syncwarp();
                ++issued;
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1u;
                }
                if (i == w.t0) {
                    // the unit's Q^T fragments, while its first tiles are under way
                    const int buf = unit & 1;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&q_empty[buf], ((unit >> 1) & 1) ^ 1, abort_flag, kCdSiteEmpty));
                    if (!ok) break;
                    q_fragments<D, kFmt, NT>(p, smem, buf, static_cast<size_t>(bkv) * (p.G * p.Nq), row0, lane);
                    mbar_arrive(&q_full[buf]);
                }
            }
        }
        // nothing may still be landing in shared memory when the CTA leaves
        if (lane == 0)
            for (int t = (issued > kStages ? issued - kStages : 0); t < issued; ++t)
                cd_drain(&full[t % kStages], (t / kStages) & 1);
        grid_wait();   // behind a prefix kernel: this one ends after it, as the combine expects
        return;
    }

    // ---------------------------------------------------------------- compute
    const int g8 = lane >> 2, t4 = lane & 3;
    const int kw = warp * 16;                       // this warp's 16 keys in a tile
    constexpr int kBlocks = D / 64;                 // and its blocks of 16 columns of V
    const uint32_t sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV), sS = smem_u32(smem + L::kScales);
    const uint32_t sQ = smem_u32(smem + L::kQ), sQScale = smem_u32(smem + L::kQScale);
    const uint32_t sP = smem_u32(smem + L::kP) + lane * 8;
    float* mx = reinterpret_cast<float*>(smem + L::kMx);   // [warp][8 NT], then [warp]
    float* ml = reinterpret_cast<float*>(smem + L::kMl);   // [warp][8 NT]
    const int R = p.G * p.Nq;
    // Where this lane reads in a K and in a V tile: the chunk of the first step;
    // chunk_at() gives the others (tile bases are multiples of the swizzle, and
    // so are 16 keys).
    //   8 bits  K: keys kw + g8 (+ 8), chunks 2 t4 + hh of 16 codes;
    //           V: matrices (keys lo, hi) x (chunks j, j + 1), at D = 64 (keys
    //           lo, hi) x (this 16 keys, the next)
    //   bf16    K: matrices (keys lo, hi) x (d lo, hi);  V: (d lo, hi) x (keys lo, hi)
    const int mi = lane >> 3;
    constexpr int kRow16 = 16 * (D * L::kElem > 128 ? 128 : D * L::kElem);   // bytes 16 keys are apart
    const uint32_t k_at = kHalf ? chunk_off<D, kFmt>(kw + g8, D == 128 ? 2 * t4 : t4)
                                : chunk_off<D, kFmt>(kw + (mi & 1) * 8 + (lane & 7), mi >> 1);
    const uint32_t v_at = !kHalf ? chunk_off<D, kFmt>((mi >> 1) * 8 + (lane & 7), 2 * kBlocks * warp + (mi & 1))
                          : D == 128 ? chunk_off<D, kFmt>((mi & 1) * 8 + (lane & 7), 2 * warp + (mi >> 1))
                                     : chunk_off<D, kFmt>(mi * 8 + (lane & 7), warp);
    bool ok = true;
    int unit = 0;
    int st = 0;            // ring stage and its parity
    uint32_t phase = 0u;
    uint32_t p_buf = 0u;   // offset of the tile's P fragments

    // After a wait that gave up, the remaining tiles are worked on as they are
    // and not written, so that the barriers stay matched.
    for (; more; w.step(p), more = w.settle(p)) {
        // ---- one unit, or the CTA's part of it
        const size_t rows_at = static_cast<size_t>(w.b * p.Hkv + w.h) * R;   // first query row of the K/V head
        const int buf = unit & 1;
        ok = ok && mbar_wait(&q_full[buf], (unit >> 1) & 1, abort_flag, kCdSiteFull);
        ok = __all_sync(0xffffffffu, ok);
        const uint32_t qf = sQ + buf * L::kQFrag + lane * 8;
        float qc[NT][2];      // factor to log2-unit scores, rows 2 t4, 2 t4 + 1
        int pos[NT][2];       // their last visible slot
        int pos_min = w.len - 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rr = row0 + n * 8 + 2 * t4 + h;
                pos[n][h] = p.causal ? w.len - p.Nq + (rr < R ? rr % p.Nq : 0) : w.len - 1;
                qc[n][h] = lds32(sQScale + (buf * NT * 8 + n * 8 + 2 * t4 + h) * 4);
            }
        if (p.causal) pos_min = w.len - p.Nq;

        float o[NT][kBlocks][4];
        // stale row maximum, kShift less it (kFar before the first key): the same in
        // all warps; partial row sum
        float m_run[NT][2], nm[NT][2], l_run[NT][2];
        float v_top = __int_as_float(1 << 23);   // power of two that bounds the V scales so far
        float v_inv = pow2_inverse(v_top);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
            m_run[n][0] = m_run[n][1] = -INFINITY;
            nm[n][0] = nm[n][1] = kFar;
            l_run[n][0] = l_run[n][1] = 0.f;
        }

        // One tile.  kEdge: some key of the warp's 16 is hidden from some row.
        auto tile = [&](auto edge_c, uint32_t kb, uint32_t vb, int key0) {
            constexpr bool kEdge = decltype(edge_c)::value;
            const int kA = key0 + g8, kB = kA + 8;           // this lane's two keys in S^T
            if (kEdge && key0 + 15 >= w.len) {
                // V rows behind the length may hold NaN, and 0 x NaN is NaN
                constexpr int kChunks = D * L::kElem / 16;
                for (int e = lane; e < 16 * kChunks; e += 32) {
                    const int row = kw + e / kChunks;
                    if (key0 + e / kChunks >= w.len)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                     ::"r"(vb + chunk_off<D, kFmt>(row, e % kChunks)), "r"(0u) : "memory");
                }
                fence_proxy_async_smem();   // the zeros before the next copy into this stage
            }
            // ---- S^T (16 keys x rows) = K Q^T; 8 rows alone in two halves, which
            // do not wait for one another
            float s[NT][4], s_odd[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s_odd[n][e] = 0.f;
            float ksA = 1.f, ksB = 1.f;
            [[maybe_unused]] float vsA, vsB;
            if constexpr (kHalf) {
                const uint32_t sc = sS + st * 2 * L::kScaleBytes + (kw + g8) * 4;
                ksA = lds32(sc);
                ksB = lds32(sc + 32);
                vsA = lds32(sc + L::kScaleBytes);
                vsB = lds32(sc + L::kScaleBytes + 32);
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh) {
                    const uint32_t at = chunk_at(kb + k_at, hh);
                    const uint4 ca = lds128(at), cb = lds128(at + 8 * D);
                    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
                    for (int w4 = 0; w4 < 4; ++w4) {
                        uint32_t a0, a1, a2, a3;
                        unpack4<kFmt>(wa[w4], a0, a2);
                        unpack4<kFmt>(wb[w4], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 q = lds64(qf + (n * kSteps + 4 * hh + w4) * 256);
                            mma16<true>(NT == 1 && (w4 & 1) ? s_odd[n] : s[n], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk) {
                    uint32_t a[4];
                    ldsm4(chunk_at(kb + k_at, 2 * kk), a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 q = lds64(qf + (n * kSteps + kk) * 256);
                        mma16<false>(NT == 1 && (kk & 1) ? s_odd[n] : s[n], a[0], a[1], a[2], a[3], q.x, q.y);
                    }
                }
            }
            if constexpr (NT == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][e] += s_odd[0][e];
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
                    if (kEdge && ((e >> 1) ? kB : kA) > pos[n][e & 1]) y[n][e] = -INFINITY;
                    grow |= y[n][e] > kShift + kCdRescale;
                }
            if constexpr (kHalf) {
                grow |= vsA > v_top && (!kEdge || kA < w.len);
                grow |= vsB > v_top && (!kEdge || kB < w.len);
            }
            // ---- P^T fragments of the warp's keys for all warps; again with new
            // maxima where a score of any warp asks for them
            float sum[NT][2];
            while (true) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float pw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) pw[e] = ex2(y[n][e]);
                    sum[n][0] = pw[0] + pw[2];
                    sum[n][1] = pw[1] + pw[3];
                    uint32_t lo, hi;
                    if constexpr (kHalf) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pw[e] *= ((e >> 1) ? vsB : vsA) * v_inv;
                            // a hidden key's scale may be anything
                            if (kEdge && y[n][e] == -INFINITY) pw[e] = 0.f;
                        }
                        lo = turn8x8(pack_half2(pw[0], pw[1]));
                        hi = turn8x8(pack_half2(pw[2], pw[3]));
                    } else {
                        lo = turn8x8(pack_bf16x2(pw[0], pw[1]));
                        hi = turn8x8(pack_bf16x2(pw[2], pw[3]));
                    }
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};"
                                 ::"r"(sP + p_buf + (warp * NT + n) * 256), "r"(lo), "r"(hi) : "memory");
                }
                if (!any_of_warps(grow)) break;
                // a maximum grew by more than kCdRescale, or a V scale past the
                // bound: take the new ones and bring the sums so far to them
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        y[n][h] = kEdge && y[n][h] == -INFINITY ? -INFINITY : s[n][h] * (ksA * qc[n][h]);
                        y[n][2 + h] = kEdge && y[n][2 + h] == -INFINITY ? -INFINITY : s[n][2 + h] * (ksB * qc[n][h]);
                        float top = fmaxf(y[n][h], y[n][2 + h]);
#pragma unroll
                        for (int k = 4; k <= 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                        if (g8 == 0) mx[warp * NT * 8 + n * 8 + 2 * t4 + h] = top;
                    }
                if constexpr (kHalf) {
                    float vm = fmaxf(!kEdge || kA < w.len ? vsA : 0.f, !kEdge || kB < w.len ? vsB : 0.f);
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, k));
                    if (lane == 0) mx[4 * NT * 8 + warp] = vm;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                float vfac = 1.f;
                if constexpr (kHalf) {
                    const float* at = mx + 4 * NT * 8;
                    const float top = fmaxf(v_top, pow2_at_least(fmaxf(fmaxf(at[0], at[1]), fmaxf(at[2], at[3]))));
                    v_inv = pow2_inverse(top);
                    vfac = v_top * v_inv;
                    v_top = top;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float alpha[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float* at = mx + n * 8 + 2 * t4 + h;
                        const float m_new = fmaxf(m_run[n][h], fmaxf(fmaxf(at[0], at[NT * 8]),
                                                                     fmaxf(at[2 * NT * 8], at[3 * NT * 8])));
                        alpha[h] = m_new == -INFINITY ? 1.f : ex2(m_run[n][h] - m_new);
                        m_run[n][h] = m_new;
                        nm[n][h] = m_new == -INFINITY ? kFar : kShift - m_new;
                        l_run[n][h] *= alpha[h];
                        alpha[h] *= vfac;
                        y[n][h] += nm[n][h];
                        y[n][2 + h] += nm[n][h];
                    }
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        o[n][j][0] *= alpha[0];
                        o[n][j][1] *= alpha[1];
                        o[n][j][2] *= alpha[0];
                        o[n][j][3] *= alpha[1];
                    }
                }
                grow = false;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l_run[n][0] += sum[n][0];
                l_run[n][1] += sum[n][1];
            }
            // ---- O^T (the warp's columns x rows) += V^T P^T over the tile's keys
            if constexpr (kHalf) {
#pragma unroll
                for (int x = 0; x < 4; x += 2) {
                    uint32_t r0[4], r1[4];
                    if constexpr (D == 128) {
                        ldsm4_t(vb + v_at + x * kRow16, r0);
                        ldsm4_t(vb + v_at + (x + 1) * kRow16, r1);
                    } else {
                        ldsm4_t(vb + v_at + x * kRow16, r0);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // D = 128: key step x + u, columns j of r0 / r1; D = 64: key step x + u in r0
                        uint2 pf[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) pf[n] = lds64(sP + p_buf + ((x + u) * NT + n) * 256);
#pragma unroll
                        for (int j = 0; j < kBlocks; ++j) {
                            const uint32_t* rr = D == 128 ? (u ? r1 : r0) + 2 * j : r0 + 2 * u;
                            uint32_t a0, a1, a2, a3;   // rows d = 2 g8 (a0, a2) and + 1 (a1, a3) of the block
                            unpack4_pairs<kFmt>(rr[0], a0, a1);
                            unpack4_pairs<kFmt>(rr[1], a2, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma16<true>(o[n][j], a0, a1, a2, a3, pf[n].x, pf[n].y);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint2 pf[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) pf[n] = lds64(sP + p_buf + (x * NT + n) * 256);
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        uint32_t r[4];
                        ldsm4_t(chunk_at(vb + v_at, 2 * j) + x * kRow16, r);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16<false>(o[n][j], r[0], r[1], r[2], r[3], pf[n].x, pf[n].y);
                    }
                }
            }
            p_buf ^= L::kPFrag;
        };

        for (int i = w.t0; i < w.t1; ++i) {
            ok = ok && mbar_wait(&full[st], phase, abort_flag, kCdSiteFull);
            ok = __all_sync(0xffffffffu, ok);
            const uint32_t kb = sK + st * L::kTileBytes, vb = sV + st * L::kTileBytes;
            const int key0 = i * kCdKeys + kw;               // slot of the warp's first key
            // bf16: the tile holds keys that some query rows see and others do not (the same
            // in all warps).  Double-buffered with P, so its barriers order the masks too.
            const bool mixed = kMixed && i * kCdKeys + kCdKeys - 1 > pos_min;
            const uint32_t p_at = sP - lane * 8 + p_buf;     // the tile's P fragments
            uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::kBad) + (p_buf ? 4 : 0);
            if constexpr (kMixed) {
                if (mixed) {
                    const uint32_t mask = take_poisoned<D>(vb, kw, key0, pos_min + 1, w.len, lane);
                    if (lane == 0) bad[warp] = mask;
                }
            }
            if (__any_sync(0xffffffffu, key0 + 15 > pos_min))
                tile(std::true_type{}, kb, vb, key0);
            else
                tile(std::false_type{}, kb, vb, key0);
            if constexpr (kMixed) {
                if (mixed) {
#pragma unroll 1
                    for (int x = 0; x < 4; ++x)
#pragma unroll 1
                        for (uint32_t left = bad[x]; left; left &= left - 1) {
                            const int key = __ffs(left) - 1, slot = i * kCdKeys + x * 16 + key;
                            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_cache) +
                                                     (static_cast<size_t>(w.b * p.Hkv + w.h) * p.capacity + slot) * D +
                                                     warp * (kBlocks * 16) + g8;
                            const uint32_t at = p_at + x * NT * 256 + (key >> 1 & 3) * 8 + (key >> 3) * 4 + (key & 1) * 2;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if (slot > pos[n][h]) continue;
                                    const float pw = lds_bf16(at + n * 256 + (2 * t4 + h) * 32);
#pragma unroll
                                    for (int j = 0; j < kBlocks; ++j) {
                                        o[n][j][h] = fmaf(pw, __bfloat162float(v[j * 16]), o[n][j][h]);
                                        o[n][j][2 + h] = fmaf(pw, __bfloat162float(v[j * 16 + 8]), o[n][j][2 + h]);
                                    }
                                }
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0) mbar_arrive(&q_empty[buf]);

        // ---- row sums over the warps, and the results
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) l_run[n][h] += __shfl_xor_sync(0xffffffffu, l_run[n][h], k);
                if (g8 == 0) ml[warp * NT * 8 + n * 8 + 2 * t4 + h] = l_run[n][h];
            }
        // (the next unit's writes to ml come after another tile's barrier)
        asm volatile("bar.sync 1, 128;" ::: "memory");
        // a part that begins before this CTA goes to its slot 2 c, one that ends after it to 2 c + 1
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        const int slot = 2 * static_cast<int>(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
        if (w.t0 == 0 && threadIdx.x == 0 && p.meta != nullptr) {
            const long long end = w.at + p.unit_cost + w.tiles;                      // past the last tile
            const int last = static_cast<int>((end * w.n - 1) / w.total);            // its run
            p.meta[(w.b * p.Hkv + w.h) * p.RB + rb] = make_int2(whole ? -1 : slot, whole ? 1 : last - run + 1);
        }
        const bool final_rows = whole && p.o_unit == nullptr;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + n * 8 + 2 * t4 + h;
                const float* at = ml + n * 8 + 2 * t4 + h;
                const float Lsum = (at[0] + at[NT * 8]) + (at[2 * NT * 8] + at[3 * NT * 8]);
                // rows without a key: 0; a NaN sum stays NaN
                const float inv = Lsum == 0.f ? 0.f : (kHalf ? v_top : 1.f) / Lsum;
                if (row >= R || !ok) continue;
                const size_t prow = final_rows || whole ? rows_at + row
                                                        : static_cast<size_t>(slot) * (8 * NT) + n * 8 + 2 * t4 + h;
                if (warp == 0 && g8 == 0) {
                    float* lse = final_rows ? p.lse : whole ? p.lse_unit : p.lse_part;
                    lse[prow] = Lsum == 0.f ? -INFINITY : (m_run[n][h] + log2f(Lsum) - kShift) * kLn2;
                }
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    // 8 bits: columns 2 g8, 2 g8 + 1 of the block; bf16: g8, g8 + 8
                    const int d = (warp * kBlocks + j) * 16;
                    const float v0 = o[n][j][h] * inv, v1 = o[n][j][2 + h] * inv;
                    if (final_rows) {
                        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.o) + prow * D + d;
                        if constexpr (kHalf) {
                            *reinterpret_cast<uint32_t*>(out + 2 * g8) = pack_bf16x2(v0, v1);
                        } else {
                            out[g8] = __float2bfloat16_rn(v0);
                            out[g8 + 8] = __float2bfloat16_rn(v1);
                        }
                    } else {
                        float* out = (whole ? p.o_unit : p.o_part) + prow * D + d;
                        if constexpr (kHalf) {
                            *reinterpret_cast<float2*>(out + 2 * g8) = make_float2(v0, v1);
                        } else {
                            out[g8] = v0;
                            out[g8 + 8] = v1;
                        }
                    }
                }
            }
        ++unit;
    }
    grid_wait();
}

// Joins the parts of a query row: those of the CTAs that share its unit, and
// the prefix's.
//   LSE = log sum_s exp(LSE_s),   O = sum_s exp(LSE_s - LSE) O_s
// kWarps warps a row, every kWarps-th part each: a lane finds one part and its
// weight, so that the loads of the parts' rows that follow depend on nothing.
template <int D, int kWarps>
__global__ void __launch_bounds__(128)
fa_cache_combine_kernel(const CacheDecodeParams p, const PrefixParams f, int n_rows) {
    constexpr int kPer = D / 32;
    __shared__ float sh_m[4], sh_z[4];
    __shared__ float sh_o[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % kWarps;
    const int R = p.G * p.Nq;
    const int gr = static_cast<int>(blockIdx.x) * (4 / kWarps) + warp / kWarps;   // row of [B, Hq, Nq]
    if (gr >= n_rows) return;                         // kWarps == 4: the grid is exact
    const int bkv = gr / R, r = gr - bkv * R;
    const int b = bkv / p.Hkv, hkv = bkv - b * p.Hkv;
    const int rb = r / p.rows_cta, in = r - rb * p.rows_cta;
    grid_wait();                                      // the main kernel's results, and the prefix's
    const int2 meta = p.meta[bkv * p.RB + rb];
    const bool whole = meta.x < 0;
    if (whole && f.n_cta == 0) return;                // written by the main kernel
    const int own = whole ? 1 : meta.y;
    // the prefix unit that holds the row, and the CTAs that share it
    int np = 0, pin = 0;
    size_t pslot = 0;
    if (f.n_cta > 0) {
        const int prow = b * R + r;
        const int pu = hkv * f.n_rowtiles + prow / f.rows_unit;
        pin = prow % f.rows_unit;
        const long long total = static_cast<long long>(f.Hkv) * f.n_rowtiles * f.n_tiles;
        const long long ts = static_cast<long long>(pu) * f.n_tiles;
        const int first = static_cast<int>(((ts + 1) * f.n_cta - 1) / total);
        np = static_cast<int>(((ts + f.n_tiles) * f.n_cta - 1) / total) - first + 1;
        pslot = static_cast<size_t>(first + pu);
    }
    const int n = own + np;
    float M = -INFINITY, Z = 0.f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int s0 = sub; s0 < n; s0 += 32 * kWarps) {
        const int s = s0 + lane * kWarps;
        const float* o = nullptr;
        float lse = -INFINITY;
        if (s < n) {
            size_t prow;
            if (s >= own) {
                prow = (pslot + static_cast<size_t>(s - own)) * f.rows_unit + pin;
                o = f.o_part + prow * D;
                lse = f.lse_part[prow];
            } else if (whole) {
                o = p.o_unit + static_cast<size_t>(gr) * D;
                lse = p.lse_unit[gr];
            } else {
                prow = static_cast<size_t>(s == 0 ? meta.x : 2 * ((meta.x >> 1) + s * p.RB)) * p.rows_cta + in;
                o = p.o_part + prow * D;
                lse = p.lse_part[prow];
            }
        }
        float top = lse;                              // NaN leaves the maximum alone and its weight NaN
#pragma unroll
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float m_new = fmaxf(M, top);
        const float a = m_new == -INFINITY ? 1.f : expf(M - m_new);
        // -1: a part without a key, whose o is to be left alone; a weight that only
        // underflows to 0 still meets its o, so that a NaN there stays one
        const float e = lse == -INFINITY ? -1.f : expf(lse - m_new);
        M = m_new;
        Z = Z * a;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] *= a;
        const int here = min(32, (n - s0 + kWarps - 1) / kWarps);
#pragma unroll 8
        for (int j = 0; j < here; ++j) {
            const float w = __shfl_sync(0xffffffffu, e, j);
            const float* oj = reinterpret_cast<const float*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), j));
            Z = w < 0.f ? Z : Z + w;
            float v[kPer];
            if constexpr (kPer == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(oj) + lane);
                v[0] = x.x;
                v[1] = x.y;
                v[2] = x.z;
                v[3] = x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2*>(oj) + lane);
                v[0] = x.x;
                v[1] = x.y;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = w < 0.f ? acc[i] : fmaf(w, v[i], acc[i]);
        }
    }
    if constexpr (kWarps > 1) {
        if (lane == 0) {
            sh_m[warp] = M;
            sh_z[warp] = Z;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) sh_o[warp][lane * kPer + i] = acc[i];
        __syncthreads();
        if (sub != 0) return;
        M = -INFINITY;
        Z = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) M = fmaxf(M, sh_m[q]);
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            const float e = sh_z[q] == 0.f ? 0.f : expf(sh_m[q] - M);
            Z += e * sh_z[q];
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += e * sh_o[q][lane * kPer + i];
        }
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + static_cast<size_t>(gr) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0) p.lse[gr] = Z == 0.f ? -INFINITY : M + logf(Z);
}

template <int D, int kFmt, int NT, bool kMixed>
cudaError_t go(const CUtensorMap& tk, const CUtensorMap& tv, const CacheDecodeParams& p, bool after_prefix,
               cudaStream_t stream) {
    auto kern = fa_cache_decode_kernel<D, kFmt, NT, kMixed>;
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.set(reinterpret_cast<const void*>(kern), CdLayout<D, kFmt, NT>::kAlloc);
    if (e != cudaSuccess) return e;
    constexpr int kSmem = CdLayout<D, kFmt, NT>::kAlloc;
    if (after_prefix) return launch_dependent(kern, p.n_cta, kCdThreads, kSmem, stream, tk, tv, p);
    kern<<<p.n_cta, kCdThreads, kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

template <int D, int kFmt, bool kMixed>
cudaError_t go_rows(const CUtensorMap& tk, const CUtensorMap& tv, const CacheDecodeParams& p, bool after_prefix,
                    cudaStream_t stream) {
    if (p.rows_cta == 8) return go<D, kFmt, 1, kMixed>(tk, tv, p, after_prefix, stream);
    if (p.rows_cta == 16) return go<D, kFmt, 2, kMixed>(tk, tv, p, after_prefix, stream);
    return go<D, kFmt, 4, kMixed>(tk, tv, p, after_prefix, stream);
}

template <int D>
cudaError_t go_fmt(int fmt, const CUtensorMap& tk, const CUtensorMap& tv, const CacheDecodeParams& p,
                   bool after_prefix, cudaStream_t stream) {
    if (fmt == 0)
        return p.causal && p.Nq > 1 ? go_rows<D, 0, true>(tk, tv, p, after_prefix, stream)
                                    : go_rows<D, 0, false>(tk, tv, p, after_prefix, stream);
    if (fmt == 1) return go_rows<D, 1, false>(tk, tv, p, after_prefix, stream);
    return go_rows<D, 2, false>(tk, tv, p, after_prefix, stream);
}

}  // namespace

int cache_decode_ctas_per_sm(int D, int fmt, int rows_cta) {
    return rows_cta == 32 || (D == 128 && fmt == 0) ? 2 : 3;
}

// Measured at a cost of 0, 1, 2, 3, 4 and 6 with 64 sequences of up to 1000 slots
// (8 rows, with the join): e4m3 at D = 128 31.9, 24.6, 22.0, 22.0, 22.3, 22.7 us, at
// 64 27.5, 21.2, 17.5, 17.2, 16.9, 17.1; bf16 at 128 36.0, 31.5, 31.5, 31.5, 32.0,
// 32.5, at 64 27.6, 21.0, 20.1, 20.4, 20.5, 20.9.  With 48 of up to 8100 (12 rows):
// e4m3 at 128 52.7, 49.2, 46.2, 45.4, 45.6, 45.9, at 64 42.6, 39.9, 37.5, 34.9,
// 33.8, 33.6; bf16 at 128 77.8, 73.8, 71.8, 71.7, 71.8, 72.6, at 64 50.4, 46.5,
// 44.1, 43.2, 43.2, 43.1.
int cache_decode_unit_cost(int rows_cta) { return rows_cta == 8 ? 2 : 4; }

cudaError_t launch_cache_decode(int D, int fmt, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, bool after_prefix, cudaStream_t stream) {
    return D == 128 ? go_fmt<128>(fmt, tk, tv, p, after_prefix, stream)
                    : go_fmt<64>(fmt, tk, tv, p, after_prefix, stream);
}

cudaError_t launch_cache_combine(int D, const CacheDecodeParams& p, const PrefixParams& f, cudaStream_t stream) {
    const int rows = p.B * p.Hkv * p.G * p.Nq;
    // One warp a row once that fills the SMs; below, four share a row's parts,
    // of which there are the more the fewer rows there are.
    const bool many = rows >= 1024;
    const unsigned grid = many ? static_cast<unsigned>((rows + 3) / 4) : static_cast<unsigned>(rows);
    if (D == 128)
        return many ? launch_dependent(fa_cache_combine_kernel<128, 1>, grid, 128u, 0, stream, p, f, rows)
                    : launch_dependent(fa_cache_combine_kernel<128, 4>, grid, 128u, 0, stream, p, f, rows);
    return many ? launch_dependent(fa_cache_combine_kernel<64, 1>, grid, 128u, 0, stream, p, f, rows)
                : launch_dependent(fa_cache_combine_kernel<64, 4>, grid, 128u, 0, stream, p, f, rows);
}

}  // namespace fa
