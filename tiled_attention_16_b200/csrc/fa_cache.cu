// fa_cache.cu — writing K/V rows into a cache at 16 or 8 bits, and reading
// them back (include/fa_cache.h has the formats and the rounding rules).
//
// A write reads 2 bytes an element and writes 1 or 2, a read the other way round.
// 8 sequences of 2048 tokens, 32 heads of 128: bf16 write 82 us (6.6 TB/s), e4m3
// 71 (5.8), both bound by HBM; int8 130 us for the bytes of e4m3, bound by the
// instructions of its rounding (code_int8).  3548 slots back: e4m3 and int8 103 us
// (6.6 TB/s), bf16 132.  D / 8 lanes hold a row, 8 values each (16-byte accesses
// on the bf16 side, 8-byte on the codes); a thread takes kRows rows and issues
// their loads together.  blockIdx.y is 0 for K and 1 for V.
#include "fa_serving.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace fa {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kRows = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest magnitude of the row as bf16 bits (sign cleared); infinities and
// NaNs are the values from 0x7f80 on, so they win the integer maximum.
template <int kLanes>
__device__ __forceinline__ uint32_t row_amax_bits(const uint4& w) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
#pragma unroll
    for (int k = kLanes / 2; k; k >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, k));
    return max(m & 0xffffu, m >> 16);
}

// 8 values to e4m3 codes.  The scale is 2^e with the smallest e >= -120 such
// that amax <= 448 * 2^e = 1.75 * 2^(8 + e): from the exponent and the seven
// mantissa bits of amax.  Multiplying by 2^-e is exact (values that leave the
// fp32 range downwards are far below half of the smallest code), so a value is
// rounded once, by the conversion.
__device__ __forceinline__ uint2 codes_e4m3(const uint4& w, uint32_t amax, float& scale) {
    int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    e = max(e, -120);
    scale = __int_as_float((127 + e) << 23);
    const float inv = __int_as_float((127 - e) << 23);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(v[2 * i]) * inv, bf16_hi(v[2 * i]) * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(bf16_lo(v[2 * i + 1]) * inv, bf16_hi(v[2 * i + 1]) * inv), __NV_SATFINITE, __NV_E4M3);
        c[i] = lo | (hi << 16);
    }
    return make_uint2(c[0], c[1]);
}

// Nearest integer to x / s, ties to even, exactly: x times the rounded 1 / s
// gives the integer up to one, and the residual x - q s is exact in fp32 (x has
// 8 significant bits and |x| >= s / 2 where q != 0, so it is a multiple of s's
// last bit below 2 s), so comparing it with s / 2 settles the rest.
__device__ __forceinline__ int code_int8(float x, float s, float inv) {
    const float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), h = 0.5f * s;
    int i = static_cast<int>(q);
    const int odd = i & 1;
    if (r > h || (r == h && odd)) ++i;
    if (r < -h || (r == -h && odd)) --i;
    return i;
}

__device__ __forceinline__ uint2 codes_int8(const uint4& w, uint32_t amax, float& scale) {
    scale = fmaxf(__fdiv_rn(__uint_as_float(amax << 16), 127.f), 7.52316385e-37f);   // 2^-120
    const float inv = __fdiv_rn(1.f, scale);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = static_cast<uint32_t>(code_int8(bf16_lo(v[i]), scale, inv)) & 0xffu;
        const uint32_t hi = static_cast<uint32_t>(code_int8(bf16_hi(v[i]), scale, inv)) & 0xffu;
        c[i >> 1] |= (lo | (hi << 8)) << (16 * (i & 1));
    }
    return make_uint2(c[0], c[1]);
}

// A CTA writes a tile of (rows / heads) tokens x heads of one sequence; heads
// is 1 unless there are fewer tokens than the tile has rows.  (Tiles of four
// heads where the rows lie token by token, heads inside, took as long.)
template <int D, int kFmt>
__global__ void __launch_bounds__(kCacheThreads)
fa_cache_write_kernel(const CacheWriteParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kSlots = kCacheThreads / kLanes;
    const int lane = threadIdx.x & (kLanes - 1);
    const RopeRows& x = blockIdx.y ? p.v : p.k;
    uint8_t* cache = static_cast<uint8_t*>(blockIdx.y ? p.v_cache : p.k_cache);
    float* scales = blockIdx.y ? p.v_scale : p.k_scale;
    const int shift = p.shift;   // log2 of the tile's heads
    const unsigned n_tiles = (static_cast<unsigned>(p.N) + (kSlots * kRows >> shift) - 1) / (kSlots * kRows >> shift);
    const unsigned h_tiles = (static_cast<unsigned>(p.H) + (1u << shift) - 1) >> shift;
    const unsigned per = n_tiles * h_tiles;
    const unsigned b = blockIdx.x / per, in = blockIdx.x - b * per;
    // this thread's first row, and what the tokens of its others are apart
    const int r = static_cast<int>(threadIdx.x / kLanes);
    const int n = static_cast<int>(in / h_tiles * (kSlots * kRows >> shift)) + (r >> shift);
    const int h = static_cast<int>((in % h_tiles) << shift) + (r & ((1 << shift) - 1));
    const int dn = kSlots >> shift;
    // tokens n in [lo, hi) have a slot
    const long long start = __ldg(p.start + b);
    const int cnt = p.count ? min(__ldg(p.count + b), p.N) : p.N;
    const int lo = static_cast<int>(min(max(0ll, -start), static_cast<long long>(p.N)));
    const int hi = h < p.H ? static_cast<int>(max(min(static_cast<long long>(cnt), p.capacity - start), -1ll)) : -1;
    const uint4* src = reinterpret_cast<const uint4*>(x.data + b * x.stride_b + h * x.stride_h + n * x.stride_n) + lane;
    const long long step = dn * x.stride_n / 8;
    const size_t slot = static_cast<size_t>((static_cast<long long>(b) * p.H + h) * p.capacity + start + n);
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (n + i * dn >= lo && n + i * dn < hi) raw[i] = __ldg(src + i * step);
    }
    uint8_t* dst = cache + slot * (kFmt == 0 ? 2 * D : D) + lane * (kFmt == 0 ? 16 : 8);
    float* scale_at = kFmt == 0 ? nullptr : scales + slot;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const bool real = n + i * dn >= lo && n + i * dn < hi;
        if constexpr (kFmt == 0) {
            if (real) *reinterpret_cast<uint4*>(dst) = raw[i];
            dst += dn * (2 * D);
        } else {
            const uint32_t amax = row_amax_bits<kLanes>(raw[i]);
            float scale;
            uint2 c = kFmt == 1 ? codes_e4m3(raw[i], amax, scale) : codes_int8(raw[i], amax, scale);
            if (amax >= 0x7f80u) {   // an infinity or a NaN: the whole row reads back as NaN
                c = make_uint2(0u, 0u);
                scale = __uint_as_float(0x7fc00000u);
            }
            if (real) {
                *reinterpret_cast<uint2*>(dst) = c;
                if (lane == 0) *scale_at = scale;
            }
            dst += dn * D;
            scale_at += dn;
        }
    }
}

// A CTA reads consecutive slots of one (sequence, head).
template <int D, int kFmt>
__global__ void __launch_bounds__(kCacheThreads)
fa_cache_read_kernel(const CacheReadParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kSlots = kCacheThreads / kLanes;
    const int lane = threadIdx.x & (kLanes - 1);
    const uint8_t* cache = static_cast<const uint8_t*>(blockIdx.y ? p.v_cache : p.k_cache);
    const float* scales = blockIdx.y ? p.v_scale : p.k_scale;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(blockIdx.y ? p.v_out : p.k_out);
    const unsigned tiles = (static_cast<unsigned>(p.N) + kSlots * kRows - 1) / (kSlots * kRows);
    const unsigned bh = blockIdx.x / tiles;
    const int n = static_cast<int>((blockIdx.x - bh * tiles) * (kSlots * kRows) + threadIdx.x / kLanes);
    const int len = p.lens ? min(__ldg(p.lens + bh / static_cast<unsigned>(p.H)), p.capacity) : p.capacity;
    const size_t slot = static_cast<size_t>(bh) * p.capacity + n;
    const uint8_t* src = cache + slot * (kFmt == 0 ? 2 * D : D) + lane * (kFmt == 0 ? 16 : 8);
    uint4 raw[kRows];
    float scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);   // rows behind the length: codes 0, scale 0
        scale[i] = 0.f;
        if (n + i * kSlots < min(len, p.N)) {
            if constexpr (kFmt == 0) {
                raw[i] = __ldg(reinterpret_cast<const uint4*>(src + i * kSlots * 2 * D));
            } else {
                const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + i * kSlots * D));
                raw[i].x = c.x;
                raw[i].y = c.y;
                scale[i] = __ldg(scales + slot + i * kSlots);
            }
        }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<size_t>(bh) * p.N + n) * D) + lane;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (n + i * kSlots >= p.N) break;
        uint4 o = raw[i];
        if constexpr (kFmt != 0) {
            const uint32_t c[2] = {raw[i].x, raw[i].y};
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = c[j >> 1] >> (16 * (j & 1));
                float2 f;
                if constexpr (kFmt == 1) {
                    const __half2_raw hr =
                        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
                    f = __half22float2(__half2(hr));
                } else {
                    f = make_float2(static_cast<float>(static_cast<int8_t>(two & 0xffu)),
                                    static_cast<float>(static_cast<int8_t>((two >> 8) & 0xffu)));
                }
                w[j] = pack_bf16x2(f.x * scale[i], f.y * scale[i]);
            }
            o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        dst[i * kSlots * (D / 8)] = o;
    }
}

template <class F>
cudaError_t cache_dispatch(int D, int fmt, F&& go) {
    auto with_d = [&](auto d) {
        if (fmt == 0) return go(d, std::integral_constant<int, 0>{});
        if (fmt == 1) return go(d, std::integral_constant<int, 1>{});
        return go(d, std::integral_constant<int, 2>{});
    };
    return D == 128 ? with_d(std::integral_constant<int, 128>{}) : with_d(std::integral_constant<int, 64>{});
}

}  // namespace

cudaError_t launch_cache_write(int D, int fmt, CacheWriteParams p, cudaStream_t stream) {
    const int slots = kCacheThreads / (D / 8), rows = slots * kRows;
    // Heads of a tile: with fewer tokens than rows as many as fill the tile, but
    // at most one a row slot (a thread's rows are tokens of one head).
    p.shift = 0;
    while ((rows >> p.shift) / 2 >= p.N && (1 << p.shift) < p.H && (2 << p.shift) <= slots) ++p.shift;
    const long long tn = rows >> p.shift, th = 1LL << p.shift;
    const dim3 grid(static_cast<unsigned>(p.B * ((p.N + tn - 1) / tn) * ((p.H + th - 1) / th)), 2);
    return cache_dispatch(D, fmt, [&](auto d, auto f) {
        fa_cache_write_kernel<decltype(d)::value, decltype(f)::value><<<grid, kCacheThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_cache_read(int D, int fmt, const CacheReadParams& p, cudaStream_t stream) {
    const int rows = kCacheThreads / (D / 8) * kRows;
    const dim3 grid(static_cast<unsigned>(p.BH) * static_cast<unsigned>((p.N + rows - 1) / rows), 2);
    return cache_dispatch(D, fmt, [&](auto d, auto f) {
        fa_cache_read_kernel<decltype(d)::value, decltype(f)::value><<<grid, kCacheThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace fa
