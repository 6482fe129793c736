/*
 * fa_cache.h — a K/V cache at 16 or 8 bits: writing it, reading it back, and
 * decoding over it, with or without a prefix that the whole batch shares
 * (C ABI, companion of fa.h).
 *
 * The cache.  k_cache, v_cache [B, Hkv, capacity, D] contiguous, one slot for
 * each token; sequence b fills slots 0 .. len_b - 1.  Slots behind a
 * sequence's length may hold anything.  Formats:
 *   FA_CACHE_BF16  bf16 values
 *   FA_CACHE_E4M3  1-byte e4m3 codes (OCP FP8 E4M3) with one fp32 scale a row
 *   FA_CACHE_INT8  1-byte signed codes with one fp32 scale a row
 * k_scale, v_scale fp32 [B, Hkv, capacity] (NULL for bf16), from 0 to 2^126 or
 * NaN: a code stands for code * scale.  The writer's rules, for a row with
 * largest magnitude amax:
 *   e4m3  scale = 2^e with the smallest e >= -120 such that amax <= 448 * 2^e
 *         (dividing by it is exact, so a value is rounded once, to the nearest
 *         code, ties to even; a scale that is no power of two would gain no
 *         precision in a floating format)
 *   int8  scale = amax / 127 rounded to fp32, at least 2^-120; code = x / scale
 *         rounded to the nearest integer, ties to even
 * A row with an infinity or a NaN gets codes 0 and the scale NaN: it reads
 * back as NaN, and a query that sees it becomes NaN.
 *
 * Ownership, streams, errors: as in fa.h.  Calls are asynchronous on `stream`,
 * allocate nothing and can be captured into a CUDA graph; lengths and slots
 * live in device memory, so a captured call follows them.  Device lengths and
 * slots are clamped by the kernels: no value of them reads or writes out of
 * the cache.
 */
#ifndef TILED_ATTENTION_FA_CACHE_H
#define TILED_ATTENTION_FA_CACHE_H

#include "fa_rope.h" /* fa_rows */

#ifdef __cplusplus
extern "C" {
#endif

#define FA_CACHE_BF16 0
#define FA_CACHE_E4M3 1
#define FA_CACHE_INT8 2

/* D = 64 or 128 (FA_ERR_UNSUPPORTED otherwise); capacity >= 1, a multiple of
 * 4 for the 8-bit formats (the rows of scales start on 16 bytes); B * Hkv <=
 * 65535.  A write or read of N rows a head takes B * Hkv * N <= 2^31 - 1. */
typedef struct {
    int B, Hkv, capacity, D;
    int format;
} fa_cache_shape;

/* Writes row n of sequence b into slot start[b] + n, for n < count[b] (count
 * NULL: all N rows).  k, v: bf16 views [B,Hkv,N,D] (see fa_rows; v may have
 * other strides than k).  start, count: int32 [B] on the device.  Rows whose
 * slot is not in 0 .. capacity - 1 are dropped; slots that no row goes to are
 * left as they are.  Caches 16-byte aligned, scales 16-byte.  k and v share no
 * memory with the caches (rows are not moved within one). */
FA_API fa_status fa_cache_write(const fa_cache_shape* shape, int N, const fa_rows* k, const fa_rows* v,
                                const int* start, const int* count, void* k_cache, void* v_cache, float* k_scale,
                                float* v_scale, void* stream);

/* Reads slots 0 .. N - 1 of every sequence back: k_out, v_out bf16
 * [B,Hkv,N,D] contiguous, bf16(code * scale); rows at or behind lens[b]
 * (int32 [B] on the device; NULL: capacity) become 0.  1 <= N <= capacity.  The
 * outputs share no memory with the cache. */
FA_API fa_status fa_cache_read(const fa_cache_shape* shape, int N, const int* lens, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale, void* k_out,
                               void* v_out, void* stream);

/* Decoding: Nq new queries of each sequence over the prefix (n_prefix keys,
 * the same for all of the batch; 0: none) followed by the sequence's own
 * slots.  Query i stands at slot len_b - Nq + i: when causal != 0 it sees
 * slots j <= len_b - Nq + i, else all slots below len_b; it always sees the
 * whole prefix.  A key whose score is -inf counts as not seen (as in
 * fa_decode) if its V row is finite.  A query that sees no key gets o = 0 and
 * lse = -inf.
 * Hq % Hkv == 0; Nq >= 1; scale finite and > 0.  Beyond the cache's limits:
 * B * Hq * Nq <= FA_CACHE_MAX_ROWS; capacity <= 2^31 - 64, and with R = Hq / Hkv
 * * Nq, B * Hkv * (ceil(capacity / 64) + (R <= 8 ? 2 : 4)) <= 2^31 - 1; n_prefix
 * <= 2^31 - 256, and Hkv * ceil(B * R / U) * ceil(n_prefix / 128) <= 2^31 - 1 with
 * U = 128 for B * R <= 128, else 256. */
#define FA_CACHE_MAX_ROWS (1 << 24)
typedef struct {
    int B, Hq, Hkv, Nq, capacity, n_prefix, D;
    int format;
    float scale;
    int causal;
} fa_cache_decode_shape;

/* Bytes of device workspace fa_decode_cache needs: 0 for caches of up to
 * FA_CACHE_UNDIVIDED slots without a prefix (each sequence's head is one CTA's
 * work there), and if the shape is invalid or there is no CUDA device. */
#define FA_CACHE_UNDIVIDED 512
FA_API size_t fa_decode_cache_workspace_bytes(const fa_cache_decode_shape* shape);

/* q [B,Hq,Nq,D] bf16; the cache as above, with lens int32 [B] on the device
 * (clamped to 0 .. capacity); k_prefix, v_prefix bf16 [Hkv,n_prefix,D] (NULL
 * when n_prefix is 0).  o [B,Hq,Nq,D] bf16, lse [B,Hq,Nq] fp32 (natural log).
 * The prefix is read once for the whole batch: its rows of all sequences meet
 * it as one matrix.  The 8-bit formats multiply in fp16 on the codes (exact
 * there), q scaled by a power of two for each row; scales enter in fp32.  P
 * times the V scales is rounded to fp16 (2^-11 of each weight, and for weights
 * far below the largest up to 2^-30 of the largest V value below the sequence's
 * length, seen by the query or not); with bf16 caches and prefixes P is rounded
 * to bf16 (2^-8).
 * workspace: 256-byte aligned (NULL allowed where 0 bytes are needed), contents
 * on entry do not matter; calls that may overlap need workspaces of their own.
 * o, lse and the workspace share no memory with the inputs.  8-bit codes below a
 * sequence's length must be numbers (the writer's always are).  bf16 caches and
 * prefixes may hold infinities and NaNs: a query that sees such a value in a row
 * of V gets no finite number in its column, whatever the row's weight; a query
 * that does not see the row is not touched by it. */
FA_API fa_status fa_decode_cache(const fa_cache_decode_shape* shape, const void* q, const void* k_cache,
                                 const void* v_cache, const float* k_scale, const float* v_scale, const int* lens,
                                 const void* k_prefix, const void* v_prefix, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_FA_CACHE_H */
