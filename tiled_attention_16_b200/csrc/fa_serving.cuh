// fa_serving.cuh — what the operators around the attention share: launch
// interface of their kernels (host side: fa_cache_api.cu) and their device
// helpers.  Apart from fa_internal.h and sm100.cuh, which the attention kernels'
// recorded measurements are keyed by.
#pragma once

#include "fa_internal.h"
#include "sm100.cuh"

#include <atomic>

#include <cuda_bf16.h>

namespace fa {

// Programmatic dependent launch: let the next kernel of the stream (if it was
// launched so) start, and wait until the kernel before has completed and its
// writes are visible.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 lanes x 32 consecutive 32-bit columns, eight columns (256 bits) at a time:
// thread 4 g + t gets, for column block c, r[4c], r[4c + 1] = lane g, columns
// 8c + 2t, + 1 and r[4c + 2], r[4c + 3] = lane g + 8, the same columns.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Raises a kernel's dynamic shared memory limit, once per device (the call
// costs about as much as half a launch).
struct SmemOptIn {
    std::atomic<bool> done[64] = {};
    cudaError_t set(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool known = dev >= 0 && dev < 64;
        if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
        return e;
    }
};

// Launch of a kernel that may start before the kernel ahead of it in the stream
// has ended; it waits for it itself (grid_wait) where it needs its results, and
// in any case before it ends.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                             const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// bf16 rows of D contiguous values, indexed [b, h, n] by strides in elements.
struct RopeRows {
    __nv_bfloat16* data;
    long long stride_b, stride_h, stride_n;
};

// Per-head norm with rotation (fa_rope.cu); q_out / k_out are written by the
// forward, the d* fields are the backward's.
struct RopeParams {
    RopeRows q, k, dq, dk;
    __nv_bfloat16 *q_out, *k_out;
    const __nv_bfloat16 *dq_out, *dk_out;
    const void *q_weight, *k_weight;
    const float* inv_freq;
    const int* positions;
    float* dw_part;    // [CTAs, 2, D]
    int Hq, Hkv, N, rot, weight_bf16;
    float eps;
    long long tokens;  // B * N
    int token_slots, parts_q, parts_k, items_q, n_items;   // filled by the launch
};
int rope_bwd_ctas(int sms);
cudaError_t launch_qk_norm_rope(int D, int interleaved, RopeParams p, int sms, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(int D, int interleaved, RopeParams p, float* dqw, float* dkw, int sms,
                                    cudaStream_t stream);

// Cache writes and reads (fa_cache.cu).
struct CacheWriteParams {
    RopeRows k, v;
    const int *start, *count;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int B, H, N, capacity;
    int shift;               // log2 of a tile's heads; filled by the launch
};
struct CacheReadParams {
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int* lens;
    void *k_out, *v_out;
    int BH, H, N, capacity;
};
cudaError_t launch_cache_write(int D, int fmt, CacheWriteParams p, cudaStream_t stream);
cudaError_t launch_cache_read(int D, int fmt, const CacheReadParams& p, cudaStream_t stream);

// Decoding over a cache (fa_cache_decode.cu).
struct CacheDecodeParams {
    const void* q;           // bf16 [B,Hq,Nq,D]
    void* o;                 // bf16 [B,Hq,Nq,D]
    float* lse;              // fp32 [B,Hq,Nq]
    const int* lens;
    const float *k_scale, *v_scale;
    const void* v_cache;     // read directly where a bf16 row holds an infinity or a NaN
    float *o_part, *lse_part;  // parts of units shared by CTAs: slots 2 c, 2 c + 1 of rows_cta rows each
    float *o_unit, *lse_unit;  // [B*Hq*Nq, D], [B*Hq*Nq]: undivided units' results for the merge with the
                               // prefix (null without one: they go to o and lse)
    int2* meta;              // [B * Hkv * RB]: a unit's first slot (-1: undivided) and parts, for each row block
                             // (null: no join follows)
    int B, Hkv, G, Nq, capacity, causal;
    int rows_cta, RB;        // query rows a CTA holds (8, 16 or 32), row blocks of a K/V head
    int n_cta;
    int unit_cost;           // positions a unit counts besides its tiles
    int undivided;           // every unit is a run
    float scale_log2;
};
// CTAs of the cache part that fit on an SM at once (shared memory and registers).
int cache_decode_ctas_per_sm(int D, int fmt, int rows_cta);
int cache_decode_unit_cost(int rows_cta);
// after_prefix: the prefix kernel is the one ahead of it in the stream.
cudaError_t launch_cache_decode(int D, int fmt, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheDecodeParams& p, bool after_prefix, cudaStream_t stream);

// Shared prefix (fa_prefix.cu).  A unit is rows_unit (128 or 256) of the
// B * G * Nq rows of a K/V head; the part of unit u that CTA c computes lies in
// slot c + u of rows_unit rows.
struct PrefixParams {
    const void* q;
    float *o_part, *lse_part;
    int B, Hkv, G, Nq, Np;
    int rows_unit, n_rowtiles, n_tiles;
    int n_cta;               // 0: no prefix
    float scale_log2;
};
cudaError_t launch_prefix(int D, const CUtensorMap& tk, const CUtensorMap& tv, const PrefixParams& p,
                          cudaStream_t stream);
cudaError_t launch_cache_combine(int D, const CacheDecodeParams& p, const PrefixParams& f, cudaStream_t stream);

}  // namespace fa
