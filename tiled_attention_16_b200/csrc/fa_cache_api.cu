// fa_cache_api.cu — the C ABI of include/fa_rope.h and include/fa_cache.h:
// argument checks, plans, tensor maps and launches.  No device memory is
// allocated here; every buffer belongs to the caller.
#include "fa_cache.h"
#include "fa_rope.h"
#include "fa_serving.cuh"

#include <algorithm>
#include <cmath>

namespace {

using namespace fa;

constexpr double kLog2e = 1.4426950408889634;
constexpr long long kIntMax = 0x7fffffffLL;

fa_status status_of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned256(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

// A view that is read: aligned rows, strides that move forward.
bool rows_ok(const fa_rows* r, int B, int H, int N) {
    if (r == nullptr || !aligned16(r->data)) return false;
    const long long st[3] = {r->stride_b, r->stride_h, r->stride_n};
    const int n[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] < 0 || (st[i] & 7) != 0 || st[i] > (1LL << 44) / n[i])) return false;
    return true;
}

// A view that is written: besides, no two rows share an element.  Sorted by
// stride, each dimension has to step over all that the smaller ones cover.
bool rows_distinct(const fa_rows* r, int B, int H, int N, int D) {
    long long st[3] = {r->stride_b, r->stride_h, r->stride_n};
    int n[3] = {B, H, N}, order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return st[a] < st[b]; });
    long long extent = D;
    for (int i : order) {
        if (n[i] == 1) continue;
        if (st[i] < extent) return false;
        extent = st[i] * (n[i] - 1) + extent;
    }
    return true;
}

RopeRows rows_of(const fa_rows* r, int B, int H, int N) {
    RopeRows x;
    x.data = static_cast<__nv_bfloat16*>(r->data);
    x.stride_b = B > 1 ? r->stride_b : 0;
    x.stride_h = H > 1 ? r->stride_h : 0;
    x.stride_n = N > 1 ? r->stride_n : 0;
    return x;
}

fa_status check_rope(const fa_rope_shape* s) {
    if (!s) return FA_ERR_INVALID_ARG;
    if (s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->N < 1 || s->D < 1) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(s->eps) || !(s->eps > 0.f)) return FA_ERR_INVALID_ARG;
    if (s->D != 64 && s->D != 128) return FA_ERR_UNSUPPORTED;
    if (s->rotary_dim < 0 || s->rotary_dim > s->D || (s->rotary_dim & 7) != 0) return FA_ERR_INVALID_ARG;
    const long long heads = static_cast<long long>(s->Hq) + s->Hkv;
    if (heads > 65535 || static_cast<long long>(s->B) * s->N > kIntMax) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Pointers that forward and backward share.
fa_status check_rope_args(const fa_rope_shape* s, const fa_rows* q, const fa_rows* k, const void* qw, const void* kw,
                          const float* inv_freq, const int* positions) {
    const fa_status st = check_rope(s);
    if (st != FA_OK) return st;
    if (!rows_ok(q, s->B, s->Hq, s->N) || !rows_ok(k, s->B, s->Hkv, s->N)) return FA_ERR_INVALID_ARG;
    if (!aligned4(qw) || !aligned4(kw)) return FA_ERR_INVALID_ARG;
    if (s->rotary_dim > 0 && !aligned4(inv_freq)) return FA_ERR_INVALID_ARG;
    if (positions != nullptr && !aligned4(positions)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

RopeParams rope_params(const fa_rope_shape& s, const fa_rows* q, const fa_rows* k, const void* qw, const void* kw,
                       const float* inv_freq, const int* positions) {
    RopeParams p{};
    p.q = rows_of(q, s.B, s.Hq, s.N);
    p.k = rows_of(k, s.B, s.Hkv, s.N);
    p.q_weight = qw;
    p.k_weight = kw;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.N = s.N;
    p.rot = s.rotary_dim;
    p.weight_bf16 = s.weight_bf16 ? 1 : 0;
    p.eps = s.eps;
    p.tokens = static_cast<long long>(s.B) * s.N;
    return p;
}

fa_status check_cache(const fa_cache_shape* s) {
    if (!s) return FA_ERR_INVALID_ARG;
    if (s->B < 1 || s->Hkv < 1 || s->capacity < 1 || s->D < 1) return FA_ERR_INVALID_ARG;
    if (s->format < FA_CACHE_BF16 || s->format > FA_CACHE_INT8) return FA_ERR_INVALID_ARG;
    if (s->format != FA_CACHE_BF16 && (s->capacity & 3) != 0) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(s->B) * s->Hkv > 65535) return FA_ERR_INVALID_ARG;
    if (s->D != 64 && s->D != 128) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

bool cache_pointers_ok(int format, const void* kc, const void* vc, const float* ks, const float* vs) {
    if (!aligned16(kc) || !aligned16(vc)) return false;
    return format == FA_CACHE_BF16 || (aligned16(ks) && aligned16(vs));
}

// Query rows of a K/V head a CTA of the cache part holds, of R.
// 8 sequences of 32K slots of 8 heads of 128, with 32 rows a CTA and with twice
// 16: 24 int8 rows 142 and 170 us, 32 rows e4m3 153 and 150, bf16 168 and 188 (171
// now that V rows hidden from some queries are looked at).
int rows_of_cta(long long R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }
// Rows of a unit of the prefix part, of head_rows: two row tiles share the key
// tiles where there are two.
int rows_of_prefix_unit(long long head_rows) { return head_rows > kTileM ? 2 * kTileM : kTileM; }

fa_status check_decode(const fa_cache_decode_shape* s) {
    if (!s) return FA_ERR_INVALID_ARG;
    const fa_cache_shape c{s->B, s->Hkv, s->capacity, s->D, s->format};
    const fa_status st = check_cache(&c);
    if (st != FA_OK && st != FA_ERR_UNSUPPORTED) return st;
    if (s->Hq < 1 || s->Nq < 1 || s->n_prefix < 0 || s->Hq % s->Hkv != 0) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(s->scale) || !(s->scale > 0.f)) return FA_ERR_INVALID_ARG;
    const long long heads = static_cast<long long>(s->B) * s->Hq;
    if (heads > FA_CACHE_MAX_ROWS || heads * s->Nq > FA_CACHE_MAX_ROWS) return FA_ERR_INVALID_ARG;
    // What the kernels number with 32 bits: slots and keys (rounded up to tiles),
    // the positions that all units cover, the prefix's key tiles of all its units.
    if (s->capacity > kIntMax - 63 || s->n_prefix > kIntMax - 255) return FA_ERR_INVALID_ARG;
    const long long R = static_cast<long long>(s->Hq / s->Hkv) * s->Nq, head_rows = s->B * R;
    const long long units = static_cast<long long>(s->B) * s->Hkv;
    if (units * ((s->capacity + 63LL) / 64 + cache_decode_unit_cost(rows_of_cta(R))) > kIntMax) return FA_ERR_INVALID_ARG;
    const int unit = rows_of_prefix_unit(head_rows);
    if (s->Hkv * ((head_rows + unit - 1) / unit) * ((s->n_prefix + kTileN - 1LL) / kTileN) > kIntMax) return FA_ERR_INVALID_ARG;
    return st;
}

// Capacity up to which a (sequence, K/V head) is one CTA's: no join is needed
// then, which saves a launch.  Measured with 32 query over 8 K/V heads and 1, 8,
// 64 sequences, device time in us undivided and divided:
//               256 slots                      512 slots                      1024 slots
//   e4m3 128    5.6  5.8 14.0,  8.2 9.2 15.1   7.7 8.0 22.3,  8.4 10.0 20.6   11.5 11.9 35.2,  9.0 10.8 31.4
//   e4m3  64    5.4  5.5  7.3,  7.7 8.5 12.9   7.0 7.2 10.8,  8.2  9.0 16.4   10.2 10.4 18.3,  8.5  9.8 21.7
//   bf16 128    5.8  5.9 17.8,  7.9 9.0 19.3   7.7 8.0 28.5,  8.3 10.0 29.2   11.7 14.6 48.9,  8.9 12.1 48.4
//   bf16  64    5.1  5.4  8.1,  7.6 8.2 13.6   6.6 6.8 15.3,  8.0  9.0 19.1    9.7  9.8 25.3,  8.3  9.6 29.8
constexpr int kUndividedSlots = FA_CACHE_UNDIVIDED;

// How a decode call is split.  The cache part runs on as many CTAs as fit on
// the SMs at once; shapes do not change that, the kernel deals its tiles out
// by the lengths it finds.
struct DecodeCachePlan {
    int rows_cta, RB, n_cta;
    bool undivided;
    int rows_unit, n_rowtiles, n_tiles, n_pcta;
    size_t o_part, lse_part, o_unit, lse_unit, meta, po_part, plse_part, total;
};

DecodeCachePlan decode_cache_plan(const fa_cache_decode_shape& s, int sms) {
    DecodeCachePlan pl{};
    const int R = s.Hq / s.Hkv * s.Nq;
    pl.rows_cta = rows_of_cta(R);
    pl.RB = (R + pl.rows_cta - 1) / pl.rows_cta;
    // runs of tiles, and RB CTAs to each
    const long long units = static_cast<long long>(s.B) * s.Hkv;
    const long long most = units * ((s.capacity + 63LL) / 64);
    const long long resident = static_cast<long long>(sms) * cache_decode_ctas_per_sm(s.D, s.format, pl.rows_cta);
    pl.undivided = s.capacity <= kUndividedSlots;
    pl.n_cta = static_cast<int>(pl.undivided ? units : std::max(1LL, std::min(most, resident / pl.RB))) * pl.RB;
    const long long rows = static_cast<long long>(s.B) * s.Hq * s.Nq;
    if (s.n_prefix > 0) {
        const long long head_rows = static_cast<long long>(s.B) * R;
        pl.rows_unit = rows_of_prefix_unit(head_rows);
        const bool two = pl.rows_unit == 2 * kTileM;
        pl.n_rowtiles = static_cast<int>((head_rows + pl.rows_unit - 1) / pl.rows_unit);
        pl.n_tiles = (s.n_prefix + kTileN - 1) / kTileN;
        const long long units = static_cast<long long>(s.Hkv) * pl.n_rowtiles, tiles = units * pl.n_tiles;
        // alternating blocks want two key tiles a CTA
        const long long most = std::min<long long>(two ? tiles : (tiles + 1) / 2, sms);
        pl.n_pcta = static_cast<int>(most);
        // A part costs about three key tiles besides its own (its Q, an empty
        // pipeline, its results).  With a multiple of the units as CTAs each has
        // one part; that is taken where it beats all SMs with two parts on most.
        const long long even = most / units * units;
        if (even > 0 && even < most && (tiles + even - 1) / even + 3 <= (tiles + most - 1) / most + 6)
            pl.n_pcta = static_cast<int>(even);
    }
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    if (!pl.undivided) {
        const size_t slots = 2 * static_cast<size_t>(pl.n_cta) * pl.rows_cta;
        pl.o_part = take(slots * s.D * 4);
        pl.lse_part = take(slots * 4);
    }
    // (undivided units without a prefix need no join, and so no workspace)
    if (!pl.undivided || s.n_prefix > 0) pl.meta = take(static_cast<size_t>(units) * pl.RB * 8);
    if (s.n_prefix > 0) {
        pl.o_unit = take(static_cast<size_t>(rows) * s.D * 4);
        pl.lse_unit = take(static_cast<size_t>(rows) * 4);
        const size_t pslots = (static_cast<size_t>(pl.n_pcta) + static_cast<size_t>(s.Hkv) * pl.n_rowtiles) * pl.rows_unit;
        pl.po_part = take(pslots * s.D * 4);
        pl.plse_part = take(pslots * 4);
    }
    pl.total = at;
    return pl;
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const fa_rope_shape* shape, const fa_rows* q, const fa_rows* k, const void* q_weight,
                          const void* k_weight, const float* inv_freq, const int* positions, void* q_out, void* k_out,
                          void* stream) {
    fa_status st = check_rope_args(shape, q, k, q_weight, k_weight, inv_freq, positions);
    if (st != FA_OK) return st;
    if (!aligned16(q_out) || !aligned16(k_out)) return FA_ERR_INVALID_ARG;
    if ((st = static_cast<fa_status>(device_status_code())) != FA_OK) return st;
    const int sms = sm_count();
    if (sms <= 0) return FA_ERR_CUDA;
    RopeParams p = rope_params(*shape, q, k, q_weight, k_weight, inv_freq, positions);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    return status_of(launch_qk_norm_rope(shape->D, shape->interleaved, p, sms, static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(const fa_rope_shape* shape) {
    if (check_rope(shape) != FA_OK) return 0;
    const int sms = sm_count();
    return sms <= 0 ? 0 : up256(static_cast<size_t>(rope_bwd_ctas(sms)) * 2 * shape->D * 4);
}

fa_status fa_qk_norm_rope_bwd(const fa_rope_shape* shape, const void* dq_out, const void* dk_out, const fa_rows* q,
                              const fa_rows* k, const void* q_weight, const void* k_weight, const float* inv_freq,
                              const int* positions, const fa_rows* dq, const fa_rows* dk, float* dq_weight,
                              float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    fa_status st = check_rope_args(shape, q, k, q_weight, k_weight, inv_freq, positions);
    if (st != FA_OK) return st;
    const fa_rope_shape& s = *shape;
    if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned4(dq_weight) || !aligned4(dk_weight))
        return FA_ERR_INVALID_ARG;
    if (!rows_ok(dq, s.B, s.Hq, s.N) || !rows_ok(dk, s.B, s.Hkv, s.N) || !rows_distinct(dq, s.B, s.Hq, s.N, s.D) ||
        !rows_distinct(dk, s.B, s.Hkv, s.N, s.D))
        return FA_ERR_INVALID_ARG;
    if (!aligned256(workspace)) return FA_ERR_INVALID_ARG;
    if ((st = static_cast<fa_status>(device_status_code())) != FA_OK) return st;
    const int sms = sm_count();
    if (sms <= 0) return FA_ERR_CUDA;
    if (workspace_bytes < fa_qk_norm_rope_bwd_workspace_bytes(shape)) return FA_ERR_INVALID_ARG;
    RopeParams p = rope_params(s, q, k, q_weight, k_weight, inv_freq, positions);
    p.dq = rows_of(dq, s.B, s.Hq, s.N);
    p.dk = rows_of(dk, s.B, s.Hkv, s.N);
    p.dq_out = static_cast<const __nv_bfloat16*>(dq_out);
    p.dk_out = static_cast<const __nv_bfloat16*>(dk_out);
    p.dw_part = static_cast<float*>(workspace);
    return status_of(launch_qk_norm_rope_bwd(s.D, s.interleaved, p, dq_weight, dk_weight, sms,
                                             static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_write(const fa_cache_shape* shape, int N, const fa_rows* k, const fa_rows* v, const int* start,
                         const int* count, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         void* stream) {
    fa_status st = check_cache(shape);
    if (st != FA_OK) return st;
    const fa_cache_shape& s = *shape;
    if (N < 1 || static_cast<long long>(s.B) * s.Hkv * N > kIntMax) return FA_ERR_INVALID_ARG;
    if (!rows_ok(k, s.B, s.Hkv, N) || !rows_ok(v, s.B, s.Hkv, N)) return FA_ERR_INVALID_ARG;
    if (!aligned4(start) || (count != nullptr && !aligned4(count))) return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(s.format, k_cache, v_cache, k_scale, v_scale)) return FA_ERR_INVALID_ARG;
    if ((st = static_cast<fa_status>(device_status_code())) != FA_OK) return st;
    CacheWriteParams p{};
    p.k = rows_of(k, s.B, s.Hkv, N);
    p.v = rows_of(v, s.B, s.Hkv, N);
    p.start = start;
    p.count = count;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.B = s.B;
    p.H = s.Hkv;
    p.N = N;
    p.capacity = s.capacity;
    return status_of(launch_cache_write(s.D, s.format, p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_read(const fa_cache_shape* shape, int N, const int* lens, const void* k_cache, const void* v_cache,
                        const float* k_scale, const float* v_scale, void* k_out, void* v_out, void* stream) {
    fa_status st = check_cache(shape);
    if (st != FA_OK) return st;
    const fa_cache_shape& s = *shape;
    if (N < 1 || N > s.capacity || static_cast<long long>(s.B) * s.Hkv * N > kIntMax) return FA_ERR_INVALID_ARG;
    if (lens != nullptr && !aligned4(lens)) return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(s.format, k_cache, v_cache, k_scale, v_scale)) return FA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return FA_ERR_INVALID_ARG;
    if ((st = static_cast<fa_status>(device_status_code())) != FA_OK) return st;
    CacheReadParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.lens = lens;
    p.k_out = k_out;
    p.v_out = v_out;
    p.BH = s.B * s.Hkv;
    p.H = s.Hkv;
    p.N = N;
    p.capacity = s.capacity;
    return status_of(launch_cache_read(s.D, s.format, p, static_cast<cudaStream_t>(stream)));
}

size_t fa_decode_cache_workspace_bytes(const fa_cache_decode_shape* shape) {
    if (check_decode(shape) != FA_OK) return 0;
    const int sms = sm_count();
    return sms <= 0 ? 0 : decode_cache_plan(*shape, sms).total;
}

fa_status fa_decode_cache(const fa_cache_decode_shape* shape, const void* q, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, const int* lens, const void* k_prefix,
                          const void* v_prefix, void* o, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
    fa_status st = check_decode(shape);
    if (st != FA_OK) return st;
    const fa_cache_decode_shape& s = *shape;
    if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(lens)) return FA_ERR_INVALID_ARG;
    if (!cache_pointers_ok(s.format, k_cache, v_cache, k_scale, v_scale)) return FA_ERR_INVALID_ARG;
    if (s.n_prefix > 0 && (!aligned16(k_prefix) || !aligned16(v_prefix))) return FA_ERR_INVALID_ARG;
    const bool no_workspace = s.capacity <= kUndividedSlots && s.n_prefix == 0;
    if (!no_workspace && !aligned256(workspace)) return FA_ERR_INVALID_ARG;
    if ((st = static_cast<fa_status>(device_status_code())) != FA_OK) return st;
    const int sms = sm_count();
    if (sms <= 0) return FA_ERR_CUDA;
    const DecodeCachePlan pl = decode_cache_plan(s, sms);
    if (workspace_bytes < pl.total) return FA_ERR_INVALID_ARG;
    const int eb = s.format == FA_CACHE_BF16 ? 2 : 1;
    CUtensorMap tk, tv;
    if (!make_map(&tk, k_cache, s.B * s.Hkv, s.capacity, s.D, eb, 64) ||
        !make_map(&tv, v_cache, s.B * s.Hkv, s.capacity, s.D, eb, 64))
        return FA_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    auto f32 = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    CacheDecodeParams p{};
    p.q = q;
    p.o = o;
    p.lse = lse;
    p.lens = lens;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.v_cache = v_cache;
    p.o_part = f32(pl.o_part);
    p.lse_part = f32(pl.lse_part);
    p.o_unit = s.n_prefix > 0 ? f32(pl.o_unit) : nullptr;
    p.lse_unit = s.n_prefix > 0 ? f32(pl.lse_unit) : nullptr;
    p.meta = no_workspace ? nullptr : reinterpret_cast<int2*>(ws + pl.meta);
    p.B = s.B;
    p.Hkv = s.Hkv;
    p.G = s.Hq / s.Hkv;
    p.Nq = s.Nq;
    p.capacity = s.capacity;
    p.causal = s.causal ? 1 : 0;
    p.rows_cta = pl.rows_cta;
    p.RB = pl.RB;
    p.n_cta = pl.n_cta;
    p.unit_cost = cache_decode_unit_cost(pl.rows_cta);
    p.undivided = pl.undivided ? 1 : 0;
    p.scale_log2 = static_cast<float>(static_cast<double>(s.scale) * kLog2e);
    PrefixParams f{};
    f.n_cta = pl.n_pcta;
    cudaStream_t strm = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (s.n_prefix > 0) {
        CUtensorMap pk, pv;
        if (!make_map(&pk, k_prefix, s.Hkv, s.n_prefix, s.D) || !make_map(&pv, v_prefix, s.Hkv, s.n_prefix, s.D))
            return FA_ERR_CUDA;
        f.q = q;
        f.o_part = f32(pl.po_part);
        f.lse_part = f32(pl.plse_part);
        f.B = s.B;
        f.Hkv = s.Hkv;
        f.G = p.G;
        f.Nq = s.Nq;
        f.Np = s.n_prefix;
        f.rows_unit = pl.rows_unit;
        f.n_rowtiles = pl.n_rowtiles;
        f.n_tiles = pl.n_tiles;
        f.scale_log2 = p.scale_log2;
        e = launch_prefix(s.D, pk, pv, f, strm);
    }
    if (e == cudaSuccess) e = launch_cache_decode(s.D, s.format, tk, tv, p, s.n_prefix > 0, strm);
    // undivided units without a prefix are complete
    if (e == cudaSuccess && (!pl.undivided || s.n_prefix > 0)) e = launch_cache_combine(s.D, p, f, strm);
    return status_of(e);
}

}  // extern "C"
