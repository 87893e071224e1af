// Host side of the token-sequence operators declared in include/vdm.h: argument checks,
// workspace layout, choice of the kernel.
#include <math.h>
#include <string.h>

#include <atomic>

#include "seq_internal.cuh"

namespace vdm {
namespace {

__device__ int g_attention_error = 0;   // site of the first wait that gave up, 0: none

// its address, asked for once per device
vdm_status attention_error_word(int** p) {
    static std::atomic<int*> known[64];
    int dev = 0;
    VDM_CUDA_TRY(cudaGetDevice(&dev));
    *p = dev < 64 ? known[dev].load() : nullptr;
    if (*p) return VDM_OK;
    VDM_CUDA_TRY(cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_attention_error));
    if (dev < 64) known[dev].store(*p);
    return VDM_OK;
}

// tokens, positions and query rows: a tile beyond the last still counts in 32 bits
constexpr int64_t kMost = 0x7fff0000ll;

size_t dtype_size(vdm_dtype d) { return d == VDM_F32 ? 4 : 2; }
bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

vdm_status check_dims(const char* what, vdm_dtype dt, int D) {
    if (dt != VDM_F32 && dt != VDM_BF16) return fail(VDM_ERR_INVALID_ARG, "%s: unknown dtype %d", what, (int)dt);
    if (D != 64 && D != 128) return fail(VDM_ERR_UNSUPPORTED, "%s: D = %d not in {64, 128}", what, D);
    return VDM_OK;
}

vdm_status check_heads(const char* what, const vdm_heads* h, int64_t T, int H, int D, vdm_dtype dt, HeadView* out) {
    if (!h || !h->data) return fail(VDM_ERR_INVALID_ARG, "%s is NULL", what);
    const int64_t el = (int64_t)dtype_size(dt);
    int64_t st = T > 1 ? h->stride_token : (int64_t)D * H, sh = H > 1 ? h->stride_head : D;
    if (!al16(h->data) || (st * el) % 16 || (sh * el) % 16)
        return fail(VDM_ERR_INVALID_ARG, "%s: rows must start on 16-byte boundaries (strides %lld, %lld elements)",
                    what, (long long)st, (long long)sh);
    // no two rows share an element: one of the strides steps over whole blocks of the other
    const bool ok = st >= D && sh >= D && (H <= 1 || T <= 1 || st >= (H - 1) * sh + D || sh >= (T - 1) * st + D);
    if (!ok) return fail(VDM_ERR_INVALID_ARG, "%s: rows overlap (strides %lld, %lld elements, %lld x %d rows of %d)",
                         what, (long long)st, (long long)sh, (long long)T, H, D);
    if (st * el >= (int64_t)1 << 40 || sh * el >= (int64_t)1 << 40)
        return fail(VDM_ERR_UNSUPPORTED, "%s: stride beyond 2^40 bytes", what);
    out->p = static_cast<char*>(h->data);
    out->st = st * el;
    out->sh = sh * el;
    return VDM_OK;
}

vdm_status check_count(const char* what, int64_t T, int B) {
    if (T < 0 || B < 0) return fail(VDM_ERR_INVALID_ARG, "%s: negative size (%lld tokens, %d sequences)", what, (long long)T, B);
    if (T > kMost) return fail(VDM_ERR_UNSUPPORTED, "%s: %lld tokens do not fit in 32-bit offsets", what, (long long)T);
    return VDM_OK;
}

vdm_status check_cache(const vdm_kv_cache* c, const int32_t* table, int max_pages, CacheView* v) {
    if (!c) return fail(VDM_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype != VDM_CACHE_F32 && c->dtype != VDM_CACHE_BF16 && c->dtype != VDM_CACHE_E4M3)
        return fail(VDM_ERR_INVALID_ARG, "cache: unknown dtype %d", (int)c->dtype);
    if (c->D != 64 && c->D != 128) return fail(VDM_ERR_UNSUPPORTED, "cache: D = %d not in {64, 128}", c->D);
    if (c->H < 1 || c->H > 65535 || c->num_pages < 0 || max_pages < 0)
        return fail(VDM_ERR_INVALID_ARG, "cache: %d heads, %d pages, %d pages per sequence", c->H, c->num_pages, max_pages);
    int shift = 0;
    while ((16 << shift) < c->page_size && shift < 4) ++shift;
    if ((16 << shift) != c->page_size)
        return fail(VDM_ERR_UNSUPPORTED, "cache: page_size = %d not in {16, 32, 64, 128, 256}", c->page_size);
    if ((int64_t)max_pages * c->page_size > kMost)
        return fail(VDM_ERR_UNSUPPORTED, "cache: %d pages of %d tokens do not fit in 32-bit positions", max_pages, c->page_size);
    if (c->num_pages > 0) {
        if (!c->k || !c->v || !al16(c->k) || !al16(c->v))
            return fail(VDM_ERR_INVALID_ARG, "cache: k and v must be 16-byte aligned device memory");
        if (c->dtype == VDM_CACHE_E4M3 && (!c->k_scale || !c->v_scale || !al16(c->k_scale) || !al16(c->v_scale)))
            return fail(VDM_ERR_INVALID_ARG, "cache: an E4M3 cache needs k_scale and v_scale, 16-byte aligned");
    }
    if (max_pages > 0 && !table) return fail(VDM_ERR_INVALID_ARG, "page table is NULL");
    v->k = static_cast<char*>(c->k);
    v->v = static_cast<char*>(c->v);
    v->ks = c->dtype == VDM_CACHE_E4M3 ? c->k_scale : nullptr;
    v->vs = c->dtype == VDM_CACHE_E4M3 ? c->v_scale : nullptr;
    v->num_pages = c->num_pages;
    v->page_size = c->page_size;
    v->page_shift = shift + 4;
    v->H = c->H;
    v->D = c->D;
    v->dtype = c->dtype;
    v->table = table;
    v->max_pages = max_pages;
    return VDM_OK;
}

vdm_status check_cache_dtype(const vdm_kv_cache* c, vdm_dtype dt) {
    if (dt != VDM_F32 && dt != VDM_BF16) return fail(VDM_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (c->dtype != VDM_CACHE_E4M3 && (c->dtype == VDM_CACHE_F32) != (dt == VDM_F32))
        return fail(VDM_ERR_UNSUPPORTED, "the cache's dtype must be E4M3 or that of the call's tensors");
    return VDM_OK;
}

vdm_status check_attention(const vdm_attention* a) {
    if (!a) return fail(VDM_ERR_INVALID_ARG, "attention parameters are NULL");
    VDM_TRY(check_dims("attention", a->dtype, a->D));
    if (a->Hq < 1 || a->Hk < 1 || a->Hq % a->Hk || a->Hk > 65535 || a->Hq > 65535)
        return fail(VDM_ERR_INVALID_ARG, "attention: %d query heads in %d groups", a->Hq, a->Hk);
    if (a->causal != 0 && a->causal != 1) return fail(VDM_ERR_INVALID_ARG, "attention: causal must be 0 or 1");
    if (!(a->scale > 0.f) || isinf(a->scale)) return fail(VDM_ERR_INVALID_ARG, "attention: scale must be positive and finite");
    return VDM_OK;
}

// Kernel and number of blocks that share a row tile's keys.  Depends on sizes alone, so that
// the workspace can be asked for beforehand.
enum Kernel : int { kSimt, kTc, kRows, kRowsF32 };
struct Plan {
    int kernel, splits, cluster;
};

Plan plan_attention(const vdm_attention* at, int B, int64_t Tq, int64_t max_kv) {
    Plan p;
    p.splits = p.cluster = 1;
    const bool bf16 = at->dtype != VDM_F32;
    p.kernel = bf16 ? kTc : kSimt;
    const int64_t G = at->Hq / at->Hk, seqs = B < Tq ? B : Tq;
    if (seqs == 0) return p;
    // Keys of a sequence and share of them that a query sees: as many keys as queries in all are taken for
    // packed self-attention with sequences of up to twice the average.
    const bool self = max_kv == Tq && Tq > seqs;
    const double kv = self ? (double)max_kv * 2.0 / seqs < (double)max_kv ? (double)max_kv * 2.0 / seqs : (double)max_kv : (double)max_kv;
    const double share = self && at->causal ? 0.5 : 1.0;

    // Large-tile kernels: row tiles, blocks that run at once, and the cost of a block in steps of N keys: its
    // own share of the keys, and its start and end.  With many blocks the longest half overlaps the others.
    // Joining s parts takes a launch, and s rows of floats written and read at 5 TB/s.  The number of splits is
    // the one with the shortest sum.  Measured, us: a step 1.85 and a start and end 7.4 (tensor cores, D = 128),
    // 1.5 and 6 (D = 64); 7 and 7 (CUDA cores).
    const int64_t M = bf16 ? tc_rows(at->D) : 64, N = bf16 ? 128 : simt_keys(at->D), at_once = bf16 ? 148 * tc_per_sm(at->D) : 296;
    const double step = !bf16 ? 7.0 : at->D == 64 ? 1.5 : 1.85, ends = bf16 ? 4.0 * step : step;
    const int64_t tiles = (Tq * G + seqs * (M - 1)) / M * at->Hk;
    const double nk = ceil(kv / N);
    double best = 0;
    for (int s = 1; s <= 64 && s * 2 <= (nk > 2 ? nk : 2); ++s) {
        const double part = ceil(nk / s) * step, mine = part + ends, all = (double)tiles * s * (part * share + ends) / at_once;
        const double cost = (tiles * s <= at_once ? mine : all + 0.5 * mine > mine ? all + 0.5 * mine : mine) +
                            (s > 1 ? 3.5 + s * (double)(Tq * at->Hq * at->D * 8) / 5e6 : 0.0);
        if (s == 1 || cost < 0.95 * best) {
            best = cost;
            p.splits = s;
        }
    }
    // The few-row kernels: tiles of R rows, keys shared by the four warps of each of up to eight blocks.
    // Measured, us: a block's start and end 4; a warp's step of 32 keys with 12 warps on an SM 6 (16 rows, D =
    // 128) and 3.6 (D = 64), with 8 rows 0.6 of that; float32 10 and 5.6 (4 rows).
    const int64_t R = bf16 ? rows_tile((int)G, Tq, B) : rows_tile_f32((int)G, Tq, B);
    const int64_t few = seqs * (((Tq * G + seqs - 1) / seqs + R - 1) / R) * at->Hk, steps = (int64_t)(kv + 31) / 32;
    const double few_step = (at->D == 64 ? (bf16 ? 3.6 : 5.6) : bf16 ? 6.0 : 10.0) * (R == 8 ? 0.6 : R < 4 ? 0.25 * R : 1.0);
    if (4.0 + (double)few * steps * share * few_step / (148 * 12) < best) {
        p.kernel = bf16 ? kRows : kRowsF32;
        p.splits = 1;
        // Blocks of a tile: one where its warps have three steps (float32: half a step) or fewer, for a cluster's
        // joining takes 2 us; else until
        // the SMs are full and a warp has half a step, or, for the sake of ragged lengths, until there are some
        // 1500 with at least 16 steps a warp.
        const int64_t full = bf16 || at->D == 64 ? 512 : 296;
        while (steps > (bf16 ? 12 : 2) && p.cluster < 8 && ((few * p.cluster * 2 <= full && p.cluster * 4 <= steps) || (few * p.cluster < 1500 && p.cluster * 128 <= steps)))
            p.cluster *= 2;
        if (p.cluster == 8)
            while (p.splits < 16 && few * 8 * p.splits < 296 && p.splits * 192 <= steps) p.splits *= 2;
    }
    return p;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

vdm_status run_attention(const vdm_attention* at, AttnArgs& a, int64_t max_kv, const vdm_heads* out, float* lse, void* ws,
                         size_t ws_bytes, vdm_stream stream) {
    VDM_TRY(check_heads("out", out, a.Tq, at->Hq, at->D, at->dtype, &a.out));
    a.Hq = at->Hq;
    a.Hk = at->Hk;
    a.G = at->Hq / at->Hk;
    a.D = at->D;
    a.causal = at->causal;
    a.scale_log2 = at->scale * 1.44269504088896340736f;
    a.lse = lse;
    if ((int64_t)a.Tq * a.G > kMost)
        return fail(VDM_ERR_UNSUPPORTED, "attention: %lld query tokens of %d heads per group", (long long)a.Tq, a.G);
    size_t need = 0;
    VDM_TRY(vdm_attention_workspace_size(at, a.B, a.Tq, max_kv, &need));
    if (need && (!ws || ws_bytes < need))
        return fail(VDM_ERR_WORKSPACE, "attention: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    if (need && ((uintptr_t)ws & 255)) return fail(VDM_ERR_INVALID_ARG, "attention: workspace must be 256-byte aligned");
    const Plan plan = plan_attention(at, a.B, a.Tq, max_kv);
    a.splits = plan.splits;
    a.cluster = plan.cluster;
    a.part_o = static_cast<float*>(ws);
    a.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + up256((size_t)a.splits * a.Tq * at->Hq * at->D * 4));
    VDM_TRY(attention_error_word(&a.err));
    a.timeout = g_debug.timeout > 0 ? g_debug.timeout : 4000000000ll;   // cycles of one bounded wait, about two seconds
    if (plan.kernel == kTc) {   // test hook: the g_debug.inject-th launch from the hook's call withholds one signal
        a.withhold = g_debug.inject == 1;
        if (g_debug.inject > 0) --g_debug.inject;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (plan.kernel == kRows) return launch_attention_rows(a, st);
    if (plan.kernel == kRowsF32) return launch_attention_rows_f32(a, st);
    return plan.kernel == kTc ? launch_attention_tc(a, st) : launch_attention_simt(a, at->dtype, st);
}

}  // namespace

}  // namespace vdm

using namespace vdm;

extern "C" {

vdm_status vdm_qk_norm_rope(vdm_dtype dtype, int64_t T, int32_t Hq, int32_t Hk, int32_t D, const vdm_heads* q,
                            const vdm_heads* k, const float* d_q_gain, const float* d_k_gain, float eps,
                            const vdm_rope* rope, const int32_t* d_positions, const vdm_heads* q_out,
                            const vdm_heads* k_out, vdm_stream stream) {
    VDM_TRY(check_dims("qk_norm_rope", dtype, D));
    VDM_TRY(check_count("qk_norm_rope", T, 0));
    if (Hq < 0 || Hk < 0 || Hq + (int64_t)Hk < 1) return fail(VDM_ERR_INVALID_ARG, "qk_norm_rope: %d query and %d key heads", Hq, Hk);
    if (!(eps >= 0.f) || isinf(eps)) return fail(VDM_ERR_INVALID_ARG, "qk_norm_rope: eps must be finite and >= 0");
    RopeArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T, a.Hq = Hq, a.Hk = Hk, a.D = D, a.eps = eps;
    a.gq = d_q_gain, a.gk = d_k_gain;
    if (rope) {
        if (rope->rot_dim < 2 || rope->rot_dim > D || rope->rot_dim % 2)
            return fail(VDM_ERR_UNSUPPORTED, "rope: rot_dim = %d must be even and in [2, %d]", rope->rot_dim, D);
        if (rope->interleaved != 0 && rope->interleaved != 1) return fail(VDM_ERR_INVALID_ARG, "rope: interleaved must be 0 or 1");
        if (isnan(rope->mscale) || isinf(rope->mscale)) return fail(VDM_ERR_INVALID_ARG, "rope: mscale must be finite");
        if (!rope->inv_freq) return fail(VDM_ERR_INVALID_ARG, "rope: inv_freq is NULL");
        if (T > 0 && !d_positions) return fail(VDM_ERR_INVALID_ARG, "rope: positions are NULL");
        a.rot = rope->rot_dim, a.interleaved = rope->interleaved, a.inv_freq = rope->inv_freq, a.mscale = rope->mscale;
        a.pos = d_positions;
    }
    if (T == 0) return VDM_OK;
    if (Hq > 0) {
        VDM_TRY(check_heads("q", q, T, Hq, D, dtype, &a.q));
        VDM_TRY(check_heads("q_out", q_out, T, Hq, D, dtype, &a.qo));
    }
    if (Hk > 0) {
        VDM_TRY(check_heads("k", k, T, Hk, D, dtype, &a.k));
        VDM_TRY(check_heads("k_out", k_out, T, Hk, D, dtype, &a.ko));
    }
    return launch_qk_norm_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

vdm_status vdm_cache_write(const vdm_kv_cache* cache, vdm_dtype dtype, const vdm_heads* k, const vdm_heads* v, int64_t T,
                           const int32_t* d_cu, const int32_t* d_kv_len, const int32_t* d_table, int32_t max_pages,
                           int32_t B, vdm_stream stream) {
    CacheIo a;
    memset(&a, 0, sizeof(a));
    VDM_TRY(check_count("cache_write", T, B));
    VDM_TRY(check_cache(cache, B > 0 ? d_table : reinterpret_cast<const int32_t*>(16), max_pages, &a.c));
    VDM_TRY(check_cache_dtype(cache, dtype));
    if (T == 0 || B == 0 || cache->num_pages == 0 || max_pages == 0) return VDM_OK;
    VDM_TRY(check_heads("k", k, T, cache->H, cache->D, dtype, &a.k));
    VDM_TRY(check_heads("v", v, T, cache->H, cache->D, dtype, &a.v));
    if (!d_cu || !d_kv_len) return fail(VDM_ERR_INVALID_ARG, "cache_write: cu or kv_len is NULL");
    a.cu = d_cu, a.kv_len = d_kv_len, a.B = B, a.T = T;
    return launch_cache_write(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

vdm_status vdm_cache_read(const vdm_kv_cache* cache, vdm_dtype dtype, const int32_t* d_kv_len, const int32_t* d_table,
                          int32_t max_pages, const int32_t* d_cu, int32_t B, int64_t T, const vdm_heads* k,
                          const vdm_heads* v, vdm_stream stream) {
    CacheIo a;
    memset(&a, 0, sizeof(a));
    VDM_TRY(check_count("cache_read", T, B));
    VDM_TRY(check_cache(cache, B > 0 ? d_table : reinterpret_cast<const int32_t*>(16), max_pages, &a.c));
    VDM_TRY(check_cache_dtype(cache, dtype));
    if (T == 0 || B == 0 || max_pages == 0) return VDM_OK;
    VDM_TRY(check_heads("k", k, T, cache->H, cache->D, dtype, &a.k));
    VDM_TRY(check_heads("v", v, T, cache->H, cache->D, dtype, &a.v));
    if (!d_cu || !d_kv_len) return fail(VDM_ERR_INVALID_ARG, "cache_read: cu or kv_len is NULL");
    a.cu = d_cu, a.kv_len = d_kv_len, a.B = B, a.T = T;
    return launch_cache_read(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

vdm_status vdm_attention_workspace_size(const vdm_attention* at, int32_t B, int64_t Tq, int64_t max_kv, size_t* bytes) {
    VDM_TRY(check_attention(at));
    VDM_TRY(check_count("attention", Tq, B));
    if (max_kv < 0 || !bytes) return fail(VDM_ERR_INVALID_ARG, "attention: max_kv < 0 or bytes is NULL");
    const int s = plan_attention(at, B, Tq, max_kv).splits;
    *bytes = s < 2 ? 0 : up256((size_t)s * Tq * at->Hq * at->D * 4) + up256((size_t)s * Tq * at->Hq * 4);
    return VDM_OK;
}

vdm_status vdm_attention_packed(const vdm_attention* at, const vdm_heads* q, const vdm_heads* k, const vdm_heads* v,
                                const int32_t* d_cu_q, const int32_t* d_cu_k, int32_t B, int64_t Tq, int64_t Tk,
                                const vdm_heads* out, float* d_lse, void* d_ws, size_t ws_bytes, vdm_stream stream) {
    VDM_TRY(check_attention(at));
    VDM_TRY(check_count("attention queries", Tq, B));
    VDM_TRY(check_count("attention keys", Tk, B));
    if (Tq == 0 || B == 0) return VDM_OK;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    VDM_TRY(check_heads("q", q, Tq, at->Hq, at->D, at->dtype, &a.q));
    if (Tk > 0) {
        VDM_TRY(check_heads("k", k, Tk, at->Hk, at->D, at->dtype, &a.k));
        VDM_TRY(check_heads("v", v, Tk, at->Hk, at->D, at->dtype, &a.v));
    }
    if (!d_cu_q || !d_cu_k) return fail(VDM_ERR_INVALID_ARG, "attention: cu_q or cu_k is NULL");
    a.cu_q = d_cu_q, a.cu_k = d_cu_k, a.B = B, a.Tq = Tq, a.Tk = Tk;
    return run_attention(at, a, Tk, out, d_lse, d_ws, ws_bytes, stream);
}

vdm_status vdm_attention_paged(const vdm_attention* at, const vdm_heads* q, const vdm_kv_cache* cache,
                               const int32_t* d_cu_q, const int32_t* d_kv_len, const int32_t* d_table,
                               int32_t max_pages, int32_t B, int64_t Tq, const vdm_heads* out, float* d_lse, void* d_ws,
                               size_t ws_bytes, vdm_stream stream) {
    VDM_TRY(check_attention(at));
    VDM_TRY(check_count("attention queries", Tq, B));
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    VDM_TRY(check_cache(cache, B > 0 ? d_table : reinterpret_cast<const int32_t*>(16), max_pages, &a.c));
    VDM_TRY(check_cache_dtype(cache, at->dtype));
    if (cache->H != at->Hk || cache->D != at->D)
        return fail(VDM_ERR_INVALID_ARG, "attention: the cache holds %d heads of %d, the call has %d of %d", cache->H, cache->D, at->Hk, at->D);
    if (Tq == 0 || B == 0) return VDM_OK;
    VDM_TRY(check_heads("q", q, Tq, at->Hq, at->D, at->dtype, &a.q));
    if (!d_cu_q || !d_kv_len) return fail(VDM_ERR_INVALID_ARG, "attention: cu_q or kv_len is NULL");
    a.cu_q = d_cu_q, a.cu_k = d_kv_len, a.paged = 1, a.B = B, a.Tq = Tq;
    return run_attention(at, a, (int64_t)max_pages * cache->page_size, out, d_lse, d_ws, ws_bytes, stream);
}

vdm_status vdm_attention_status(vdm_stream stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the word of the stream's device, whichever is current
    struct On {
        int was = 0, dev = 0;
        bool moved = false;
        ~On() {
            if (moved) cudaSetDevice(was);
        }
    } on;
    VDM_CUDA_TRY(cudaGetDevice(&on.was));
    VDM_CUDA_TRY(cudaStreamGetDevice(s, &on.dev));
    if (on.dev != on.was) {
        VDM_CUDA_TRY(cudaSetDevice(on.dev));
        on.moved = true;
    }
    int* word = nullptr;
    VDM_TRY(attention_error_word(&word));
    int site = 0;
    VDM_CUDA_TRY(cudaMemcpyAsync(&site, word, sizeof(int), cudaMemcpyDeviceToHost, s));
    VDM_CUDA_TRY(cudaStreamSynchronize(s));
    if (!site) return VDM_OK;
    VDM_CUDA_TRY(cudaMemsetAsync(word, 0, sizeof(int), s));
    VDM_CUDA_TRY(cudaStreamSynchronize(s));
    return fail(VDM_ERR_TIMEOUT, "attention: bounded wait expired at site %d", site);
}

}  // extern "C"
