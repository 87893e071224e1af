// Internal declarations of the token-sequence operators (not part of the ABI).
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "vdm_internal.cuh"

namespace vdm {

// a [tokens][heads][D] view, strides in bytes
struct HeadView {
    char* p;
    int64_t st, sh;
};

struct CacheView {
    char *k, *v;
    uint8_t *ks, *vs;       // E4M3: one scale byte per row, else NULL
    int num_pages, page_size, page_shift, H, D;
    int dtype;              // vdm_cache_dtype
    const int32_t* table;   // [B][max_pages]
    int max_pages;
};

struct AttnArgs {
    HeadView q, out, k, v;   // k, v: packed only
    CacheView c;             // paged only
    const int32_t* cu_q;
    const int32_t* cu_k;     // packed: offsets; paged: lengths
    int paged;
    int B, Hq, Hk, G, D, causal;
    int64_t Tq, Tk;
    float scale_log2;        // softmax scale times log2 e
    float* lse;              // [Tq][Hq] or NULL
    // keys split over `splits` blocks: partial results (normalised rows and log2 of their sums)
    int splits;
    float* part_o;           // [splits][Tq][Hq][D]
    float* part_lse;         // [splits][Tq][Hq]
    int cluster;             // few rows: blocks that share a tile's keys and join in shared memory
    int* err;                // error word of bounded waits
    long long timeout;
    int withhold;            // test hook: one completion signal of the tensor-core kernel is not given
};

// One block of query rows of one sequence and key head.  Rows are (token, query head of the
// group) with the head fastest: row r is token r / G, head hk * G + r % G.
struct RowTile {
    int b;
    int64_t q0, k0;    // first query token / first key token (packed)
    int nq, nk;        // query tokens and keys of the sequence
    int row0;          // first row of the tile
};

__device__ __forceinline__ int clamp_len(int64_t lo, int64_t hi, int64_t T, int64_t* start) {
    lo = lo < 0 ? 0 : lo > T ? T : lo;
    hi = hi < lo ? lo : hi > T ? T : hi;
    *start = lo;
    return (int)(hi - lo);
}

__device__ __forceinline__ int cache_len(const CacheView& c, int32_t len) {
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    return len < 0 ? 0 : len > cap ? (int)cap : len;
}

// Row tiles of M rows that a launch provides for: see find_tile.
__host__ __device__ inline int64_t row_tiles(int64_t Tq, int G, int B, int M) { return Tq * G / M + B; }

// Tile `idx` of the sequences' row tiles of M rows (whole warps, converged); false: no such tile.
// With `last_first` a sequence's tiles come in descending order (causal: longest first).
// Sequence b's tiles take the numbers from floor(cu[b] G / M) + b on - room for ceil(n G / M) of them
// before the next sequence's - so that a tile's sequence is found by a search of the offsets.
// Large tiles of up to 32 sequences come by the sequences' keys, longest first: a launch then ends
// with its short blocks.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int64_t idx, int M, bool last_first, RowTile& t) {
    const int lane = threadIdx.x & 31;
    if (M > 16 && a.B > 1 && a.B <= 32) {
        int64_t q0 = 0, k0 = 0;
        int n = 0, nk = -1;
        if (lane < a.B) {
            n = clamp_len(a.cu_q[lane], a.cu_q[lane + 1], a.Tq, &q0);
            if (a.paged) nk = cache_len(a.c, a.cu_k[lane]);
            else nk = clamp_len(a.cu_k[lane], a.cu_k[lane + 1], a.Tk, &k0);
        }
        const int64_t tiles = ((int64_t)n * a.G + M - 1) / M;
        int64_t before = 0;   // tiles of the sequences that come earlier
        for (int j = 0; j < a.B; ++j) {
            const int nj = __shfl_sync(0xffffffffu, nk, j);
            const int64_t tj = __shfl_sync(0xffffffffu, tiles, j);
            if (nj > nk || (nj == nk && j < lane)) before += tj;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before <= idx && idx < before + tiles);
        if (!hit) return false;
        const int src = __ffs(hit) - 1;
        const int64_t cnt = __shfl_sync(0xffffffffu, tiles, src), local = idx - __shfl_sync(0xffffffffu, before, src);
        t.b = src;
        t.nq = __shfl_sync(0xffffffffu, n, src);
        t.nk = __shfl_sync(0xffffffffu, nk, src);
        t.q0 = __shfl_sync(0xffffffffu, q0, src);
        t.k0 = __shfl_sync(0xffffffffu, k0, src);
        t.row0 = (int)((last_first ? cnt - 1 - local : local) * M);
        return true;
    }
    auto number = [&](int b) {
        const int64_t c = a.cu_q[b];
        return (c < 0 ? 0 : c > a.Tq ? a.Tq : c) * a.G / M + b;
    };
    int lo = 0, hi = a.B;   // in [lo, hi), 32 probes at a time
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, b = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, b < hi && number(b) <= idx);
        if (!m) return false;
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
    }
    // asked for together: these are a block's first loads, and everything waits for them
    const int32_t q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1], k0 = a.cu_k[lo], k1 = a.paged ? 0 : a.cu_k[lo + 1];
    const int64_t local = idx - ((q0 < 0 ? 0 : q0 > a.Tq ? a.Tq : q0) * (int64_t)a.G / M + lo);
    t.b = lo;
    t.nq = clamp_len(q0, q1, a.Tq, &t.q0);
    const int64_t cnt = ((int64_t)t.nq * a.G + M - 1) / M;
    if (local < 0 || local >= cnt) return false;
    t.row0 = (int)((last_first ? cnt - 1 - local : local) * M);
    t.k0 = 0;
    if (a.paged) t.nk = cache_len(a.c, k0);
    else t.nk = clamp_len(k0, k1, a.Tk, &t.k0);
    return true;
}

// Grid of the large-tile kernels, and key head, tile number and split of a block of it.  Packed: the heads of
// a tile beside one another, so that blocks start in the order of their lengths, whatever their head (six sets of
// up to 4096 tokens, 8 heads of 64: 111 us, head after head 120; five prompts of up to 4096 tokens, 32/8 heads
// of 128: 356 and 368).  Paged: a head's tiles beside one another, since contexts are long and a head's tiles
// then meet its keys in the cache (512 new tokens after 15000, 32/8 heads of 128: 217 us, the other way 228).
// The head is a coordinate of the grid: computed from one it cost 4 %.
constexpr int64_t kTilesY = 65535;
inline dim3 tile_grid(const AttnArgs& a, int64_t tiles) {
    if (a.paged) return dim3((unsigned)tiles, a.Hk, a.splits);
    return dim3(a.Hk, (unsigned)(tiles < kTilesY ? tiles : kTilesY), (unsigned)((tiles + kTilesY - 1) / kTilesY * a.splits));
}
struct BlockPlace {
    int hk, split;
    int64_t tile;
};
template <bool PAGED>
__device__ __forceinline__ BlockPlace place_of(const AttnArgs& a) {
    if (PAGED) return {(int)blockIdx.y, (int)blockIdx.z, blockIdx.x};
    if (gridDim.z == a.splits) return {(int)blockIdx.x, (int)blockIdx.z, blockIdx.y};
    return {(int)blockIdx.x, (int)(blockIdx.z % a.splits), blockIdx.y + kTilesY * (blockIdx.z / a.splits)};
}

// keys that query token i of the tile's sequence sees: [0, result)
__device__ __forceinline__ int keys_seen(const AttnArgs& a, const RowTile& t, int i) {
    if (!a.causal) return t.nk;
    const int64_t lim = (int64_t)t.nk - t.nq + i + 1;
    return lim < 0 ? 0 : (int)lim;
}

// row of position j of sequence b, head h in the cache, or -1 where there is no page
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int b, int h, int j) {
    const int32_t page = c.table[(int64_t)b * c.max_pages + (j >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return (((int64_t)page * c.H + h) << c.page_shift) + (j & (c.page_size - 1));
}

__device__ __forceinline__ float scale_of(uint8_t s) {
    // 2^(s - 127); s = 0 never comes from vdm_cache_write and stands for 2^-127
    return s ? __uint_as_float((uint32_t)s << 23) : __uint_as_float(0x00400000u);
}

// the same twice, as bf16
__device__ __forceinline__ uint32_t scale_bf16x2(uint8_t s) { return (s ? (uint32_t)s << 7 : 0x40u) * 0x10001u; }

// bf16 pairs times a power of two
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// two e4m3 codes as floats (exact)
__device__ __forceinline__ float2 e4m3x2_to_f(uint16_t u) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(u, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// 4 consecutive elements as floats
__device__ __forceinline__ float4 load4f(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4f(const __nv_bfloat16* p) { return load4(p); }
__device__ __forceinline__ float4 load4f(const uint8_t* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    const float2 a = e4m3x2_to_f((uint16_t)u), b = e4m3x2_to_f((uint16_t)(u >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a);
    u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
}

// rows of one key head of the tile's sequence
template <typename TC, bool PAGED>
struct KvRows {
    const AttnArgs& a;
    const RowTile& t;
    int hk;
    // elements [d, d + 4) of key (or value) j, dequantised
    __device__ __forceinline__ float4 get(bool value, int j, int d) const {
        if (PAGED) {
            const int64_t r = cache_row(a.c, t.b, hk, j);
            if (r < 0) return make_float4(0.f, 0.f, 0.f, 0.f);
            float4 x = load4f(reinterpret_cast<const TC*>(value ? a.c.v : a.c.k) + r * a.D + d);
            if (sizeof(TC) == 1) {
                const float s = scale_of(value ? a.c.vs[r] : a.c.ks[r]);
                x.x *= s, x.y *= s, x.z *= s, x.w *= s;
            }
            return x;
        }
        const HeadView& h = value ? a.v : a.k;
        return load4f(reinterpret_cast<const TC*>(h.p + (t.k0 + j) * h.st + hk * h.sh) + d);
    }
};

// Values of masked keys.  A key that a row does not see has weight 0, but 0 * NaN or 0 * inf of its value would still
// reach the row through a matrix product.  Where rows of a block see different numbers of keys, the elements of the
// values that not all of them see are therefore made finite (zeros for the others) before the product, and rows that do
// see such an element get it added at the end, which leaves what its product with a positive weight would: infinity or NaN.
// Whether 16 bytes of bf16 (E8: of e4m3 codes) hold a non-finite element: its exponent's (magnitude's) bits are all ones, and one more
// reaches the sign's place.
template <bool E8>
__device__ __forceinline__ bool any_odd(uint4 v) {
    constexpr uint32_t BITS = E8 ? 0x7f7f7f7fu : 0x7f807f80u, ONE = E8 ? 0x01010101u : 0x00800080u;
    return ((((v.x & BITS) + ONE) | ((v.y & BITS) + ONE) | ((v.z & BITS) + ONE) | ((v.w & BITS) + ONE)) & (E8 ? 0x80808080u : 0x80008000u)) != 0u;
}
// these elements as zeros
template <bool E8>
__device__ __forceinline__ uint4 without_odd(uint4 v) {
    auto f = [](uint32_t w) { return w & ~(E8 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u)); };
    return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
}
__device__ __forceinline__ float odd_only(float x) { return fabsf(x) < INFINITY ? 0.f : x; }

// rows of a tile of the few-rows kernel
inline int rows_tile(int G, int64_t Tq, int B) { return Tq * G <= 8 * (B < Tq ? B : Tq) ? 8 : 16; }
inline int rows_tile_f32(int G, int64_t Tq, int B) {
    const int64_t n = B < Tq ? B : Tq, rows = Tq * G;
    return rows <= n ? 1 : rows <= 2 * n ? 2 : 4;
}

// keys of a tile of the CUDA-core kernel: a block's Q, K, V and weights fit an SM three times (D = 64) or twice
__host__ __device__ constexpr int simt_keys(int D) { return D == 64 ? 64 : 48; }
// query rows of a block of the tensor-core kernel, and such blocks on an SM
__host__ __device__ constexpr int tc_rows(int D) { return D == 64 ? 128 : 256; }
constexpr int tc_per_sm(int D) { return D == 64 ? 2 : 1; }

// Shared memory size of a kernel, set once per device.
inline vdm_status prepare_kernel(std::atomic<uint64_t>& ready, const void* f, int smem) {
    int dev = 0;
    VDM_CUDA_TRY(cudaGetDevice(&dev));
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (ready.load() & bit) return VDM_OK;
    if (smem) VDM_CUDA_TRY(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    ready.fetch_or(bit);
    return VDM_OK;
}

// launchers
vdm_status launch_attention_rows(const AttnArgs& a, cudaStream_t s);
vdm_status launch_attention_rows_f32(const AttnArgs& a, cudaStream_t s);
vdm_status launch_attention_simt(const AttnArgs& a, vdm_dtype dt, cudaStream_t s);
vdm_status launch_attention_tc(const AttnArgs& a, cudaStream_t s);
vdm_status launch_combine(const AttnArgs& a, vdm_dtype dt, cudaStream_t s);

struct RopeArgs {
    int64_t T;
    int Hq, Hk, D;
    HeadView q, k, qo, ko;
    const float *gq, *gk;
    float eps;
    int rot, interleaved;
    const double* inv_freq;
    float mscale;
    const int32_t* pos;
};
vdm_status launch_qk_norm_rope(const RopeArgs& a, vdm_dtype dt, cudaStream_t s);

struct CacheIo {
    CacheView c;
    HeadView k, v;
    const int32_t *cu, *kv_len;
    int B;
    int64_t T;
};
vdm_status launch_cache_write(const CacheIo& a, vdm_dtype dt, cudaStream_t s);
vdm_status launch_cache_read(const CacheIo& a, vdm_dtype dt, cudaStream_t s);

}  // namespace vdm
