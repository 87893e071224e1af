// Paged cache of keys and values: writing (as is, or 8-bit with a power-of-two scale per
// row) and reading back.
//
// E4M3 row: e = min { e : max |x| <= 448 2^e }, code = rn(x 2^-e).  The scale is a power of
// two, so that code * scale is exact in float32 and bf16 and a reader adds no rounding of
// its own; the codes' relative precision is that of any other scale, since e4m3 is a
// floating format (at most one binade of its 18 goes unused).
//
// Bound by memory: an element is read once and written once.  One warp per token: its sequence and
// page are looked up once for the keys and values of all heads (the sequence by counting offsets,
// 32 at a time: one load's latency where a binary search has log2 B), and a lane has eight 16-byte
// pieces under way; a writer asks for its first eight before the lookup.
#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

// Small blocks, many on an SM.  Contexts of 460 MB read in 76 us with twenty (128 threads without a bound: 85); prompts
// of 200 MB written in 47 us with twenty and 8 elements a lane, 36 with sixteen and 16.
constexpr int CT = 64;

// Sequence that owns token t (offsets ascending), by a whole warp; -1: none.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
    const int lane = threadIdx.x & 31;
    int b = -1;   // sequences that start at or before t, minus one
    for (int b0 = 0; b0 < B; b0 += 32) {
        const uint32_t m = __ballot_sync(0xffffffffu, b0 + lane < B && cu[b0 + lane] <= t);
        b += __popc(m);
        if (m != 0xffffffffu) break;
    }
    return b >= 0 && t < cu[b + 1] ? b : -1;
}

// exponent of a row with largest finite magnitude m = f 2^E, f in [1/2, 1): 448 = 0.875 2^9, so that a
// mantissa above 1.75 needs the next one
__device__ __forceinline__ int row_exponent(float m) {
    const uint32_t u = __float_as_uint(m);
    const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u);
    return m == 0.f ? 0 : e < -100 ? -100 : e > 119 ? 119 : e;
}

// 16 bytes as floats, and their largest magnitude (bits of a float; infinities and NaN stay)
__device__ __forceinline__ uint32_t open16(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t open16(uint4 u, float (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]), m = max(m, w[i] & 0x7fffffffu);
    return m;
}

// As they are: a lane has 8 elements of a row.  E4M3: 16, so that a row's maximum takes fewer shuffles and codes leave
// 16 bytes at a time.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(CT, 16) cache_write_kernel(const __grid_constant__ CacheIo a) {
    constexpr int N = E4M3 ? 16 : 8, V = 16 / (int)sizeof(T), W = N / V, U = 8 / W;   // elements of a lane and of a load, loads, pieces under way
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int lph = a.c.D / N, hpw = 32 / lph, groups = (a.c.H + hpw - 1) / hpw;   // lanes of a head, heads of the warp
    const int e0 = (lane % lph) * N, sub = lane / lph;
    uint4 raw[U][W];
    auto load = [&](int v0) {   // v: group of heads, keys then values
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u, side = v >= groups, h = (v - side * groups) * hpw + sub;
            if (v < 2 * groups && h < a.c.H) {
                const HeadView& in = side ? a.v : a.k;
                const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(in.p + t * in.st + h * in.sh) + e0);
#pragma unroll
                for (int w = 0; w < W; ++w) raw[u][w] = p[w];
            } else {
#pragma unroll
                for (int w = 0; w < W; ++w) raw[u][w] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    load(0);
    const int b = sequence_of(a.cu, a.B, t);
    if (b < 0) return;
    const int64_t pos = (int64_t)a.kv_len[b] - (min((int64_t)a.cu[b + 1], a.T) - t);
    if (pos < 0 || pos >= (int64_t)a.c.max_pages * a.c.page_size) return;
    const int64_t r0 = cache_row(a.c, b, 0, (int)pos);
    if (r0 < 0) return;
    for (int v0 = 0; v0 < 2 * groups; v0 += U) {
        if (v0) load(v0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u, side = v >= groups, h = (v - side * groups) * hpw + sub;
            if (v >= 2 * groups) break;
            const bool on = h < a.c.H;
            char* dst = side ? a.c.v : a.c.k;
            const int64_t r = r0 + ((int64_t)h << a.c.page_shift);
            if (!E4M3) {   // the bits as they are
                if (on)
#pragma unroll
                    for (int w = 0; w < W; ++w) reinterpret_cast<uint4*>(reinterpret_cast<T*>(dst) + r * a.c.D + e0)[w] = raw[u][w];
                continue;
            }
            float x[W][V];
            uint32_t mb = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) mb = max(mb, open16(raw[u][w], x[w]));
            for (int o = 1; o < lph; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
            if (__any_sync(0xffffffffu, mb >= 0x7f800000u)) {   // infinities become NaN, and neither counts
                mb = 0;
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if (!isfinite(x[w][e])) x[w][e] = __uint_as_float(0x7fc00000u);
                        else mb = max(mb, __float_as_uint(fabsf(x[w][e])));
                    }
                for (int o = 1; o < lph; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
            }
            const int e = row_exponent(__uint_as_float(mb));
            const uint64_t inv = ptx::f32x2(pow2i(-e), pow2i(-e));
            uint32_t c[N / 4];
#pragma unroll
            for (int p = 0; p < N / 4; ++p) {
                const float* q = &x[4 * p / V][4 * p % V];
                float y[4];
                ptx::f32x2_split(ptx::mul_f32x2(ptx::f32x2(q[0], q[1]), inv), y[0], y[1]);
                ptx::f32x2_split(ptx::mul_f32x2(ptx::f32x2(q[2], q[3]), inv), y[2], y[3]);
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
                c[p] = lo | (hi << 16);
            }
            if (on) {
                *reinterpret_cast<uint4*>(dst + r * a.c.D + e0) = make_uint4(c[0], c[1], c[2 % (N / 4)], c[3 % (N / 4)]);
                if (e0 == 0) (side ? a.c.vs : a.c.ks)[r] = (uint8_t)(e + 127);
            }
        }
    }
}

template <typename TC, typename T>
__global__ void __launch_bounds__(CT, 20) cache_read_kernel(const __grid_constant__ CacheIo a) {
    constexpr bool E8 = sizeof(TC) == 1;
    // U: pieces of 16 output bytes under way, as many as keys and values of 8 heads of 128 in bf16 have for a lane.  Tokens of fewer
    // heads have fewer: 3 heads of 128 reach half the rate (51 us for 177 MB, 8 heads 76 for 463).
    constexpr int U = 8, N = 16 / (int)sizeof(T);   // N: elements of a piece
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int b = sequence_of(a.cu, a.B, t);
    if (b < 0) return;
    const int64_t pos = t - max(a.cu[b], 0);
    if (pos >= cache_len(a.c, a.kv_len[b])) return;
    const int64_t r0 = cache_row(a.c, b, 0, (int)pos);
    const int lph = a.c.D / N, hpw = 32 / lph, groups = (a.c.H + hpw - 1) / hpw;
    const int e0 = (lane % lph) * N, sub = lane / lph;
    for (int v0 = 0; v0 < 2 * groups; v0 += U) {   // groups of heads, keys then values
        uint4 raw[U];
        uint8_t sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u, side = v >= groups, h = (v - side * groups) * hpw + sub;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 127;
            if (v < 2 * groups && h < a.c.H && r0 >= 0) {   // no page: zeros
                const int64_t r = r0 + ((int64_t)h << a.c.page_shift);
                const TC* src = reinterpret_cast<const TC*>(side ? a.c.v : a.c.k) + r * a.c.D + e0;
                if constexpr (!E8) raw[u] = *reinterpret_cast<const uint4*>(src);
                else {
                    if constexpr (N == 8) {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        raw[u].x = x.x, raw[u].y = x.y;
                    } else raw[u].x = *reinterpret_cast<const uint32_t*>(src);
                    sc[u] = (side ? a.c.vs : a.c.ks)[r];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u, side = v >= groups, h = (v - side * groups) * hpw + sub;
            if (v >= 2 * groups || h >= a.c.H) continue;
            const HeadView& out = side ? a.v : a.k;
            T* d = reinterpret_cast<T*>(out.p + t * out.st + h * out.sh) + e0;
            if constexpr (!E8) *reinterpret_cast<uint4*>(d) = raw[u];
            else {
                const float s = scale_of(sc[u]);
                const uint32_t w[2] = {raw[u].x, raw[u].y};
                if constexpr (N == 8) {
                    // a code has 4 significant bits: exact in bf16, and so is its product with a power of two
                    const uint32_t ss = ptx::pack_bf16(s, s);
                    uint32_t y[4];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 lo = e4m3x2_to_f((uint16_t)w[p]), hi = e4m3x2_to_f((uint16_t)(w[p] >> 16));
                        y[2 * p] = mul_bf16x2(ptx::pack_bf16(lo.x, lo.y), ss);
                        y[2 * p + 1] = mul_bf16x2(ptx::pack_bf16(hi.x, hi.y), ss);
                    }
                    *reinterpret_cast<uint4*>(d) = make_uint4(y[0], y[1], y[2], y[3]);
                } else {
                    const float2 lo = e4m3x2_to_f((uint16_t)w[0]), hi = e4m3x2_to_f((uint16_t)(w[0] >> 16));
                    store4(reinterpret_cast<float*>(d), make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s));
                }
            }
        }
    }
}

dim3 token_grid(int64_t T) { return dim3((unsigned)((T + CT / 32 - 1) / (CT / 32))); }

}  // namespace

vdm_status launch_cache_write(const CacheIo& a, vdm_dtype dt, cudaStream_t s) {
    const dim3 g = token_grid(a.T);
    const bool q = a.c.dtype == VDM_CACHE_E4M3;
    if (dt == VDM_F32) q ? cache_write_kernel<float, true><<<g, CT, 0, s>>>(a) : cache_write_kernel<float, false><<<g, CT, 0, s>>>(a);
    else q ? cache_write_kernel<__nv_bfloat16, true><<<g, CT, 0, s>>>(a) : cache_write_kernel<__nv_bfloat16, false><<<g, CT, 0, s>>>(a);
    return check_launch("cache_write_kernel");
}

vdm_status launch_cache_read(const CacheIo& a, vdm_dtype dt, cudaStream_t s) {
    const dim3 g = token_grid(a.T);
    if (a.c.dtype == VDM_CACHE_E4M3)
        dt == VDM_F32 ? cache_read_kernel<uint8_t, float><<<g, CT, 0, s>>>(a) : cache_read_kernel<uint8_t, __nv_bfloat16><<<g, CT, 0, s>>>(a);
    else if (a.c.dtype == VDM_CACHE_F32) cache_read_kernel<float, float><<<g, CT, 0, s>>>(a);
    else cache_read_kernel<__nv_bfloat16, __nv_bfloat16><<<g, CT, 0, s>>>(a);
    return check_launch("cache_read_kernel");
}

}  // namespace vdm
