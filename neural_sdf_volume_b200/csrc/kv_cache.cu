// Paged cache of keys and values: writing (as is, or 8-bit with a power-of-two scale per
// row) and reading back.
//
// E4M3 row: e = min { e : max |x| <= 448 2^e }, code = rn(x 2^-e).  The scale is a power of
// two, so that code * scale is exact in float32 and bf16 and a reader adds no rounding of
// its own; the codes' relative precision is that of any other scale, since e4m3 is a
// floating format (at most one binade of its 18 goes unused).  Bound by memory: an element
// is read once and written once.  One warp per token and side (keys, values), all heads: the
// token's sequence and page are looked up once.
#include "seq_internal.cuh"

namespace vdm {
namespace {

constexpr int CT = 128;

// sequence that owns token t (offsets ascending): the largest b with cu[b] <= t; -1 behind the last
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    int lo = 0, hi = B;   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// exponent of a row with largest finite magnitude m: m = f 2^E, f in [1/2, 1), 448 = 0.875 2^9
__device__ __forceinline__ int row_exponent(float m) {
    if (m == 0.f) return 0;
    int E;
    const float f = frexpf(m, &E);
    const int e = f <= 0.875f ? E - 9 : E - 8;
    return e < -100 ? -100 : e > 119 ? 119 : e;
}

// 8 elements as they are (also the bits of a NaN)
template <typename T>
__device__ __forceinline__ void copy8(T* d, const T* s) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(d)[i] = reinterpret_cast<const uint4*>(s)[i];
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(CT) cache_write_kernel(const CacheIo a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int b = sequence_of(a.cu, a.B, t);
    if (b < 0) return;
    const int64_t pos = (int64_t)a.kv_len[b] - (min((int64_t)a.cu[b + 1], a.T) - t);
    if (pos < 0 || pos >= (int64_t)a.c.max_pages * a.c.page_size) return;
    const HeadView& in = blockIdx.y ? a.v : a.k;
    char* dst = blockIdx.y ? a.c.v : a.c.k;
    uint8_t* sc = blockIdx.y ? a.c.vs : a.c.ks;
    const int64_t r0 = cache_row(a.c, b, 0, (int)pos);
    if (r0 < 0) return;
    const int lph = a.c.D / 8, hpw = 32 / lph;   // 8 elements per lane
    const int e0 = (lane % lph) * 8;
    for (int h0 = 0; h0 < a.c.H; h0 += hpw) {
        const int h = h0 + lane / lph;
        const bool on = h < a.c.H;
        const T* src = reinterpret_cast<const T*>(in.p + t * in.st + (on ? h : 0) * in.sh) + e0;
        const int64_t r = r0 + ((int64_t)h << a.c.page_shift);
        if (!E4M3) {
            if (on) copy8(reinterpret_cast<T*>(dst) + r * a.c.D + e0, src);
            continue;
        }
        const float4 x0 = load4f(src), x1 = load4f(src + 4);
        float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!isfinite(x[i])) x[i] = __uint_as_float(0x7fc00000u);   // fmaxf drops NaN
            m = fmaxf(m, fabsf(x[i]));
        }
        for (int o = 1; o < lph; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = row_exponent(m);
        const float inv = pow2i(-e);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        if (on) {
            *reinterpret_cast<uint2*>(dst + r * a.c.D + e0) = make_uint2(w[0], w[1]);
            if (e0 == 0) sc[r] = (uint8_t)(e + 127);
        }
    }
}

template <typename TC, typename T>
__global__ void __launch_bounds__(CT) cache_read_kernel(const CacheIo a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int b = sequence_of(a.cu, a.B, t);
    if (b < 0) return;
    const int64_t pos = t - max(a.cu[b], 0);
    if (pos >= cache_len(a.c, a.kv_len[b])) return;
    const HeadView& out = blockIdx.y ? a.v : a.k;
    const TC* src = reinterpret_cast<const TC*>(blockIdx.y ? a.c.v : a.c.k);
    const uint8_t* sc = blockIdx.y ? a.c.vs : a.c.ks;
    const int64_t r0 = cache_row(a.c, b, 0, (int)pos);
    const int lph = a.c.D / 8, hpw = 32 / lph;
    const int e0 = (lane % lph) * 8;
    for (int h = lane / lph; h < a.c.H; h += hpw) {
        T* d = reinterpret_cast<T*>(out.p + t * out.st + h * out.sh) + e0;
        float4 x0 = make_float4(0.f, 0.f, 0.f, 0.f), x1 = x0;
        if (r0 >= 0) {
            const int64_t r = r0 + ((int64_t)h << a.c.page_shift);
            if constexpr (sizeof(TC) > 1) {
                copy8(d, src + r * a.c.D + e0);
                continue;
            }
            x0 = load4f(src + r * a.c.D + e0);
            x1 = load4f(src + r * a.c.D + e0 + 4);
            if (sizeof(TC) == 1) {
                const float s = scale_of(sc[r]);
                x0.x *= s, x0.y *= s, x0.z *= s, x0.w *= s;
                x1.x *= s, x1.y *= s, x1.z *= s, x1.w *= s;
            }
        }
        store4(d, x0);
        store4(d + 4, x1);
    }
}

dim3 token_grid(int64_t T) { return dim3((unsigned)((T + CT / 32 - 1) / (CT / 32)), 2); }

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
