// RMS norm of query and key heads with the rotary position in the same pass.
//
//   y = x rsqrt(mean(x^2) + eps) gain ; (y_a, y_b) -> m (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
//
// One block per token: the token's angles are turned into cos and sin once (float64
// product pos * inv_freq, reduced to a fraction of a turn in float64, so that a position
// of a million keeps float32 accuracy; then sincospif) and every head of the token is
// rotated with them.  A head takes D / VEC lanes of 16 bytes each; a lane's elements and
// therefore its cos, sin and gains are the same for all heads of its side, so they stay in
// registers.  The norm is a shuffle sum inside the head's lanes.  Bound by memory: each
// element is read once and written once.
#include "seq_internal.cuh"

namespace vdm {
namespace {

constexpr int RT = 128;   // threads per block

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const char* p, float (&x)[4]) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    static __device__ __forceinline__ void store(char* p, const float (&x)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const char* p, float (&x)[8]) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(char* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// MODE 0: no rotation, 1: interleaved pairs, 2: halves
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(RT) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int N = Vec<T>::N, LPH = D / N, HPW = 32 / LPH;
    __shared__ float s_cos[D / 2], s_sin[D / 2];
    __shared__ float s_row[RT / 32][HPW][MODE == 2 ? D : 1];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = a.rot >> 1;
    if (MODE != 0) {
        for (int i = threadIdx.x; i < half; i += RT) {
            double turns = (double)a.pos[t] * a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
            turns -= rint(turns);
            float sn, cs;
            sincospif(2.0f * (float)turns, &sn, &cs);
            s_cos[i] = cs * a.mscale;
            s_sin[i] = sn * a.mscale;
        }
        __syncthreads();
    }
    const int sub = lane / LPH, e0 = (lane % LPH) * N;   // head of the warp's group, first element
    // element e0 + i: its angle and the sign of its partner's sine
    float cs[N], sn[N];
    if (MODE != 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = e0 + i;
            const int pr = MODE == 1 ? e >> 1 : e < half ? e : e - half;
            const bool first = MODE == 1 ? !(e & 1) : e < half;
            const bool in = e < a.rot;
            cs[i] = in ? s_cos[pr] : 1.0f;
            sn[i] = in ? (first ? -s_sin[pr] : s_sin[pr]) : 0.0f;
        }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int H = side ? a.Hk : a.Hq;
        const HeadView& in = side ? a.k : a.q;
        const HeadView& out = side ? a.ko : a.qo;
        const float* gain = side ? a.gk : a.gq;
        float g[N];
        if (gain) {
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = gain[e0 + i];
        }
        for (int h0 = warp * HPW; h0 < H; h0 += (RT / 32) * HPW) {
            const int h = h0 + sub;
            float x[N];
            if (h < H) Vec<T>::load(in.p + t * in.st + h * in.sh + e0 * sizeof(T), x);
            else {
#pragma unroll
                for (int i = 0; i < N; ++i) x[i] = 0.f;
            }
            if (gain) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < N; ++i) x[i] = x[i] * r * g[i];
            }
            if (MODE == 1) {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float u = x[i], w = x[i + 1];
                    x[i] = fmaf(u, cs[i], w * sn[i]);
                    x[i + 1] = fmaf(w, cs[i + 1], u * sn[i + 1]);
                }
                if (e0 >= a.rot) { /* cs = 1, sn = 0: unchanged */ }
            }
            if (MODE == 2) {
                float* row = s_row[warp][sub];
#pragma unroll
                for (int i = 0; i < N; ++i) row[e0 + i] = x[i];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int e = e0 + i;
                    if (e < a.rot) x[i] = fmaf(x[i], cs[i], row[e < half ? e + half : e - half] * sn[i]);
                }
                __syncwarp();
            }
            if (h < H) Vec<T>::store(out.p + t * out.st + h * out.sh + e0 * sizeof(T), x);
        }
    }
}

template <typename T, int D>
void launch(const RopeArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.T);
    if (!a.rot) qk_norm_rope_kernel<T, D, 0><<<grid, RT, 0, s>>>(a);
    else if (a.interleaved) qk_norm_rope_kernel<T, D, 1><<<grid, RT, 0, s>>>(a);
    else qk_norm_rope_kernel<T, D, 2><<<grid, RT, 0, s>>>(a);
}

}  // namespace

vdm_status launch_qk_norm_rope(const RopeArgs& a, vdm_dtype dt, cudaStream_t s) {
    if (dt == VDM_F32) a.D == 64 ? launch<float, 64>(a, s) : launch<float, 128>(a, s);
    else a.D == 64 ? launch<__nv_bfloat16, 64>(a, s) : launch<__nv_bfloat16, 128>(a, s);
    return check_launch("qk_norm_rope_kernel");
}

}  // namespace vdm
