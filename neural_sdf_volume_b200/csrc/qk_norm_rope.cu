// RMS norm of query and key heads with the rotary position in the same pass.
//
//   y = x rsqrt(mean(x^2) + eps) gain ; (y_a, y_b) -> m (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
//
// A head takes D / N lanes of 16 bytes each.  One, two or four warps of a block share a token; a
// lane's elements and therefore its cos and sin are the same for all heads, so they stay in
// registers.  A lane asks for five heads before it uses the first, and for the first five before
// the token's angles are turned into cos and sin (float64 product pos * inv_freq, reduced to a
// fraction of a turn in float64, so that a position of a million keeps float32 accuracy; then
// sincospif).  The norm is a shuffle sum inside the head's lanes.  Bound by memory: each element is
// read once and written once.
#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

constexpr int RT = 128;   // threads per block
// Loads of a lane under way: five of 16 bytes fit 64 registers, and with them eight blocks on an SM.  40 heads of 128 are one full
// round of a block's four warps (73 us for 16381 tokens); other numbers leave slots of the last round empty: 24 + 2 heads of 64 use
// seven of ten (29 us for a third of the bytes).
constexpr int RU = 5;

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(uint4 u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// MODE 0: no rotation, 1: interleaved pairs, 2: halves, 3: halves of a multiple of N / 2 elements: a lane then takes N / 2
// elements of each half, so that its pairs are its own (16381 tokens of 40 heads of 128: 74 us; by an exchange through
// shared memory, as for other halves, 145: it spills)
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(RT, 8) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a, const int wpt) {
    constexpr int N = Vec<T>::N, LPH = D / N, HPW = 32 / LPH;
    constexpr int NP = MODE == 2 ? N : N / 2;   // angles of a lane: of each element, or of each pair
    __shared__ float s_cos[RT / 32][D / 2], s_sin[RT / 32][D / 2];
    __shared__ __align__(16) float s_gain[2][D];
    __shared__ __align__(16) float s_row[RT / 32][HPW][MODE == 2 ? D : 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = warp / wpt, part = warp % wpt;
    const int64_t t = (int64_t)blockIdx.x * (RT / 32 / wpt) + slot;
    const bool live = t < a.T;
    const int half = a.rot >> 1, H = a.Hq + a.Hk;
    const int sub = lane / LPH, li = lane % LPH;   // head of the warp's group
    // a lane's elements: N / 2 from e0 and N / 2 from e1
    const bool split = MODE == 3 && li * N < a.rot;
    const int e0 = split ? li * (N / 2) : li * N, e1 = split ? half + e0 : e0 + N / 2;
    uint4 raw[RU];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int h = h0 + u * wpt * HPW;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h < H) {
                const char* p = h < a.Hq ? a.q.p + t * a.q.st + h * a.q.sh : a.k.p + t * a.k.st + (h - a.Hq) * a.k.sh;
                if (MODE == 3) {
                    const uint2 lo = *reinterpret_cast<const uint2*>(p + e0 * (int)sizeof(T)), hi = *reinterpret_cast<const uint2*>(p + e1 * (int)sizeof(T));
                    raw[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                } else raw[u] = *reinterpret_cast<const uint4*>(p + e0 * (int)sizeof(T));
            }
        }
    };
    const int first = part * HPW + sub;
    load(first);
    for (int i = threadIdx.x; i < D; i += RT) {
        s_gain[0][i] = a.gq ? a.gq[i] : 1.0f;
        s_gain[1][i] = a.gk ? a.gk[i] : 1.0f;
    }
    float cs[NP], sn[NP];
    if (MODE == 0) __syncthreads();
    else {
        if (live)
            for (int i = part * 32 + lane; i < half; i += 32 * wpt) {
                double turns = (double)a.pos[t] * a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
                turns -= rint(turns);
                float s, c;
                sincospif(2.0f * (float)turns, &s, &c);
                s_cos[slot][i] = c * a.mscale;
                s_sin[slot][i] = s * a.mscale;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int e = MODE == 1 ? e0 + 2 * i : e0 + i;
            const bool in = e < a.rot;
            const int pr = !in ? 0 : MODE == 1 ? e >> 1 : e < half ? e : e - half;
            cs[i] = in ? s_cos[slot][pr] : 1.0f;
            sn[i] = in ? s_sin[slot][pr] : 0.0f;
            if (MODE == 2 && e < half) sn[i] = -sn[i];   // the first of a pair
        }
    }
    for (int h0 = first; h0 < H + sub; h0 += RU * wpt * HPW) {   // the same number of rounds for the whole warp
        if (h0 != first) load(h0);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int h = h0 + u * wpt * HPW;
            if (h - sub >= H) break;
            float x[N];
            Vec<T>::open(raw[u], x);
            const bool isq = h < a.Hq;
            uint64_t sq = ptx::f32x2(0.f, 0.f);   // pairs of elements: half the instructions
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t p = ptx::f32x2(x[i], x[i + 1]);
                sq = ptx::fma_f32x2(p, p, sq);
            }
            float ss, s1;
            ptx::f32x2_split(sq, ss, s1);
            ss += s1;
#pragma unroll
            for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (isq ? a.gq != nullptr : a.gk != nullptr) {
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
                const uint64_t rr = ptx::f32x2(r, r);
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 g = *reinterpret_cast<const float2*>(&s_gain[isq ? 0 : 1][i < N / 2 ? e0 + i : e1 + i - N / 2]);
                    ptx::f32x2_split(ptx::mul_f32x2(ptx::mul_f32x2(ptx::f32x2(x[i], x[i + 1]), rr), ptx::f32x2(g.x, g.y)), x[i], x[i + 1]);
                }
            }
            if (MODE == 1) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float v = x[2 * i], w = x[2 * i + 1];
                    if (e0 + 2 * i < a.rot) {
                        x[2 * i] = fmaf(v, cs[i], -(w * sn[i]));
                        x[2 * i + 1] = fmaf(w, cs[i], v * sn[i]);
                    }
                }
            }
            if (MODE == 3 && split) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float v = x[i], w = x[i + N / 2];
                    x[i] = fmaf(v, cs[i], -(w * sn[i]));
                    x[i + N / 2] = fmaf(w, cs[i], v * sn[i]);
                }
            }
            if (MODE == 2) {
                float* row = s_row[warp][sub];
#pragma unroll
                for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(row + e0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int e = e0 + i;
                    if (e < a.rot) x[i] = fmaf(x[i], cs[i], row[e < half ? e + half : e - half] * sn[i]);
                }
                __syncwarp();
            }
            if (live && h < H) {
                char* p = isq ? a.qo.p + t * a.qo.st + h * a.qo.sh : a.ko.p + t * a.ko.st + (h - a.Hq) * a.ko.sh;
                const uint4 y = Vec<T>::pack(x);
                if (MODE == 3) {
                    *reinterpret_cast<uint2*>(p + e0 * (int)sizeof(T)) = make_uint2(y.x, y.y);
                    *reinterpret_cast<uint2*>(p + e1 * (int)sizeof(T)) = make_uint2(y.z, y.w);
                } else *reinterpret_cast<uint4*>(p + e0 * (int)sizeof(T)) = y;
            }
        }
    }
}

template <typename T, int D>
void launch(const RopeArgs& a, cudaStream_t s) {
    // warps of a token: as many as its heads keep busy; all four where tokens are few
    const int vecs = (a.Hq + a.Hk) * (D / Vec<T>::N);
    const int wpt = a.T <= 592 || vecs >= 4 * 32 * RU ? 4 : vecs >= 2 * 32 * RU ? 2 : 1;
    const int64_t per = RT / 32 / wpt;
    const dim3 grid((unsigned)((a.T + per - 1) / per));
    if (!a.rot) qk_norm_rope_kernel<T, D, 0><<<grid, RT, 0, s>>>(a, wpt);
    else if (a.interleaved) qk_norm_rope_kernel<T, D, 1><<<grid, RT, 0, s>>>(a, wpt);
    else if (a.rot % Vec<T>::N == 0) qk_norm_rope_kernel<T, D, 3><<<grid, RT, 0, s>>>(a, wpt);
    else qk_norm_rope_kernel<T, D, 2><<<grid, RT, 0, s>>>(a, wpt);
}

}  // namespace

vdm_status launch_qk_norm_rope(const RopeArgs& a, vdm_dtype dt, cudaStream_t s) {
    if (dt == VDM_F32) a.D == 64 ? launch<float, 64>(a, s) : launch<float, 128>(a, s);
    else a.D == 64 ? launch<__nv_bfloat16, 64>(a, s) : launch<__nv_bfloat16, 128>(a, s);
    return check_launch("qk_norm_rope_kernel");
}

}  // namespace vdm
