// Attention of few query rows to many keys in float32: keys and values float32 (packed or paged)
// or 8-bit.  Bound by memory for float32 keys.
//
// A tile is up to R = 4 rows (token, query head of the group) of one sequence and key head; its
// keys are shared out over the warps of a cluster of blocks as in the bf16 kernel.  A warp takes four
// keys at a time, eight lanes to a key with D / 8 elements each: a key's scores need three
// shuffles a row where a key to the whole warp needs five, and q and o of the rows stay in
// registers.  Each group of eight lanes runs the softmax on its own keys (maximum, sum,
// o <- o 2^(m - m') + 2^(s - m') v); the four groups join at the end, then the warps and blocks.
// A value row counts only for rows that see it, so that what masked keys hold has no influence.
// Measured: 16 sequences of 2000 to 4000 tokens, one query token each, 32/8 heads of 128, float32: 154 us for 0.8 GB,
// 5.2 TB/s; with the keys' loads waited for step by step a 14-sequence step of 340 tokens took 17 us, two steps under
// way 11.6.
#include "attention_join.cuh"

namespace vdm {
namespace {

template <typename TC, int D, bool PAGED, int R>
__global__ void __launch_bounds__(RW * 32) attention_rows_f32_kernel(const __grid_constant__ AttnArgs a, const int cluster) {
    constexpr bool E8 = sizeof(TC) == 1;
    constexpr int NI = D / 32;            // groups of 4 elements of a lane
    constexpr int WARP = R * D * 4;
    __shared__ __align__(16) float s_part[RW][R][D];
    __shared__ float s_m[RW][RM], s_l[RW][RM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane >> 3, c = lane & 7;
    RowTile t;
    if (!find_tile(a, blockIdx.x, R, a.causal, t)) return;   // the whole cluster alike
    if (cluster > 1) cluster_started();
    const int hk = blockIdx.y, rank = blockIdx.z % cluster, split = blockIdx.z / cluster;
    const int n_rows = min(R, t.nq * a.G - t.row0);
    const int most = keys_seen(a, t, (t.row0 + n_rows - 1) / a.G);
    const int n_steps = (most + 3) / 4, per = (n_steps + a.splits - 1) / a.splits;
    const int s0 = min(n_steps, split * per), s1 = min(n_steps, s0 + per);
    auto dim = [&](int i) { return E8 ? c * (D / 8) + 4 * i : 4 * (c + 8 * i); };   // a lane's i-th group of elements

    float4 q[R][NI], o[R][NI];
    float m[R], l[R];
    int seen[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool on = r < n_rows;
        const int rr = t.row0 + (on ? r : 0);
        seen[r] = on ? keys_seen(a, t, rr / a.G) : 0;
        const float* p = reinterpret_cast<const float*>(a.q.p + (t.q0 + rr / a.G) * a.q.st + (int64_t)(hk * a.G + rr % a.G) * a.q.sh);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            q[r][i] = load4f(p + dim(i));
            o[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    // a lane's share of a key and its value, as stored; zeros where there is no key or no page
    struct Step {
        float4 k[E8 ? 1 : NI], v[E8 ? 1 : NI];
        uint32_t kc[E8 ? NI : 1], vc[E8 ? NI : 1];   // codes
        uint8_t ks, vs;
    };
    auto fetch = [&](Step& x, int step) {
        const int key = 4 * step + j;
        int64_t row = -1;
        if (step < s1 && key < most) row = PAGED ? cache_row(a.c, t.b, hk, key) : t.k0 + key;
        if constexpr (E8) {
            x.ks = x.vs = 127;
#pragma unroll
            for (int i = 0; i < NI; ++i) x.kc[i] = x.vc[i] = 0u;
            if (row >= 0) {
                const char *pk = a.c.k + row * D + dim(0), *pv = a.c.v + row * D + dim(0);
#pragma unroll
                for (int i = 0; i < NI; i += 2) {
                    const uint2 ck = *reinterpret_cast<const uint2*>(pk + 4 * i), cv = *reinterpret_cast<const uint2*>(pv + 4 * i);
                    x.kc[i] = ck.x, x.kc[i + 1] = ck.y, x.vc[i] = cv.x, x.vc[i + 1] = cv.y;
                }
                x.ks = a.c.ks[row], x.vs = a.c.vs[row];
            }
        } else {
            const char *pk = PAGED ? a.c.k + row * (D * 4) : a.k.p + row * a.k.st + hk * a.k.sh;
            const char *pv = PAGED ? a.c.v + row * (D * 4) : a.v.p + row * a.v.st + hk * a.v.sh;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                x.k[i] = x.v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0) x.k[i] = load4f(reinterpret_cast<const float*>(pk) + dim(i)), x.v[i] = load4f(reinterpret_cast<const float*>(pv) + dim(i));
            }
        }
    };
    auto use = [&](const Step& x, int step) {
        const int key = 4 * step + j;
        const float fk = E8 ? scale_of(x.ks) : 1.f, fv = E8 ? scale_of(x.vs) : 1.f;
        float s[R];
        bool raise = false;
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float4 k;
            if constexpr (E8) {
                const float2 lo = e4m3x2_to_f((uint16_t)x.kc[i]), hi = e4m3x2_to_f((uint16_t)(x.kc[i] >> 16));
                k = make_float4(lo.x * fk, lo.y * fk, hi.x * fk, hi.y * fk);
            } else k = x.k[i];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = fmaf(q[r][i].x, k.x, fmaf(q[r][i].y, k.y, fmaf(q[r][i].z, k.z, fmaf(q[r][i].w, k.w, s[r]))));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 4);
            s[r] = key < seen[r] ? s[r] * a.scale_log2 : -INFINITY;
            raise = raise || s[r] > m[r];
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float mn = fmaxf(m[r], s[r]), f = mn == -INFINITY ? 1.0f : exp2f(m[r] - mn);
                m[r] = mn;
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < NI; ++i) o[r][i].x *= f, o[r][i].y *= f, o[r][i].z *= f, o[r][i].w *= f;
            }
        }
        float p[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            p[r] = 0.f;
            if (key < seen[r]) p[r] = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r])), l[r] += p[r];
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float4 v;
            if constexpr (E8) {
                const float2 lo = e4m3x2_to_f((uint16_t)x.vc[i]), hi = e4m3x2_to_f((uint16_t)(x.vc[i] >> 16));
                v = make_float4(lo.x * fv, lo.y * fv, hi.x * fv, hi.y * fv);
            } else v = x.v[i];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (key >= seen[r]) continue;
                o[r][i].x = fmaf(p[r], v.x, o[r][i].x), o[r][i].y = fmaf(p[r], v.y, o[r][i].y);
                o[r][i].z = fmaf(p[r], v.z, o[r][i].z), o[r][i].w = fmaf(p[r], v.w, o[r][i].w);
            }
        }
    };
    // two steps under way
    const int stride = cluster * RW;
    Step x0, x1;
    int step = s0 + rank * RW + warp;
    fetch(x0, step);
    while (step < s1) {
        fetch(x1, step + stride);
        use(x0, step);
        if (step + stride >= s1) break;
        fetch(x0, step + 2 * stride);
        use(x1, step + stride);
        step += 2 * stride;
    }
    // the four groups as one, in a fixed order
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int w = 8; w < 32; w <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m[r], w), lo = __shfl_xor_sync(0xffffffffu, l[r], w);
            const float mn = fmaxf(m[r], mo), base = mn == -INFINITY ? 0.f : mn;
            // a group without keys has m = -inf, l = 0, o = 0; its factor is 0
            const float f = exp2f(m[r] - base), fo = exp2f(mo - base);
            l[r] = l[r] * f + lo * fo;
            m[r] = mn;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                o[r][i].x = o[r][i].x * f + __shfl_xor_sync(0xffffffffu, o[r][i].x, w) * fo;
                o[r][i].y = o[r][i].y * f + __shfl_xor_sync(0xffffffffu, o[r][i].y, w) * fo;
                o[r][i].z = o[r][i].z * f + __shfl_xor_sync(0xffffffffu, o[r][i].z, w) * fo;
                o[r][i].w = o[r][i].w * f + __shfl_xor_sync(0xffffffffu, o[r][i].w, w) * fo;
            }
        }
        if (lane == 0) s_m[warp][r] = m[r], s_l[warp][r] = l[r];
        if (j == 0)
#pragma unroll
            for (int i = 0; i < NI; ++i) *reinterpret_cast<float4*>(&s_part[warp][r][dim(i)]) = o[r][i];
    }
    join_rows<float, TC, D, PAGED, WARP, R, false, false>(a, t, hk, split, rank, cluster, n_rows, 0, 0, s_m, s_l, nullptr, ptx::smem_u32(&s_part[0][0][0]));
}

template <typename TC, int D, bool PAGED, int R>
vdm_status launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = attention_rows_f32_kernel<TC, D, PAGED, R>;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), 0));
    const int64_t tiles = row_tiles(a.Tq, a.G, a.B, R);
    VDM_TRY(launch_cluster(kern, dim3((unsigned)tiles, a.Hk, a.splits * a.cluster), RW * 32, 0, a.cluster, s, a, a.cluster));
    VDM_TRY(check_launch("attention_rows_f32_kernel"));
    return a.splits > 1 ? launch_combine(a, VDM_F32, s) : VDM_OK;
}

template <typename TC, bool PAGED>
vdm_status launch_d(const AttnArgs& a, cudaStream_t s) {
    const int R = rows_tile_f32(a.G, a.Tq, a.B);
    if (a.D == 64) return R == 1 ? launch<TC, 64, PAGED, 1>(a, s) : R == 2 ? launch<TC, 64, PAGED, 2>(a, s) : launch<TC, 64, PAGED, 4>(a, s);
    return R == 1 ? launch<TC, 128, PAGED, 1>(a, s) : R == 2 ? launch<TC, 128, PAGED, 2>(a, s) : launch<TC, 128, PAGED, 4>(a, s);
}

}  // namespace

vdm_status launch_attention_rows_f32(const AttnArgs& a, cudaStream_t s) {
    if (a.paged ? a.c.num_pages == 0 || a.c.max_pages == 0 : a.Tk == 0) return launch_attention_simt(a, VDM_F32, s);   // no keys at all
    if (!a.paged) return launch_d<float, false>(a, s);
    return a.c.dtype == VDM_CACHE_E4M3 ? launch_d<uint8_t, true>(a, s) : launch_d<float, true>(a, s);
}

}  // namespace vdm
