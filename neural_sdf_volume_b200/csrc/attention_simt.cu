// Attention on the CUDA cores, float32 arithmetic: the kernel of float32 calls, and the
// joining of split keys.
//
// A block takes 64 query rows (query heads of a group beside one another: row = token x
// group) of one sequence and key head and runs over its keys in tiles of 64 (48 at D = 128) with the running
// maximum m and sum l of the softmax: o <- o 2^(m - m') + 2^(s - m') v, out = o / l, with
// the scale and log2 e folded into s.  Thread (ty, tx) of 8 x 16 owns rows 8 ty .. 8 ty + 7 and
// keys tx + 16 j of the scores, and columns 4 tx + 64 j of the output: 128 fused multiply-adds
// for twelve 16-byte shared loads, eight of them the same for half a warp (2 cycles of the shared memory each, 4 for
// the others): as long as the multiplications.  Measured: 2.3 GFLOP of causal sequences of up to 1027 tokens, 8/4
// heads of 64, 106 us - 21 TFLOP/s, a third of the FMA pipe, with the SMs a third of the time short of blocks.
//
// Float32 tiles come by asynchronous copies: the next keys while this tile's softmax and product
// with the values run, the next values during the next scores.
//
// A key that a row does not see has score -inf and weight 0; since 0 * NaN would still reach
// the row through the product with v, a tile whose rows see different numbers of keys multiplies
// a value only where the row sees it.
#include "seq_internal.cuh"
#include "tc_ptx.cuh"

#include <type_traits>

namespace vdm {
namespace {

constexpr int BR = 64, ST = 128, TR = 8;   // rows of a tile, threads, rows of a thread
constexpr float kLn2 = 0.69314718055994530942f;

constexpr int simt_smem(int D) { return ((BR + 2 * simt_keys(D)) * (D + 4) + BR * (simt_keys(D) + 4)) * 4; }

template <typename T, typename TC, int D, bool PAGED>
__global__ void __launch_bounds__(ST, D == 64 ? 3 : 2) attention_simt_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int BK = simt_keys(D), LD = D + 4, LP = BK + 4, NC = D / 64, TK = BK / 16;
    constexpr bool COPY = sizeof(TC) == 4;   // as they are
    extern __shared__ float4 smem4[];
    float* Qs = reinterpret_cast<float*>(smem4);
    float* Ks = Qs + BR * LD;
    float* Vs = Ks + BK * LD;
    float* Ps = Vs + BK * LD;
    RowTile t;
    const BlockPlace place = place_of<PAGED>(a);
    if (!find_tile(a, place.tile, BR, a.causal, t)) return;
    const int hk = place.hk, split = place.split;
    const KvRows<TC, PAGED> kv{a, t, hk};
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n_rows = min(BR, (int)((int64_t)t.nq * a.G - t.row0));

#pragma unroll 8
    for (int i = tid; i < BR * (D / 4); i += ST) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_rows) {
            const int row = t.row0 + r;
            x = load4f(reinterpret_cast<const T*>(a.q.p + (t.q0 + row / a.G) * a.q.st +
                                                  (int64_t)(hk * a.G + row % a.G) * a.q.sh) + d);
        }
        *reinterpret_cast<float4*>(Qs + r * LD + d) = x;
    }
    int seen[TR];
    float m[TR], l[TR], o[TR][NC][4];
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        const int r = TR * ty + i;
        seen[i] = r < n_rows ? keys_seen(a, t, (t.row0 + r) / a.G) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
    }
    // the tile's rows see at most `most` keys, and all of them see the first `least`
    const int most = keys_seen(a, t, (t.row0 + n_rows - 1) / a.G), least = keys_seen(a, t, t.row0 / a.G);
    const int n_tiles = (most + BK - 1) / BK, per = (n_tiles + a.splits - 1) / a.splits;
    const int j_end = min(most, (split + 1) * per * BK);
    // a tile of keys or values into shared memory; rows from `most` on are zeros
    auto fetch = [&](bool value, int j0) {
        float* dst = value ? Vs : Ks;
        if (COPY) {
#pragma unroll
            for (int i = 0; i < BK * (D / 4) / ST; ++i) {
                const int x = tid + ST * i, r = x / (D / 4), d = (x % (D / 4)) * 4, key = j0 + r;
                const char* src = nullptr;
                if (key < most) {
                    if (PAGED) {
                        const int64_t row = cache_row(a.c, t.b, hk, key);
                        if (row >= 0) src = (value ? a.c.v : a.c.k) + (row * D + d) * 4;
                    } else {
                        const HeadView& h = value ? a.v : a.k;
                        src = h.p + (t.k0 + key) * h.st + hk * h.sh + d * 4;
                    }
                }
                ptx::cp_async16(ptx::smem_u32(dst + r * LD + d), src ? src : a.q.p, src != nullptr);
            }
        } else {
#pragma unroll 8
            for (int i = 0; i < BK * (D / 4) / ST; ++i) {
                const int x = tid + ST * i, r = x / (D / 4), d = (x % (D / 4)) * 4;
                *reinterpret_cast<float4*>(dst + r * LD + d) = j0 + r < most ? kv.get(value, j0 + r, d) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        ptx::cp_async_commit();
    };
    const int j_begin = split * per * BK;
    if (j_begin < j_end) {
        fetch(false, j_begin);
        fetch(true, j_begin);
    }
    for (int j0 = j_begin; j0 < j_end; j0 += BK) {
        ptx::cp_async_wait<1>();   // the keys are there
        __syncthreads();
        float s[TR][TK] = {};
#pragma unroll 2
        for (int d = 0; d < D; d += 4) {
            float4 kk[TK];
#pragma unroll
            for (int j = 0; j < TK; ++j) kk[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float4 qv = *reinterpret_cast<const float4*>(Qs + (TR * ty + i) * LD + d);
#pragma unroll
                for (int j = 0; j < TK; ++j) {
                    s[i][j] = fmaf(qv.x, kk[j].x, s[i][j]);
                    s[i][j] = fmaf(qv.y, kk[j].y, s[i][j]);
                    s[i][j] = fmaf(qv.z, kk[j].z, s[i][j]);
                    s[i][j] = fmaf(qv.w, kk[j].w, s[i][j]);
                }
            }
        }
        __syncthreads();
        if (j0 + BK < j_end) fetch(false, j0 + BK);
        else ptx::cp_async_commit();
#pragma unroll
        for (int i = 0; i < TR; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                s[i][j] = j0 + tx + 16 * j < seen[i] ? s[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            float sum = 0.f;   // of this thread's keys; the row's at the end
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                Ps[(TR * ty + i) * LP + tx + 16 * j] = p;
            }
            l[i] = l[i] * f + sum;
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][c][e] *= f;
        }
        ptx::cp_async_wait<1>();   // the values are there
        __syncthreads();
        auto product = [&](auto masked) {
#pragma unroll 2
            for (int j = 0; j < BK; j += 4) {
                float4 v[4][NC];
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[jj][c] = *reinterpret_cast<const float4*>(Vs + (j + jj) * LD + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < TR; ++i) {
                    const float4 p = *reinterpret_cast<const float4*>(Ps + (TR * ty + i) * LP + j);
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        const float w = jj == 0 ? p.x : jj == 1 ? p.y : jj == 2 ? p.z : p.w;
                        if (decltype(masked)::value && j0 + j + jj >= seen[i]) continue;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            o[i][c][0] = fmaf(w, v[jj][c].x, o[i][c][0]);
                            o[i][c][1] = fmaf(w, v[jj][c].y, o[i][c][1]);
                            o[i][c][2] = fmaf(w, v[jj][c].z, o[i][c][2]);
                            o[i][c][3] = fmaf(w, v[jj][c].w, o[i][c][3]);
                        }
                    }
                }
            }
        };
        if (j0 + BK > least) product(std::true_type{});
        else product(std::false_type{});
        __syncthreads();
        if (j0 + BK < j_end) fetch(true, j0 + BK);
        else ptx::cp_async_commit();
    }
    ptx::cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
#pragma unroll
    for (int i = 0; i < TR; ++i) {
        const int r = TR * ty + i;
        if (r >= n_rows) continue;
        const int row = t.row0 + r;
        const int64_t tok = t.q0 + row / a.G;
        const int h = hk * a.G + row % a.G;
        const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
        const float lse2 = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
        const int64_t prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float4 v = make_float4(o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv, o[i][c][3] * inv);
            const int d = 64 * c + 4 * tx;
            if (a.splits > 1) store4(a.part_o + prow * D + d, v);
            else store4(reinterpret_cast<T*>(a.out.p + tok * a.out.st + h * a.out.sh) + d, v);
        }
        if (tx == 0) {
            if (a.splits > 1) a.part_lse[prow] = lse2;
            else if (a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
        }
    }
}

// Joins the splits of a query row: weights 2^(lse_s - max) over their sum.  One warp per row;
// the splits are added in order, so the result does not depend on which block ended first.
template <typename T, int D>
__global__ void __launch_bounds__(128) combine_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), rows = a.Tq * a.Hq;
    if (row >= rows) return;
    const int64_t tok = row / a.Hq;
    const int h = (int)(row % a.Hq);
    if (tok < max(a.cu_q[0], 0) || tok >= a.cu_q[a.B]) return;   // behind the last sequence: as it was
    float mx = -INFINITY;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, a.part_lse[s * rows + row]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, o[D / 32] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float lse = a.part_lse[s * rows + row];
        if (lse == -INFINITY) continue;   // no key: its part holds zeros
        const float w = exp2f(lse - base);
        sum += w;
        const float* p = a.part_o + (s * rows + row) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = fmaf(w, p[lane + 32 * e], o[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    T* out = reinterpret_cast<T*>(a.out.p + tok * a.out.st + h * a.out.sh);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[lane + 32 * e] = from_f<T>(o[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
}

template <typename T, typename TC, int D, bool PAGED>
vdm_status launch(const AttnArgs& a, cudaStream_t s) {
    const int smem = simt_smem(D);
    auto kern = attention_simt_kernel<T, TC, D, PAGED>;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), smem));
    const int64_t tiles = row_tiles(a.Tq, a.G, a.B, BR);
    kern<<<tile_grid(a, tiles), ST, smem, s>>>(a);
    VDM_TRY(check_launch("attention_simt_kernel"));
    return a.splits > 1 ? launch_combine(a, sizeof(T) == 4 ? VDM_F32 : VDM_BF16, s) : VDM_OK;
}

template <typename T, typename TC>
vdm_status launch_d(const AttnArgs& a, cudaStream_t s) {
    if (a.paged) return a.D == 64 ? launch<T, TC, 64, true>(a, s) : launch<T, TC, 128, true>(a, s);
    if constexpr (sizeof(TC) > 1) return a.D == 64 ? launch<T, TC, 64, false>(a, s) : launch<T, TC, 128, false>(a, s);
    return fail(VDM_ERR_INTERNAL, "packed keys are not 8-bit");
}

}  // namespace

vdm_status launch_attention_simt(const AttnArgs& a, vdm_dtype dt, cudaStream_t s) {
    const bool q8 = a.paged && a.c.dtype == VDM_CACHE_E4M3;
    if (dt == VDM_F32) return q8 ? launch_d<float, uint8_t>(a, s) : launch_d<float, float>(a, s);
    return q8 ? launch_d<__nv_bfloat16, uint8_t>(a, s) : launch_d<__nv_bfloat16, __nv_bfloat16>(a, s);
}

vdm_status launch_combine(const AttnArgs& a, vdm_dtype dt, cudaStream_t s) {
    const unsigned g = (unsigned)((a.Tq * a.Hq + 3) / 4);
    if (dt == VDM_F32) a.D == 64 ? combine_kernel<float, 64><<<g, 128, 0, s>>>(a) : combine_kernel<float, 128><<<g, 128, 0, s>>>(a);
    else a.D == 64 ? combine_kernel<__nv_bfloat16, 64><<<g, 128, 0, s>>>(a) : combine_kernel<__nv_bfloat16, 128><<<g, 128, 0, s>>>(a);
    return check_launch("combine_kernel");
}

}  // namespace vdm
