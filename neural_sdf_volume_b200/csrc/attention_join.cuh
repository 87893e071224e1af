// What the few-row attention kernels share: the joining of a tile's parts.  Every warp of the
// tile's blocks has left its rows' maxima (log2 units), sums and unnormalised elements in shared
// memory; a row's parts are added in order - first the block's warps, then the blocks of the
// cluster through distributed shared memory - so that a result does not depend on timing.
#pragma once

#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

constexpr int RM = 16;   // rows of a tile, at most
constexpr int RW = 4;    // warps of a block
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

// A row's parts of the block's warps as one: maximum (result), sum and elements.
template <int WARP>
__device__ __forceinline__ float join_warps(const float (&sm)[RW][RM], const float (&sl)[RW][RM], uint32_t at, int row, bool on, float& L, float4& x) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < RW; ++w) M = fmaxf(M, sm[w][row]);
    const float ref = M == -INFINITY ? 0.f : M;
    L = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < RW; ++w) {
        const float pm = sm[w][row], pl = sl[w][row];
        const float f = pm == -INFINITY && pl == 0.f ? 0.f : exp2f(pm - ref);
        L = fmaf(f, pl, L);
        if (on) {
            const uint4 y = lds128(at + w * WARP);
            x.x = fmaf(f, __uint_as_float(y.x), x.x), x.y = fmaf(f, __uint_as_float(y.y), x.y);
            x.z = fmaf(f, __uint_as_float(y.z), x.z), x.w = fmaf(f, __uint_as_float(y.w), x.w);
        }
    }
    return M;
}

// Rows row * D floats at part + w WARP of warp w.  Keys [j0, j1) are the ones of this split; a row that sees
// fewer of them and ends up not finite is computed again (REPAIR).
template <typename T, typename TC, int D, bool PAGED, int WARP, bool REPAIR>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const RowTile& t, int hk, int split, int rank, int cluster, int n_rows, int j0,
                                          int j1, float (&s_m)[RW][RM], float (&s_l)[RW][RM], uint32_t part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool on = 4 * lane < D;
    __syncthreads();
    if (cluster > 1) {
        for (int row = warp; row < n_rows; row += RW) {
            float L;
            float4 x;
            const float M = join_warps<WARP>(s_m, s_l, part + (row * D + 4 * lane) * 4, row, on, L, x);
            __syncwarp();
            if (on)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(part + (row * D + 4 * lane) * 4), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
            if (lane == 0) s_m[0][row] = M, s_l[0][row] = L;
        }
        ptx::cluster_sync();
    }
    for (int row = rank * RW + warp; row < n_rows; row += cluster * RW) {
        float L = 0.f, ref;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cluster == 1) {
            const float M = join_warps<WARP>(s_m, s_l, part + (row * D + 4 * lane) * 4, row, on, L, x);
            ref = M == -INFINITY ? 0.f : M;
        } else {
            // lane k: block k's maximum and sum
            float pm = -INFINITY, pl = 0.f;
            if (lane < cluster) {
                pm = ld_cluster_f32(ptx::mapa(ptx::smem_u32(&s_m[0][row]), lane));
                pl = ld_cluster_f32(ptx::mapa(ptx::smem_u32(&s_l[0][row]), lane));
            }
            float M = pm;
#pragma unroll
            for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
            ref = M == -INFINITY ? 0.f : M;
            const float pf = pm == -INFINITY && pl == 0.f ? 0.f : exp2f(pm - ref);   // no key: nothing
#pragma unroll 4
            for (int k = 0; k < cluster; ++k) {
                const float f = __shfl_sync(0xffffffffu, pf, k);
                L = fmaf(f, __shfl_sync(0xffffffffu, pl, k), L);
                if (on) {
                    const float4 y = ld_cluster_f4(ptx::mapa(part + (row * D + 4 * lane) * 4, k));
                    x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
                }
            }
        }
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        float lse2 = L == 0.f ? -INFINITY : ref + log2f(L);
        const int rr = t.row0 + row, see = keys_seen(a, t, rr / a.G);
        if (REPAIR) {
            const bool bad = !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY && fabsf(x.w) < INFINITY);
            if (see < j1 && __any_sync(0xffffffffu, bad)) lse2 = repair_row<TC, D, PAGED>(a, t, hk, rr, j0, min(see, j1), x);
        }
        const int64_t tok = t.q0 + rr / a.G;
        const int h = hk * a.G + rr % a.G;
        if (a.splits > 1) {
            const int64_t prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
            if (on) store4(a.part_o + prow * D + 4 * lane, x);
            if (lane == 0) a.part_lse[prow] = lse2;
        } else {
            if (on) store4(reinterpret_cast<T*>(a.out.p + tok * a.out.st + h * a.out.sh) + 4 * lane, x);
            if (lane == 0 && a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
        }
    }
    if (cluster > 1) ptx::cluster_sync();   // no block leaves while another reads its shared memory
}

// a launch whose blocks along z form clusters
template <typename K, typename... A>
vdm_status launch_cluster(K kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 1, at.val.clusterDim.y = 1, at.val.clusterDim.z = cluster;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    VDM_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
    return VDM_OK;
}

}  // namespace
}  // namespace vdm
