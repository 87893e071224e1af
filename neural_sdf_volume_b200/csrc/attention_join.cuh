// What the few-row attention kernels share: the joining of a tile's parts.  Every warp of the
// tile's blocks has left its rows' references (log2 units), sums and unnormalised elements in shared
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
__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f4(uint32_t a, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
// "this block runs", told to the cluster early and asked for before the first write into another block
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What a row's four elements x get of the non-finite values of keys [j0, j1), which the product left out (see odd_only).  Out of
// line, with arguments that need no place in memory: the few-row kernels run their code once, and what they do not run is
// better elsewhere (by references: 3 us of 44, four tokens each over 2000 to 8000).
template <typename TC, int D, bool PAGED>
__device__ __noinline__ float4 add_odd(const AttnArgs* a, int b, int64_t k0, int hk, int j0, int j1, float4 x) {
    const int d = 4 * (threadIdx.x & 31);
    RowTile t;
    t.b = b, t.k0 = k0;
    const KvRows<TC, PAGED> kv{*a, t, hk};
    for (int j = j0; j < j1 && d < D; ++j) {
        const float4 v = kv.get(true, j, d);
        x.x += odd_only(v.x), x.y += odd_only(v.y), x.z += odd_only(v.z), x.w += odd_only(v.w);
    }
    return x;
}

// Parts of a lane's row (row = lane % 16) as factors of one sum: references pm of their elements, their sums pl against
// these - or, LOG, the log2 of the sums - -> factors f of the elements, the sum L; returns the reference that f refers to,
// sum_ref the one of L (0 for -inf).
template <bool LOG, int P>
__device__ __forceinline__ float join_factors(const float (&pm)[P], const float (&pl)[P], float (&f)[P], float& L, float& sum_ref) {
    auto top = [](const float (&x)[P]) {
        float M = x[0];
#pragma unroll
        for (int p = 1; p < P; ++p) M = fmaxf(M, x[p]);
        return M == -INFINITY ? 0.f : M;
    };
    const float ref = top(pm);
    sum_ref = LOG ? top(pl) : ref;
    L = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        f[p] = pm[p] == -INFINITY && pl[p] == (LOG ? -INFINITY : 0.f) ? 0.f : exp2f(pm[p] - ref);   // no key: nothing
        L = LOG ? L + exp2f(pl[p] - sum_ref) : fmaf(f[p], pl[p], L);
    }
    return ref;
}

__device__ __forceinline__ void add_part(float4& x, float f, const float4& y) {
    x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
}

// Rows row * D floats at part + w WARP of warp w.  What is one number a row (maxima, factors, addresses) is
// computed for all rows at once, a lane each; then a warp adds up its rows' elements.  In a cluster block b
// finishes the rows b, b + n, ...: the others write their parts of them into its shared memory, so that one
// barrier is enough (reading them there took a second one, before a block may leave, and 2 us in all).
// CLEAN: the values of keys [j0, j1) have lost their non-finite elements before the product, if a warp says so in s_odd;
// they are added here to the rows that see them.  ROWS: rows of a tile, at most.  LOG: s_l holds the log2 of the sums, which may lie some 200 from the
// elements' references.
template <typename T, typename TC, int D, bool PAGED, int WARP, int ROWS, bool CLEAN, bool LOG>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const RowTile& t, int hk, int split, int rank, int cluster, int n_rows, int j0,
                                          int j1, float (&s_m)[RW][RM], float (&s_l)[RW][RM], const int* s_odd, uint32_t part) {
    constexpr int MAXC = 8;                          // blocks of a cluster, at most
    constexpr int TAKE = ROWS > MAXC ? ROWS : MAXC;  // rows that come in: a row of every block for each of its own
    __shared__ __align__(16) float s_in[TAKE][D];
    __shared__ float s_mi[TAKE], s_li[TAKE], s_oi[MAXC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = lane & (RM - 1);
    const bool on = 4 * lane < D;
    const uint32_t at = part + 16 * lane;
    __syncthreads();
    bool odd = CLEAN && j0 < j1 && (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]);
    float fw[RW], L, sum_ref, ref;
    {
        float pm[RW], pl[RW];
#pragma unroll
        for (int w = 0; w < RW; ++w) pm[w] = s_m[w][mine], pl[w] = s_l[w][mine];
        ref = join_factors<LOG>(pm, pl, fw, L, sum_ref);
    }
    auto warps_sum = [&](int row) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            const float f = __shfl_sync(0xffffffffu, fw[w], row);
            if (on) {
                const uint4 y = lds128(at + w * WARP + row * D * 4);
                add_part(x, f, make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w)));
            }
        }
        return x;
    };
    // row -> block row % cluster, its row / cluster -th; that block's place for part k: k own + row / cluster
    const int own = (ROWS + cluster - 1) / cluster;
    if (cluster > 1) {
        cluster_wait();
        for (int row = warp; row < n_rows; row += RW) {
            const float4 x = warps_sum(row);
            if (on) st_cluster_f4(ptx::mapa(ptx::smem_u32(&s_in[rank * own + row / cluster][4 * lane]), row % cluster), x);
        }
        if (warp == 0 && lane < n_rows) {   // no key: -inf and 0
            const int place = rank * own + mine / cluster;
            st_cluster_f32(ptx::mapa(ptx::smem_u32(&s_mi[place]), mine % cluster), L == 0.f ? -INFINITY : ref);
            st_cluster_f32(ptx::mapa(ptx::smem_u32(&s_li[place]), mine % cluster), LOG ? (L == 0.f ? -INFINITY : sum_ref + log2f(L)) : L);
        }
        if (CLEAN && j0 < j1 && warp == 1 && lane < cluster) st_cluster_f32(ptx::mapa(ptx::smem_u32(&s_oi[rank]), lane), odd ? 1.0f : 0.f);
        ptx::cluster_sync();
        if (CLEAN && j0 < j1)
            for (int k = 0; k < cluster; ++k) odd = odd || s_oi[k] != 0.f;
    }
    // from here a lane's row is the mine-th of the block's own (all rows without a cluster)
    const int n_own = cluster == 1 ? n_rows : (n_rows - rank + cluster - 1) / cluster;
    float fc[MAXC];
    if (cluster > 1) {
        float pm[MAXC], pl[MAXC];
#pragma unroll
        for (int k = 0; k < MAXC; ++k) {
            const bool there = k < cluster && mine < n_own;
            pm[k] = there ? s_mi[k * own + mine] : -INFINITY;
            pl[k] = there ? s_li[k * own + mine] : LOG ? -INFINITY : 0.f;
        }
        ref = join_factors<LOG>(pm, pl, fc, L, sum_ref);
    }
    const float lse2 = L == 0.f ? -INFINITY : sum_ref + log2f(L), inv = L == 0.f ? 0.f : LOG ? exp2f(ref - lse2) : 1.0f / L;
    const int rr = t.row0 + min(mine * cluster + rank, n_rows - 1), see = keys_seen(a, t, rr / a.G), h = hk * a.G + rr % a.G;
    const int64_t tok = t.q0 + rr / a.G, prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
    const bool parts = a.splits > 1;
    char* const dst = parts ? reinterpret_cast<char*>(a.part_o + prow * D) : a.out.p + tok * a.out.st + h * a.out.sh;
    if (warp == 0 && lane < n_own) {
        if (parts) a.part_lse[prow] = lse2;
        else if (a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
    }
    for (int row = warp; row < n_own; row += RW) {
        float4 x;
        if (cluster == 1) x = warps_sum(row);
        else {
            x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < MAXC; ++k) {
                const float f = __shfl_sync(0xffffffffu, fc[k], row);
                if (k < cluster && on) add_part(x, f, *reinterpret_cast<const float4*>(&s_in[k * own + row][4 * lane]));
            }
        }
        const float i = __shfl_sync(0xffffffffu, inv, row);
        x.x *= i, x.y *= i, x.z *= i, x.w *= i;
        char* const p = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
        if (CLEAN && odd) {
            const int end = min(__shfl_sync(0xffffffffu, see, row), j1);
            if (__shfl_sync(0xffffffffu, L, row) != 0.f) x = add_odd<TC, D, PAGED>(&a, t.b, t.k0, hk, j0, end, x);
        }
        if (on) {
            if (parts) store4(reinterpret_cast<float*>(p) + 4 * lane, x);
            else store4(reinterpret_cast<T*>(p) + 4 * lane, x);
        }
    }
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
