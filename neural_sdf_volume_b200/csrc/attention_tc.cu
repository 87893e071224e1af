// Attention on the 5th-generation tensor cores: bf16 queries with packed bf16, paged bf16 or
// paged 8-bit keys and values.
//
//   S = Q K^T (bf16 in, fp32 in TMEM) ; softmax with the running maximum m and sum l ;
//   O <- O + P V (P bf16 in TMEM, O fp32 in TMEM) ; out = O / l
//
// One CTA takes 256 query rows (row = token x group: the query heads of a key head beside one
// another, so that a group shares its keys' loads) as two tiles of 128, and runs over the keys
// in tiles of 128.  Roles:
//   warps 0-3, 4-7  softmax of tile 0 and 1, one row per thread: S from TMEM, maximum,
//                   2^(scale log2e s - m), P back into the columns of S (bf16), sum in fp32;
//   warp 8          issues the MMAs of both tiles in turn: while one tile's softmax runs, the
//                   tensor cores work on the other's;
//   warp 9          TMA loads of K and V tiles into a ring of slots (packed: one box of 128
//                   tokens per 64 columns; paged: one box per page);
//   warps 9-11      (8-bit cache) instead read codes from global memory, widen them to bf16 -
//                   exact: a code times a power of two - and write the ring's slots.
// The maximum that the exponents refer to follows the running maximum only when that has
// grown by more than 8 (log2 units): then O and l are rescaled, which needs the previous
// product to have finished; otherwise P stays below 2^8 and nothing is lost.  l sums the fp32
// exponentials; only the product uses their bf16 roundings.
//
// TMEM (512 columns): S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D); P_w overwrites
// the first 64 columns of S_w.
//
// Masked keys: a key that a row does not see has weight 0.  V rows behind the sequence's end
// are zeroed in shared memory (0 * NaN would reach every row); V rows inside the sequence that
// only later queries see can still bring 0 * NaN or 0 * inf, so that a row which ends up not
// finite while keys of its tiles were masked is computed again, over its own keys alone
// (repair_row, one warp per row; never taken with finite values).
//
// Every wait is bounded; on expiry the kernel sets the error word, winds down and frees TMEM.
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

using namespace ptx;

constexpr int BM = 128, BN = 128;
#ifndef VDM_POLY64
#define VDM_POLY64 3
#define VDM_POLY128 2
#endif
constexpr int THREADS = 384;                        // three warpgroups, launched with 168 registers a thread
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;  // 2 * 208 + 88 = 3 * 168
enum Source : int { kPacked = 0, kPagedBf16 = 1, kPagedE4m3 = 2 };
constexpr uint32_t T_O = 256;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D> struct Cfg {
    static constexpr int PANELS = D / 64;
    static constexpr int QBYTES = BM * D * 2;        // one query tile
    static constexpr int SLOT = BN * D * 2;          // one key or value tile
    static constexpr int NS = D == 128 ? 5 : 8;      // slots beside two query tiles in 227 KB
    static constexpr int SMEM = 2 * QBYTES + NS * SLOT + 1024;
};

struct Shared {
    uint64_t full[8], empty[8], s_full[2], p_full[2], pv_done[2];
    uint32_t tmem;
    int abort;
};

struct Wait {
    Shared* sh;
    int* err;
    long long timeout;
    // whole warps; false: gave up
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, int site) const {
        const uint32_t b = smem_u32(bar);
        long long t0 = 0;
        bool done = false;
        for (uint32_t it = 0;; ++it) {
            if (mbar_try_wait(b, parity)) {
                done = true;
                break;
            }
            if ((it & 63) == 63) {
                if (*reinterpret_cast<volatile int*>(&sh->abort)) break;
                const long long t = clock64();
                if (t0 == 0) t0 = t;
                else if (t - t0 > timeout) {
                    *reinterpret_cast<volatile int*>(&sh->abort) = 1;
                    atomicCAS(err, 0, site);
                    break;
                }
            }
        }
        return __all_sync(0xffffffffu, done);
    }
};

// waits for the kernel's own loads and MMAs, which complete by themselves; bounded all the same
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, long long cycles) {
    const long long t0 = clock64();
    while (!mbar_try_wait(smem_u32(bar), parity) && clock64() - t0 < cycles) {
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// value tile as B operand read along its rows (MN-major, 128-byte swizzle): 8-row groups 1024
// bytes apart, 64-column panels 16 KB apart
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// byte offset of 16-byte chunk c (of D / 8) of row r in a tile of 128-byte-swizzled 64-column panels
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)((c >> 3) * (BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void st_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, int SRC>
__global__ void __launch_bounds__(THREADS, 1)
attention_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ AttnArgs a, const int tok_first) {
    using C = Cfg<D>;
    constexpr int NS = C::NS;
    constexpr int NPROD = SRC == kPagedE4m3 ? 96 : 1;   // arrivals that complete a slot
    extern __shared__ uint8_t dyn_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    RowTile t;
    if (!find_tile(a, blockIdx.x, 2 * BM, a.causal, t)) return;
    const int hk = blockIdx.y, split = blockIdx.z;
    const int total_rows = t.nq * a.G;
    const uint32_t base = (smem_u32(dyn_raw) + 1023u) & ~1023u;
    const uint32_t s_ring = base + 2 * C::QBYTES;

    // key tiles of each row tile: [jb, je[w])
    int je[2], jb;
    {
        int n[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int first = t.row0 + w * BM, last = min(first + BM, total_rows) - 1;
            n[w] = first < total_rows ? (keys_seen(a, t, last / a.G) + BN - 1) / BN : 0;
        }
        const int most = max(n[0], n[1]), per = (most + a.splits - 1) / a.splits;
        jb = split * per;
        je[0] = max(jb, min(n[0], jb + per));
        je[1] = max(jb, min(n[1], jb + per));
    }
    const int jmax = max(je[0], je[1]);
    const Wait wait{&sh, a.err, a.timeout};

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&sh.full[i]), NPROD);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&sh.s_full[w]), 1);
            mbar_init(smem_u32(&sh.p_full[w]), BM);
            mbar_init(smem_u32(&sh.pv_done[w]), 1);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    // queries: rows beyond the last are zeros
    if (tid < 256) {
        for (int i = tid; i < 2 * BM * (D / 8); i += 256) {
            const int r = i / (D / 8), c = i % (D / 8), row = t.row0 + r;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (row < total_rows)
                x = *reinterpret_cast<const uint4*>(a.q.p + (t.q0 + row / a.G) * a.q.st +
                                                    (int64_t)(hk * a.G + row % a.G) * a.q.sh + c * 16);
            st_v4(base + (r >> 7) * C::QBYTES + tile_off(r & 127, c), x.x, x.y, x.z, x.w);
        }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_up<REGS_SOFTMAX>();
        const int w = warp >> 2;
        const int row = t.row0 + w * BM + (tid & 127);
        const int seen = row < total_rows ? keys_seen(a, t, row / a.G) : 0;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128 * w + lanes, to = tmem + T_O + 128 * w + lanes;
        const float sc = a.scale_log2;
        float m = -INFINITY, l = 0.f;   // m: reference of the exponents (unscaled score units)
        bool ok = true;
        for (int j = jb; j < je[w]; ++j) {
            const uint32_t par = (j - jb) & 1;
            if (!(ok = wait(&sh.s_full[w], par, 1))) break;
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) reg_fence(s[c]);
            const int left = seen - j * BN;   // keys of this tile that the row sees
            if (__any_sync(0xffffffffu, left < BN)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[c][i] = 32 * c + i < left ? s[c][i] : -INFINITY;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mx[c] = fmax3_nan(s[c][0], s[c][1], s[c][2]);
#pragma unroll
                for (int i = 3; i < 31; i += 2) mx[c] = fmax3_nan(mx[c], s[c][i], s[c][i + 1]);
            }
            const float mt = fmax3_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3], fmax3_nan(s[0][31], s[1][31], fmax3_nan(s[2][31], s[3][31], s[3][31])));
            // a score that is NaN or +inf: the row's result is NaN, whatever becomes of its weights
            if (!(mt < INFINITY)) l = __uint_as_float(0x7fc00000u);
            const float mn = fmaxf(m, mt);
            // raise the reference only when it has grown by more than 2^8 (or was -inf)
            const bool raise = (mn - m) * sc > 8.0f;
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise ? exp2f((m - mn) * sc) : 1.0f;
                if (raise) m = mn;
                l *= f;
                if (j > jb) {
                    if (!(ok = wait(&sh.pv_done[w], (j - jb - 1) & 1, 2))) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(to + 32 * c, o);
                        tmem_wait_ld();
                        reg_fence(o);
                        uint32_t u[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
                        tmem_st32(to + 32 * c, u);
                    }
                    tmem_wait_st();
                }
            }
            const float ref = m == -INFINITY ? 0.f : m * sc;
            const uint64_t sc2 = f32x2(sc, sc), ref2 = f32x2(-ref, -ref);
            uint64_t sum = f32x2(0.f, 0.f);
            // Of every 8 pairs POLY are computed on the FMA pipe: the special-function unit alone takes as
            // long for a tile as the matrix products at D = 128, twice as long at D = 64.  Masked scores, and
            // rows that have seen none above -inf, need exact zeros: no polynomials there.
            const bool plain = __any_sync(0xffffffffu, left < BN || m == -INFINITY);
            auto weights = [&](auto poly) {
                constexpr int POLY = decltype(poly)::value;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x = fma_f32x2(f32x2(s[c][2 * i], s[c][2 * i + 1]), sc2, ref2);
                        uint64_t e;
                        if (i % 8 < POLY) e = exp2_pair_poly(x);
                        else {
                            float x0, x1;
                            f32x2_split(x, x0, x1);
                            e = f32x2(ex2(x0), ex2(x1));
                        }
                        sum = add_f32x2(sum, e);
                        float e0, e1;
                        f32x2_split(e, e0, e1);
                        p[i] = pack_bf16(e0, e1);
                    }
                    tmem_st16(ts + 16 * c, p);
                }
            };
            if (plain) weights(std::integral_constant<int, 0>{});
            else weights(std::integral_constant<int, D == 64 ? VDM_POLY64 : VDM_POLY128>{});
            float s0, s1;
            f32x2_split(sum, s0, s1);
            l += s0 + s1;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.p_full[w]));
        }
        // ------------------------------------------------------------ output
        const int cnt = je[w] - jb;
        if (ok && cnt > 0) ok = wait(&sh.pv_done[w], (cnt - 1) & 1, 3);
        tc_fence_after();
        if (ok && __any_sync(0xffffffffu, row < total_rows)) {
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * sc) + log2f(l);
            const bool live = row < total_rows;
            const int64_t tok = t.q0 + (live ? row / a.G : 0);
            const int h = hk * a.G + (live ? row % a.G : 0);
            const int64_t prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
            char* dst = a.splits > 1 ? reinterpret_cast<char*>(a.part_o + prow * D) : a.out.p + tok * a.out.st + h * a.out.sh;
            bool finite = true;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (cnt > 0) {
                    tmem_ld32(to + 32 * c, o);
                    tmem_wait_ld();
                    reg_fence(o);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    o[i] = l == 0.f ? 0.f : o[i] * inv;
                    finite = finite && fabsf(o[i]) < INFINITY;
                }
                if (!live) continue;
                if (a.splits > 1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(dst + (32 * c + i) * 4) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4*>(dst + (32 * c + i) * 2) =
                            make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]), pack_bf16(o[i + 4], o[i + 5]),
                                       pack_bf16(o[i + 6], o[i + 7]));
                }
            }
            if (live) {
                if (a.splits > 1) a.part_lse[prow] = lse2;
                else if (a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
            }
            // a row that masked keys of its tiles and is not finite: again over its own keys
            uint32_t again = __ballot_sync(0xffffffffu, live && !finite && seen < min(je[w] * BN, t.nk));
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const int r = __shfl_sync(0xffffffffu, row, src), end = __shfl_sync(0xffffffffu, seen, src);
                const int64_t pr = __shfl_sync(0xffffffffu, prow, src);
                float4 o;
                const float lg = repair_row<typename std::conditional<SRC == kPagedE4m3, uint8_t, __nv_bfloat16>::type, D, SRC != kPacked>(
                    a, t, hk, r, jb * BN, min(end, je[w] * BN), o);
                const int64_t rt = t.q0 + r / a.G;
                const int rh = hk * a.G + r % a.G;
                if (4 * lane < D) {
                    if (a.splits > 1) store4(a.part_o + pr * D + 4 * lane, o);
                    else store4(reinterpret_cast<__nv_bfloat16*>(a.out.p + rt * a.out.st + rh * a.out.sh) + 4 * lane, o);
                }
                if (lane == 0) {
                    if (a.splits > 1) a.part_lse[pr] = lg;
                    else if (a.lse) a.lse[rt * a.Hq + rh] = lg * kLn2;
                }
            }
        }
        tc_fence_before();
    } else {
      regs_down<REGS_OTHER>();
      if (warp == 8) {
        // ------------------------------------------------------------ MMA issue
        constexpr uint32_t id_s = idesc_bf16(BM, BN, false), id_o = idesc_bf16(BM, D, true);
        const int n = jmax - jb;
        auto issue_s = [&](int w, uint32_t slot) {
            const uint64_t dq = desc_sw128(base + w * C::QBYTES), dk = desc_sw128(s_ring + slot * C::SLOT);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)((kk >> 2) * (BN * 128 / 16) + (kk & 3) * 2);
                mma_ss_w(tmem + 128 * w, dq + off, dk + off, id_s, kk > 0);
            }
            mma_commit_w(smem_u32(&sh.s_full[w]));
        };
        bool ok = true;
        if (n > 0 && (ok = wait(&sh.full[0], 0, 4))) {
            tc_fence_after();
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if (je[w] > jb) issue_s(w, 0);
            mma_commit_w(smem_u32(&sh.empty[0]));
        }
        for (int i = 0; ok && i < n; ++i) {
            const uint32_t iv = 2 * i + 1, ik = 2 * i + 2, sv = iv % NS, sk = ik % NS;
            if (!(ok = wait(&sh.full[sv], (iv / NS) & 1, 5))) break;
            const int valid = t.nk - (jb + i) * BN;
            if (SRC != kPagedE4m3 && valid < BN) {
                // rows behind the sequence's end: zeros (whole rows, so the swizzle does not matter)
                for (int x = valid * 8 + lane; x < BN * 8; x += 32)
#pragma unroll
                    for (int p = 0; p < C::PANELS; ++p) st_v4(s_ring + sv * C::SLOT + p * (BN * 128) + x * 16, 0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
            }
            const bool more = i + 1 < n;
            bool have_k = false;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!ok) break;
                if (jb + i < je[w]) {
                    if (!(ok = wait(&sh.p_full[w], i & 1, 6))) break;
                    tc_fence_after();
                    const uint64_t dv = desc_v(s_ring + sv * C::SLOT);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        mma_ts_w(tmem + T_O + 128 * w, tmem + 128 * w + 8 * kk, dv + 128 * kk, id_o, i > 0 || kk > 0);
                    mma_commit_w(smem_u32(&sh.pv_done[w]));
                }
                if (jb + i + 1 < je[w]) {
                    if (!have_k) {
                        if (!(ok = wait(&sh.full[sk], (ik / NS) & 1, 7))) break;
                        tc_fence_after();
                        have_k = true;
                    }
                    issue_s(w, sk);
                }
            }
            if (!ok) break;
            mma_commit_w(smem_u32(&sh.empty[sv]));
            if (more) mma_commit_w(smem_u32(&sh.empty[sk]));
        }
    } else if (SRC != kPagedE4m3) {
        // ------------------------------------------------------------ TMA loads
        if (warp == 9) {
            const int items = 2 * (jmax - jb);   // K_0 V_0 K_1 V_1 ...
            int issued = 0;
            for (; issued < items; ++issued) {
                const int slot = issued % NS, j0 = (jb + (issued >> 1)) * BN;
                if (issued >= NS && !wait(&sh.empty[slot], ((issued / NS) - 1) & 1, 8)) break;
                const CUtensorMap* tm = issued & 1 ? &tm_v : &tm_k;
                const uint32_t dst = s_ring + slot * C::SLOT, bar = smem_u32(&sh.full[slot]);
                if (SRC == kPacked) {
                    if (lane == 0) {
                        mbar_expect_tx(bar, C::SLOT);
                        const int tok = (int)(t.k0 + j0);
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_3d(dst + p * (BN * 128), tm, 64 * p, tok_first ? tok : hk, tok_first ? hk : tok, bar);
                    }
                } else {
                    // a box per page (two halves of a page of 256); no page or none left: zeros
                    const int box = min(a.c.page_size, BN), boxes = BN / box;
                    if (lane == 0) mbar_expect_tx(bar, C::SLOT);
                    __syncwarp();
                    if (lane < boxes) {
                        const int pos = j0 + lane * box;
                        int page = a.c.num_pages;   // out of range: the fill value
                        if (pos < t.nk) {
                            page = a.c.table[(int64_t)t.b * a.c.max_pages + (pos >> a.c.page_shift)];
                            if (page < 0 || page >= a.c.num_pages) page = a.c.num_pages;
                        }
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_4d(dst + p * (BN * 128) + lane * box * 128, tm, 64 * p, pos & (a.c.page_size - 1), hk, page, bar);
                    }
                }
                __syncwarp();
            }
            // no load may be in flight when the CTA's shared memory goes
            for (int i = max(0, issued - NS); i < issued; ++i) drain(&sh.full[i % NS], (i / NS) & 1, a.timeout);
        }
    } else {
        // ------------------------------------------------------------ 8-bit tiles widened to bf16
        const int ct = tid - 288;   // 0..95
        for (int it = 0; it < 2 * (jmax - jb); ++it) {
            const int slot = it % NS, j0 = (jb + (it >> 1)) * BN;
            if (it >= NS && !wait(&sh.empty[slot], ((it / NS) - 1) & 1, 9)) break;
            const char* src = it & 1 ? a.c.v : a.c.k;
            const uint8_t* sc = it & 1 ? a.c.vs : a.c.ks;
            const uint32_t dst = s_ring + slot * C::SLOT;
            constexpr int CH = D / 16;   // 16-code chunks of a row
#pragma unroll 4
            for (int x = ct; x < BN * CH; x += 96) {
                const int r = x / CH, c = x % CH;
                const int64_t row = j0 + r < t.nk ? cache_row(a.c, t.b, hk, j0 + r) : -1;
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                float f = 0.f;
                if (row >= 0) {
                    u = *reinterpret_cast<const uint4*>(src + row * D + c * 16);
                    f = scale_of(sc[row]);
                }
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 lo = e4m3x2_to_f((uint16_t)in[i]), hi = e4m3x2_to_f((uint16_t)(in[i] >> 16));
                    o[2 * i] = pack_bf16(lo.x * f, lo.y * f);
                    o[2 * i + 1] = pack_bf16(hi.x * f, hi.y * f);
                }
                st_v4(dst + tile_off(r, 2 * c), o[0], o[1], o[2], o[3]);
                st_v4(dst + tile_off(r, 2 * c + 1), o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async();
            mbar_arrive(smem_u32(&sh.full[slot]));
        }
      }
    }

    // MMAs in flight read shared memory and write TMEM: wait for the last ones before either goes
    __syncthreads();
    if (warp == 8) {
        mma_commit_w(smem_u32(&sh.s_full[0]));   // completes once every MMA issued so far has; the barrier has no waiter left
        const int used = max(0, je[0] - jb);
        if (sh.abort == 0) drain(&sh.s_full[0], used & 1, a.timeout);
        else for (long long t0 = clock64(); clock64() - t0 < 2000000;) {   // gave up: phases unknown, MMAs end by themselves
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

vdm_status encode(CUtensorMap* m, void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiled>(p) : (EncodeTiled) nullptr;
    }();
    if (!fn) return fail(VDM_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(VDM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return VDM_OK;
}

// [tokens][heads][D] with any strides: the dimension of the smaller stride first
vdm_status packed_map(CUtensorMap* m, const HeadView& h, int64_t T, int H, int D, bool tok_first) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)(tok_first ? T : H), (cuuint64_t)(tok_first ? H : T)};
    const cuuint64_t strides[2] = {(cuuint64_t)(tok_first ? h.st : h.sh), (cuuint64_t)(tok_first ? h.sh : h.st)};
    const cuuint32_t box[3] = {64, tok_first ? (cuuint32_t)BN : 1u, tok_first ? 1u : (cuuint32_t)BN};
    return encode(m, h.p, 3, dims, strides, box);
}

vdm_status paged_map(CUtensorMap* m, char* base, const CacheView& c) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page_size, (cuuint64_t)c.H, (cuuint64_t)c.num_pages};
    const cuuint64_t row = (cuuint64_t)c.D * 2;
    const cuuint64_t strides[3] = {row, row * c.page_size, row * c.page_size * c.H};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < BN ? c.page_size : BN), 1, 1};
    return encode(m, base, 4, dims, strides, box);
}

template <int D, int SRC>
vdm_status launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, bool tok_first, cudaStream_t s) {
    auto kern = attention_tc_kernel<D, SRC>;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), Cfg<D>::SMEM));
    const int64_t tiles = (a.Tq * a.G + (a.B < a.Tq ? a.B : a.Tq) * (int64_t)(2 * BM - 1)) / (2 * BM);
    kern<<<dim3((unsigned)tiles, a.Hk, a.splits), THREADS, Cfg<D>::SMEM, s>>>(mk, mv, a, tok_first);
    VDM_TRY(check_launch("attention_tc_kernel"));
    return a.splits > 1 ? launch_combine(a, VDM_BF16, s) : VDM_OK;
}

}  // namespace

vdm_status launch_attention_tc(const AttnArgs& a, cudaStream_t s) {
    // no keys at all: nothing to describe to the copy engine
    if (a.paged ? a.c.num_pages == 0 || a.c.max_pages == 0 : a.Tk == 0) return launch_attention_simt(a, VDM_BF16, s);
    CUtensorMap mk, mv;
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    if (a.paged && a.c.dtype == VDM_CACHE_E4M3)
        return a.D == 64 ? launch<64, kPagedE4m3>(mk, mv, a, false, s) : launch<128, kPagedE4m3>(mk, mv, a, false, s);
    if (a.paged) {
        VDM_TRY(paged_map(&mk, a.c.k, a.c));
        VDM_TRY(paged_map(&mv, a.c.v, a.c));
        return a.D == 64 ? launch<64, kPagedBf16>(mk, mv, a, false, s) : launch<128, kPagedBf16>(mk, mv, a, false, s);
    }
    const bool tf = a.k.st < a.k.sh;
    if (tf != (a.v.st < a.v.sh)) return launch_attention_simt(a, VDM_BF16, s);   // keys and values laid out differently
    VDM_TRY(packed_map(&mk, a.k, a.Tk, a.Hk, a.D, tf));
    VDM_TRY(packed_map(&mv, a.v, a.Tk, a.Hk, a.D, tf));
    return a.D == 64 ? launch<64, kPacked>(mk, mv, a, tf, s) : launch<128, kPacked>(mk, mv, a, tf, s);
}

}  // namespace vdm
