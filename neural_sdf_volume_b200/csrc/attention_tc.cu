// Attention on the 5th-generation tensor cores: bf16 queries with packed bf16, paged bf16 or
// paged 8-bit keys and values.
//
//   S = Q K^T (bf16 in, fp32 in TMEM) ; softmax with the running maximum m and sum l ;
//   O <- O + P V (P bf16 in TMEM, O fp32 in TMEM) ; out = O / l
//
// A CTA takes 256 query rows (D = 128) or 128 (D = 64, two CTAs on an SM) of one sequence and key
// head - a row is a token and a query head of the group, so that a group shares its keys' loads -
// as tiles of 128, and runs over the keys in tiles of 128.  Roles, with NT row tiles:
//   warps 0 .. 4 NT - 1  softmax, one row per thread: S from TMEM, maximum, 2^(scale log2e s - m),
//                        P as bf16 back into TMEM, sum in fp32; before and after the loop the
//                        tile's queries into shared memory and its rows out;
//   warp 4 NT            issues the MMAs of the tiles in turn: while one tile's softmax runs, the
//                        tensor cores work on the other's (D = 64: on the other CTA's);
//   warp 4 NT + 1        TMA loads of K and V tiles into a ring of slots (packed: one box of 128
//                        tokens per 64 columns; paged: one box per page);
//   warps 4 NT + 2, 3    masked values made finite, in the last key tiles of causal calls;
//   warps from 4 NT + 1  (8-bit cache) instead read codes from global memory, widen them to bf16 -
//                        exact: a code times a power of two - and write the ring's slots.
// The maximum that the exponents refer to follows the running maximum only when that has
// grown by more than 8 (log2 units): then O and l are rescaled, which needs the previous
// product to have finished; otherwise P stays below 2^8 and nothing is lost.  l sums the fp32
// exponentials; only the product uses their bf16 roundings.
//
// TMEM, D = 128 (512 columns): S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512); P_w overwrites the
// first 64 columns of S_w, so that a tile's next scores come after its product P V.
// D = 64 (256 columns): S [0,128) P [128,192) O [192,256), and the next scores are computed while the
// softmax of these runs.
//
// What bounds it (measured with clocks in the kernel, 128 x 128 scores): D = 64, the special-function unit: a
// tile takes 1024 cycles of its exponentials, two CTAs of an SM 2840 a step.  D = 128: the chain scores ->
// softmax -> P V -> next scores, 3390 cycles a step of two tiles, 2050 of them matrix products.
// Measured and not kept: a quarter of the exponentials by a polynomial on the FMA pipe (23 issue slots a
// pair against 16 cycles of the unit: 1 % at D = 64, a loss at 128); two threads per row; one S for both
// tiles, P apart (its users wait for one another: 3670 cycles); steps of 64 keys, S in two halves
// (a 128 x 64 x 16 MMA takes as long as a 128 x 128 x 16 one).
//
// Masked keys: a key that a row does not see has weight 0.  V rows behind the sequence's end
// are zeroed in shared memory (0 * NaN would reach every row).  V rows inside the sequence that
// not all rows of the CTA see lose their non-finite elements there, by the two warps that are idle otherwise (8-bit: while they
// are widened), and the rows that do see such an element get it at the end: see odd_only.
//
// Every wait is bounded; on expiry the kernel sets the error word, leaves NaN in the rows it could not finish, winds down and
// frees TMEM.
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

using namespace ptx;

constexpr int BM = 128, BN = 128;
enum Source : int { kPacked = 0, kPagedBf16 = 1, kPagedE4m3 = 2 };
constexpr float kLn2 = 0.69314718055994530942f;

template <int D> struct Cfg {
    static constexpr int PANELS = D / 64;
    static constexpr int NT = tc_rows(D) / BM;       // row tiles of a CTA
    static constexpr int PER_SM = NT == 1 ? 2 : 1;
    // warps that widen 8-bit tiles: a tile of D = 128 keeps seven busy
    static constexpr int WIDEN = NT == 1 ? 3 : 7;
    static constexpr int threads(int src) { return 128 * NT + (src == kPagedE4m3 ? 32 + 32 * WIDEN : 128); }
    // registers a thread, out of 128 at launch (two CTAs of 256 threads, one of 512) or 168 (one of 384); widening
    // warps want more (chunks at D = 64: 80 registers 330 us, 88 294, 96 298)
    static constexpr int regs_softmax(int src) { return threads(src) == 384 ? 208 : src != kPagedE4m3 ? 192 : NT == 1 ? 168 : 184; }
    static constexpr int regs_other(int src) { return threads(src) == 384 ? 88 : src != kPagedE4m3 ? 64 : NT == 1 ? 88 : 72; }
    static constexpr int QBYTES = BM * D * 2;        // one query tile
    static constexpr int SLOT = BN * D * 2;          // one key or value tile
    static constexpr int NS = D == 128 ? 5 : 6;      // slots beside the query tiles in 227 KB (113 KB)
    static constexpr int TILES = NT * QBYTES + NS * SLOT;
    static constexpr bool APART = NT == 1;           // P has columns of its own
    static constexpr bool EARLY = !APART;            // P V in two parts (372 us, in one 384, for 343 GFLOP of prompts)
    static constexpr uint32_t T_P = APART ? 128 : 0, T_O = APART ? 192 : 256, T_ALL = 256 * NT;   // tile w: 128 w further
};

// behind the tiles
template <int NT> struct Shared {
    uint64_t q_full, full[8], empty[8], s_full[NT], s_read[NT], p_half[NT], p_full[NT], pv_done[NT], look[8], clean[8];
    uint32_t tmem;
    int abort, odd;                      // odd: a value has been made finite
    int odd_hk, odd_b, odd_from, odd_to;   // then wanted: key head, sequence and keys that this may be true of
    long long odd_k0;
};
template <int D> constexpr int smem_bytes() { return Cfg<D>::TILES + (int)sizeof(Shared<Cfg<D>::NT>); }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 115712, "shared memory of an SM");

struct Wait {
    int* abort;
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
                if (*reinterpret_cast<volatile int*>(abort)) break;
                const long long t = clock64();
                if (t0 == 0) t0 = t;
                else if (t - t0 > timeout) {
                    *reinterpret_cast<volatile int*>(abort) = 1;
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

// one arrival for the warp, after what all its lanes did
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
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

__device__ __forceinline__ uint4 ld_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The non-finite values of keys [j0, j1), which the products left out, to a warp's rows (see odd_only): lane's row at `mine`, `parts` as
// float32, sees `seen` keys.  For each element the first key of each kind; then row by row.
template <typename TC, int D, bool PAGED>
__device__ __noinline__ void add_odd(const AttnArgs* a, int b, int64_t k0, int hk, int j0, int j1, char* mine, bool parts, int seen) {
    const int lane = threadIdx.x & 31;
    RowTile t;
    t.b = b, t.k0 = k0;
    const KvRows<TC, PAGED> kv{*a, t, hk};
    int up[4], down[4], nan[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) up[i] = down[i] = nan[i] = 0x7fffffff;
#pragma unroll 4
    for (int j = j1 - 1; j >= j0; --j) {
        const float4 v4 = 4 * lane < D ? kv.get(true, j, 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (v[i] == INFINITY) up[i] = j;
            if (v[i] == -INFINITY) down[i] = j;
            if (v[i] != v[i]) nan[i] = j;
        }
    }
    for (int r = 0; r < 32; ++r) {
        const int sees = __shfl_sync(0xffffffffu, seen, r);
        char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r));
        float add[4];
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            add[i] = (sees > up[i] ? INFINITY : 0.f) + (sees > down[i] ? -INFINITY : 0.f) + (sees > nan[i] ? NAN : 0.f);
            any = any || add[i] != 0.f;
        }
        if (any) {
            float* p32 = reinterpret_cast<float*>(dst) + 4 * lane;
            __nv_bfloat16* p16 = reinterpret_cast<__nv_bfloat16*>(dst) + 4 * lane;
            float4 x = parts ? load4f(p32) : load4f(p16);
            x = make_float4(x.x + add[0], x.y + add[1], x.z + add[2], x.w + add[3]);
            if (parts) store4(p32, x);
            else store4(p16, x);
        }
        __syncwarp();
    }
}

// A row that could not be finished: NaN, so that it is not taken for a result.
__device__ __noinline__ void give_up(const AttnArgs* a, int split, int64_t tok, int h) {
    const int64_t prow = ((int64_t)split * a->Tq + tok) * a->Hq + h;
    const bool parts = a->splits > 1;
    char* const row = parts ? reinterpret_cast<char*>(a->part_o + prow * a->D) : a->out.p + tok * a->out.st + h * a->out.sh;
    for (int i = 0; i < a->D * (parts ? 4 : 2); i += 16) *reinterpret_cast<uint4*>(row + i) = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (parts) a->part_lse[prow] = NAN;
    else if (a->lse) a->lse[tok * a->Hq + h] = NAN;
}

// What a widening thread has written of a value tile from row `from` on - chunks c and c + 1 of rows r0 + i ROWS - made finite;
// *any says that something was not.
template <int ROWS>
__device__ __noinline__ void make_finite(uint32_t tile, int r0, int c, int from, int* any) {
    bool odd = false;
    for (int r = r0; r < BN; r += ROWS) {
        if (r < from) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = tile + tile_off(r, c + i);
            uint4 v = ld_v4(at);
            if (!any_odd<false>(v)) continue;
            odd = true;
            v = without_odd<false>(v);
            st_v4(at, v.x, v.y, v.z, v.w);
        }
    }
    if (odd) *reinterpret_cast<volatile int*>(any) = 1;
}

template <int D, int SRC>
__global__ void __launch_bounds__(Cfg<D>::threads(SRC), Cfg<D>::PER_SM)
attention_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ AttnArgs a, const bool tok_first_k, const bool tok_first_v) {
    using C = Cfg<D>;
    constexpr int NS = C::NS, NT = C::NT, MMA_WARP = 4 * NT;
    constexpr int NPROD = SRC == kPagedE4m3 ? C::WIDEN : 1;   // arrivals that complete a slot
    extern __shared__ __align__(1024) uint8_t dyn_raw[];
    Shared<NT>& sh = *reinterpret_cast<Shared<NT>*>(dyn_raw + C::TILES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    RowTile t;
    const BlockPlace place = place_of<SRC != kPacked>(a);
    if (!find_tile(a, place.tile, NT * BM, a.causal, t)) return;
    const int hk = place.hk, split = place.split;
    const int total_rows = t.nq * a.G;
    const uint32_t base = smem_u32(dyn_raw);
    const uint32_t s_ring = base + NT * C::QBYTES;

    // key tiles of each row tile: [jb, je[w])
    int je[NT], jb, jmax = 0;
    {
        int most = 0;
#pragma unroll
        for (int w = 0; w < NT; ++w) {
            const int first = t.row0 + w * BM, last = min(first + BM, total_rows) - 1;
            je[w] = first < total_rows ? (keys_seen(a, t, last / a.G) + BN - 1) / BN : 0;
            most = max(most, je[w]);
        }
        const int per = (most + a.splits - 1) / a.splits;
        jb = split * per;
#pragma unroll
        for (int w = 0; w < NT; ++w) {
            je[w] = max(jb, min(je[w], jb + per));
            jmax = max(jmax, je[w]);
        }
    }
    // Keys that not all rows see: from `least` on.  From key tile jd on, tiles hold some (none: jd = jmax).
    const int least = min(keys_seen(a, t, t.row0 / a.G), t.nk), jd = least < t.nk ? max(jb, least / BN) : jmax;
    const Wait wait{&sh.abort, a.err, a.timeout};

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&sh.full[i]), NPROD);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            mbar_init(smem_u32(&sh.look[i]), 1);
            mbar_init(smem_u32(&sh.clean[i]), 2);
        }
        mbar_init(smem_u32(&sh.q_full), 4 * NT);
        for (int w = 0; w < NT; ++w) {
            mbar_init(smem_u32(&sh.s_full[w]), 1);
            mbar_init(smem_u32(&sh.s_read[w]), 4);
            mbar_init(smem_u32(&sh.p_half[w]), 4);
            mbar_init(smem_u32(&sh.p_full[w]), 4);
            mbar_init(smem_u32(&sh.pv_done[w]), 1);
        }
        sh.abort = sh.odd = 0;
        sh.odd_hk = hk, sh.odd_b = t.b, sh.odd_k0 = t.k0;
        sh.odd_from = max(least, jb * BN), sh.odd_to = min(jmax * BN, t.nk);
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(&sh.tmem), C::T_ALL);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp < MMA_WARP) {
        // ------------------------------------------------------------ softmax
        regs_up<C::regs_softmax(SRC)>();
        const int w = warp >> 2, trow = tid & 127, wrow = trow & ~31;   // tile, row of it, the warp's first
        const int row = t.row0 + w * BM + trow;
        const bool live = row < total_rows;
        const int64_t tok = t.q0 + (live ? row / a.G : 0);
        const int h = hk * a.G + (live ? row % a.G : 0);
        const int seen = live ? keys_seen(a, t, row / a.G) : 0;
        const int live_rows = min(32, total_rows - (row - lane));   // of the warp
        const uint32_t q_tile = base + w * C::QBYTES;
        constexpr int CPR = D / 8, RPI = 32 / CPR;   // 16-byte chunks of a row, rows of one instruction
        {
            // the warp's queries, a row's chunks on neighbouring lanes; rows beyond the last are zeros
            const char* mine = a.q.p + tok * a.q.st + (int64_t)h * a.q.sh;
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
                const int r = RPI * i + lane / CPR, c = lane % CPR;
                const char* src = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r));
                cp_async16(q_tile + tile_off(wrow + r, c), src + c * 16, r < live_rows);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async();
            warp_arrive(&sh.q_full);
        }
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128 * w + lanes, tp = ts + C::T_P, to = ts + C::T_O;
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
            if (C::APART) {   // the next scores may come
                tc_fence_before();
                warp_arrive(&sh.s_read[w]);
            }
            bool ended = j == jb;             // the previous product has
            const int left = seen - j * BN;   // keys of this tile that the row sees
            if (__any_sync(0xffffffffu, left < BN)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[c][i] = 32 * c + i < left ? s[c][i] : -INFINITY;
            }
            float mx[4];   // four chains of dependent maxima
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = fmax3(mx[c], s[c][i], s[c][i + 1]);
            const float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
            const float mn = fmaxf(m, mt);
            // raise the reference only when it has grown by more than 2^8 (or was -inf)
            const bool raise = (mn - m) * sc > 8.0f;
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise ? ex2((m - mn) * sc) : 1.0f;
                if (raise) m = mn;
                l *= f;
                if (!ended) {
                    if (!(ok = wait(&sh.pv_done[w], par ^ 1, 2))) break;
                    tc_fence_after();
                    ended = true;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        tmem_ld16(to + 16 * c, o);
                        tmem_wait_ld();
                        reg_fence16(o);
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * f);
                        tmem_st16(to + 16 * c, u);
                    }
                    tmem_wait_st();
                }
            }
            const float ref = m == -INFINITY ? 0.f : m * sc;
            const uint64_t sc2 = f32x2(sc, sc), ref2 = f32x2(-ref, -ref);
            uint64_t sum[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
            auto exps = [&](int c) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x0, x1;
                    f32x2_split(fma_f32x2(f32x2(s[c][2 * i], s[c][2 * i + 1]), sc2, ref2), x0, x1);
                    s[c][2 * i] = ex2(x0);
                    s[c][2 * i + 1] = ex2(x1);
                }
            };
            exps(0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c < 3) exps(c + 1);   // the next exponentials on their way before these are used
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum[i & 1] = add_f32x2(sum[i & 1], f32x2(s[c][2 * i], s[c][2 * i + 1]));
                    p[i] = pack_bf16(s[c][2 * i], s[c][2 * i + 1]);
                }
                if (C::APART && c == 0 && !ended) {   // the previous weights are still being read
                    if (!(ok = wait(&sh.pv_done[w], par ^ 1, 2))) break;
                    tc_fence_after();
                }
                tmem_st16(tp + 16 * c, p);
                if (C::EARLY && c == 1) {   // the product of the first 64 keys may start
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&sh.p_half[w]);
                }
            }
            if (!ok) break;
            float s0, s1;
            f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&sh.p_full[w]);
        }
        // ------------------------------------------------------------ output
        const int cnt = je[w] - jb;
        if (ok && cnt > 0) ok = wait(&sh.pv_done[w], (cnt - 1) & 1, 3);
        tc_fence_after();
        if (ok && live_rows > 0) {
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * sc) + log2f(l);
            const int64_t prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
            const bool parts = a.splits > 1;
            char* mine = parts ? reinterpret_cast<char*>(a.part_o + prow * D) : a.out.p + tok * a.out.st + h * a.out.sh;
            // The tile's queries are no longer read: their place takes the rows (as bf16, or half of each as
            // fp32), so that they leave with a row's chunks on neighbouring lanes.
            auto leave = [&](int bytes) {
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int r = RPI * i + lane / CPR, c = lane % CPR;
                    char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r));
                    const uint4 v = ld_v4(q_tile + tile_off(wrow + r, c));
                    if (r < live_rows) *reinterpret_cast<uint4*>(dst + bytes + c * 16) = v;
                }
                __syncwarp();
            };
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (cnt > 0) {
                    tmem_ld32(to + 32 * c, o);
                    tmem_wait_ld();
                    reg_fence(o);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
                if (parts) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_v4(q_tile + tile_off(trow, (8 * c + i) % CPR), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                              __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
                    if ((8 * c + 8) % CPR == 0) leave(((8 * c + 8) / CPR - 1) * CPR * 16);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_v4(q_tile + tile_off(trow, 4 * c + i), pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                              pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
                }
            }
            if (!parts) leave(0);
            if (live) {
                if (parts) a.part_lse[prow] = lse2;
                else if (a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
            }
            if (__builtin_expect(*reinterpret_cast<volatile int*>(&sh.odd), 0)) {
                __syncwarp();
                add_odd<typename std::conditional<SRC == kPagedE4m3, uint8_t, __nv_bfloat16>::type, D, SRC != kPacked>(
                    &a, sh.odd_b, sh.odd_k0, sh.odd_hk, sh.odd_from, sh.odd_to, mine, parts, live && l != 0.f ? seen : 0);
            }
        }
        if (!ok && live) give_up(&a, split, tok, h);
        tc_fence_before();
    } else {
      regs_down<C::regs_other(SRC)>();
      if (warp == MMA_WARP) {
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
            if (!a.withhold) mma_commit_w(smem_u32(&sh.s_full[w]));
        };
        auto issue_pv = [&](int w, int i, uint32_t slot) {
            if (!wait(C::EARLY ? &sh.p_half[w] : &sh.p_full[w], i & 1, 6)) return false;
            tc_fence_after();
            const uint64_t dv = desc_v(s_ring + slot * C::SLOT);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk) {
                if (C::EARLY && kk == BN / 32) {
                    if (!wait(&sh.p_full[w], i & 1, 6)) return false;
                    tc_fence_after();
                }
                mma_ts_w(tmem + C::T_O + 128 * w, tmem + C::T_P + 128 * w + 8 * kk, dv + 128 * kk, id_o, i > 0 || kk > 0);
            }
            mma_commit_w(smem_u32(&sh.pv_done[w]));
            return true;
        };
        bool ok = wait(&sh.q_full, 0, 12);
        if (ok && n > 0 && (ok = wait(&sh.full[0], 0, 4))) {
            tc_fence_after();
#pragma unroll
            for (int w = 0; w < NT; ++w)
                if (je[w] > jb) issue_s(w, 0);
            mma_commit_w(smem_u32(&sh.empty[0]));
        }
        uint32_t cleaned = 0;   // phases of `clean`
        for (int i = 0; ok && i < n; ++i) {
            const uint32_t iv = 2 * i + 1, ik = 2 * i + 2, sv = iv % NS, sk = ik % NS;
            const bool more = i + 1 < n;
            if (C::APART && more) {
                // the next scores, as soon as these have been read
                if (!(ok = wait(&sh.full[sk], (ik / NS) & 1, 7)) || !(ok = wait(&sh.s_read[0], i & 1, 10))) break;
                tc_fence_after();
                issue_s(0, sk);
                mma_commit_w(smem_u32(&sh.empty[sk]));
            }
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
            if (SRC != kPagedE4m3 && jb + i >= jd) {   // not all rows see all of the tile's keys
                if (!(ok = wait(&sh.clean[sv], (cleaned >> sv) & 1, 13))) break;
                cleaned ^= 1u << sv;
            }
            if (!C::APART && more) {
                if (!(ok = wait(&sh.full[sk], (ik / NS) & 1, 7))) break;
                tc_fence_after();
            }
#pragma unroll
            for (int w = 0; w < NT; ++w) {
                if (!ok) break;
                if (jb + i < je[w] && !(ok = issue_pv(w, i, sv))) break;
                if (!C::APART && jb + i + 1 < je[w]) issue_s(w, sk);
            }
            if (!ok) break;
            mma_commit_w(smem_u32(&sh.empty[sv]));
            if (!C::APART && more) mma_commit_w(smem_u32(&sh.empty[sk]));
        }
    } else if (SRC != kPagedE4m3) {
        // ------------------------------------------------------------ TMA loads
        if (warp == MMA_WARP + 1) {
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
                        const bool tok_first = issued & 1 ? tok_first_v : tok_first_k;
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
                if ((issued & 1) && jb + (issued >> 1) >= jd) warp_arrive(&sh.look[slot]);
                __syncwarp();
            }
            // no load may be in flight when the CTA's shared memory goes
            for (int i = max(0, issued - NS); i < issued; ++i) drain(&sh.full[i % NS], (i / NS) & 1, a.timeout);
        } else {
            // ---------------------------------------------------------- masked values made finite
            uint32_t looked = 0;   // phases of `look`
            for (int j = jd; j < jmax; ++j) {
                const int iv = 2 * (j - jb) + 1, sv = iv % NS;
                // The load warp says when the tile's load is under way: `full` then waits for that one's end.  The
                // slot's next load comes after the tile's product, and that after `clean`.
                if (!wait(&sh.look[sv], (looked >> sv) & 1, 14) || !wait(&sh.full[sv], (iv / NS) & 1, 15)) break;
                looked ^= 1u << sv;
                const int from = max(0, least - j * BN) * 8, to = min(BN, t.nk - j * BN) * 8;   // chunks of a panel; the swizzle stays in a row
                bool odd = false;
#pragma unroll 4
                for (int x = from + lane + 32 * (warp - MMA_WARP - 2); x < to; x += 64)
#pragma unroll
                    for (int p = 0; p < C::PANELS; ++p) {
                        const uint32_t at = s_ring + sv * C::SLOT + p * (BN * 128) + x * 16;
                        uint4 v = ld_v4(at);
                        if (any_odd<false>(v)) {
                            odd = true;
                            v = without_odd<false>(v);
                            st_v4(at, v.x, v.y, v.z, v.w);
                        }
                    }
                if (odd) *reinterpret_cast<volatile int*>(&sh.odd) = 1;
                fence_proxy_async();
                warp_arrive(&sh.clean[sv]);
            }
        }
    } else {
        // ------------------------------------------------------------ 8-bit tiles widened to bf16
        // A thread keeps one column of 16 codes and every ROWS-th row of a tile; the next tile's are asked for once
        // this one is announced, as the announcement's fence waits for loads too.  Pages are looked up a key tile
        // ahead, lane i those of its keys 16 i .. 16 i + 15, and rows once for keys and values.  Two chunks of up to 512
        // tokens over up to 15000, 32/8 heads: 313 us at D = 128 (bf16 pages 216), 300 at 64.  An earlier form with pages looked
        // up right before its loads, these before the announcement, took 384 and 504; codes by asynchronous copies through
        // shared memory 318 and 438.
        constexpr int CH = D / 16, ROWS = 32 * C::WIDEN / CH, U = (BN + ROWS - 1) / ROWS;
        const int ct = tid - 32 * (MMA_WARP + 1), c = ct % CH, r0 = ct / CH;
        const int items = 2 * (jmax - jb);
        const int32_t* table = a.c.table + (int64_t)t.b * a.c.max_pages;
        uint4 code[U];
        uint32_t scale[U];
        auto look_up = [&](int j) {
            const int key = j * BN + 16 * lane;
            return lane < BN / 16 && key < t.nk ? table[key >> a.c.page_shift] : -1;
        };
        int page = look_up(jb);
        int64_t row[U];   // of the key tile asked for, -1: none
        auto rows = [&](int j) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * ROWS, key = j * BN + r;
                const int p = __shfl_sync(0xffffffffu, page, r >> 4);   // lanes behind the tile's hold -1
                row[u] = key < t.nk && (uint32_t)p < (uint32_t)a.c.num_pages
                             ? (((int64_t)p * a.c.H + hk) << a.c.page_shift) + (key & (a.c.page_size - 1)) : -1;
            }
        };
        auto ask = [&](int it, int u) {
            code[u] = make_uint4(0u, 0u, 0u, 0u);
            scale[u] = 127;
            if (it < items && row[u] >= 0) {
                code[u] = *reinterpret_cast<const uint4*>((it & 1 ? a.c.v : a.c.k) + row[u] * D + c * 16);
                scale[u] = (it & 1 ? a.c.vs : a.c.ks)[row[u]];
            }
        };
        rows(jb);
#pragma unroll
        for (int u = 0; u < U; ++u) ask(0, u);
        for (int it = 0; it < items; ++it) {
            const int slot = it % NS;
            if (it >= NS && !wait(&sh.empty[slot], ((it / NS) - 1) & 1, 9)) break;
            const uint32_t dst = s_ring + slot * C::SLOT;
            if (!(it & 1)) page = look_up(jb + (it >> 1) + 1);
            else if (D == 128 && jb + (it >> 1) >= jd) {
                // values that not all rows see: finite, as codes (D = 128: 312 us, in the slot 358) or in the slot (D = 64: 319, as codes 350)
                bool odd = false;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if ((jb + (it >> 1)) * BN + r0 + u * ROWS < least) continue;
                    odd = odd || any_odd<true>(code[u]);
                    code[u] = without_odd<true>(code[u]);
                    scale[u] = min(scale[u], 246u);
                }
                if (odd) *reinterpret_cast<volatile int*>(&sh.odd) = 1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * ROWS;
                const uint32_t f = scale_bf16x2((uint8_t)scale[u]);
                const uint32_t in[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 lo = e4m3x2_to_f((uint16_t)in[i]), hi = e4m3x2_to_f((uint16_t)(in[i] >> 16));
                    o[2 * i] = mul_bf16x2(pack_bf16(lo.x, lo.y), f);
                    o[2 * i + 1] = mul_bf16x2(pack_bf16(hi.x, hi.y), f);
                }
                if (r < BN) {
                    st_v4(dst + tile_off(r, 2 * c), o[0], o[1], o[2], o[3]);
                    st_v4(dst + tile_off(r, 2 * c + 1), o[4], o[5], o[6], o[7]);
                }
            }
            if (it & 1) {
                rows(jb + (it >> 1) + 1);
                if (D == 64 && jb + (it >> 1) >= jd) make_finite<ROWS>(dst, r0, 2 * c, max(0, least - (jb + (it >> 1)) * BN), &sh.odd);
            }
            fence_proxy_async();
            warp_arrive(&sh.full[slot]);
#pragma unroll
            for (int u = 0; u < U; ++u) ask(it + 1, u);
        }
      }
    }

    // MMAs in flight read shared memory and write TMEM: wait for the last ones before either goes
    __syncthreads();
    if (warp == MMA_WARP) {
        mma_commit_w(smem_u32(&sh.s_full[0]));   // completes once every MMA issued so far has; the barrier has no waiter left
        const int used = max(0, je[0] - jb);
        if (sh.abort == 0) drain(&sh.s_full[0], used & 1, a.timeout);
        else for (long long t0 = clock64(); clock64() - t0 < 2000000;) {   // gave up: phases unknown, MMAs end by themselves
        }
        tc_fence_after();
        tmem_dealloc(tmem, C::T_ALL);
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
vdm_status launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, bool tok_first_k, bool tok_first_v, cudaStream_t s) {
    auto kern = attention_tc_kernel<D, SRC>;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), smem_bytes<D>()));
    const int64_t tiles = row_tiles(a.Tq, a.G, a.B, tc_rows(D));
    kern<<<tile_grid(a, tiles), Cfg<D>::threads(SRC), smem_bytes<D>(), s>>>(mk, mv, a, tok_first_k, tok_first_v);
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
        return a.D == 64 ? launch<64, kPagedE4m3>(mk, mv, a, false, false, s) : launch<128, kPagedE4m3>(mk, mv, a, false, false, s);
    if (a.paged) {
        VDM_TRY(paged_map(&mk, a.c.k, a.c));
        VDM_TRY(paged_map(&mv, a.c.v, a.c));
        return a.D == 64 ? launch<64, kPagedBf16>(mk, mv, a, false, false, s) : launch<128, kPagedBf16>(mk, mv, a, false, false, s);
    }
    const bool tk = a.k.st < a.k.sh, tv = a.v.st < a.v.sh;   // each in its own order
    VDM_TRY(packed_map(&mk, a.k, a.Tk, a.Hk, a.D, tk));
    VDM_TRY(packed_map(&mv, a.v, a.Tk, a.Hk, a.D, tv));
    return a.D == 64 ? launch<64, kPacked>(mk, mv, a, tk, tv, s) : launch<128, kPacked>(mk, mv, a, tk, tv, s);
}

}  // namespace vdm
