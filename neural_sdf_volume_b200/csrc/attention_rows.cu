// Attention of few query rows to many keys (single tokens, short chunks): bf16 queries over
// packed or paged bf16 or paged 8-bit keys and values.  Bound by memory: every key and value is
// read once per 16 rows, and nothing else of size is moved.
//
// A row is (token, query head of the group); a tile is up to 16 rows of one sequence and key
// head.  The tile's keys are shared out over the warps of a cluster of blocks (and, beyond
// 16 blocks, over grid z with partial results in the workspace): warp w takes steps w, w + n, ...
// of KS keys.  Each warp keeps a ring of steps in shared memory of its own, filled by 16-byte
// asynchronous copies (no barrier between warps until the end), and runs the softmax's running
// maximum and sum on its keys alone:
//   S = Q K^T    mma.sync m16n8k16, rows of the tile as M, keys as N.  A contraction's order is
//                free, so lane t of a key's four takes 16 contiguous bytes of it and Q is laid out
//                to match: K goes from shared memory into fragments without a transposition.
//   O += P V     P's fragments are S's accumulators; lane g takes 16 contiguous bytes (as columns
//                of O) of the four rows it needs, paired by byte permutations.
// mma.sync, not tcgen05: with 1 to 16 rows the tensor work is 1/8 of a tile's and hidden behind the
// loads, and operands in registers skip the staging that widening 8-bit codes in shared memory
// would take.
//
// 8-bit codes are widened to fp16 (exact).  Q is scaled per row by a power of two so that
// its largest element is in [2^14, 2^15): what of a bf16 row fp16 cannot hold lies below 2^-38 of
// that.  A key's scale goes into its score.  A value's scale 2^e goes into the exponent of its weight,
// w = 2^(s + e - M), with M the running maximum of s + e, and l sums w 2^-e: a row's largest product
// w v sets the reference whatever the scales of its keys are.  w is rounded to fp16 at 2^12 times
// its value: its relative precision is 2^-12 down to w = 2^-26, below that an error of 2^-37.
// bf16 values: e = 0 and w is rounded to bf16.
// The reference follows the maximum when that has grown by more than 2^3.
//
// Masked keys: rows of V behind the sequence's end are read as zeros.  Rows inside it that
// only later queries of the tile see can bring 0 * NaN; see repair_row.
#include <type_traits>

#include "seq_internal.cuh"
#include "tc_ptx.cuh"

namespace vdm {
namespace {

using namespace ptx;

constexpr int RM = 16;   // rows of a tile
constexpr int RW = 4;    // warps of a block
enum Source : int { kPacked = 0, kPagedBf16 = 1, kPagedE4m3 = 2 };
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int SRC> struct Cfg {
    static constexpr bool E8 = SRC == kPagedE4m3;
    static constexpr int RB = E8 ? D : 2 * D;               // bytes of a row
    static constexpr int KS = RB > 128 ? 16 : 32;           // keys of a step
    static constexpr int STAGE = 2 * KS * RB + (E8 ? 2 * KS : 0);
    static constexpr int NS = RB > 64 ? 3 : 4;              // steps in a warp's ring
    static constexpr int PART = RM * D * 4;                 // a warp's O, in its ring at the end
    static constexpr int WARP = NS * STAGE > PART ? NS * STAGE : PART;
    static constexpr int SMEM = RW * WARP;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
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

// D += A B, 16 x 8 x 16: fp16 or bf16 in, fp32 out
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 codes (low or high half of w) as fp16
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(HI ? w >> 16 : w & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ROWS8: tiles have at most 8 rows, the other half of the matrix product's rows stays empty
template <int D, int SRC, bool ROWS8>
__global__ void __launch_bounds__(RW * 32) attention_rows_kernel(const __grid_constant__ AttnArgs a, const int cluster) {
    using C = Cfg<D, SRC>;
    constexpr bool E8 = C::E8, PAGED = SRC != kPacked;
    constexpr int RB = C::RB, KS = C::KS, NS = C::NS, CH = RB / 16;   // CH: 16-byte chunks of a row
    constexpr int NR = ROWS8 ? 1 : 2;                                 // rows of a lane: g and g + 8
    constexpr int EC = E8 ? 16 : 8;                                   // elements of a chunk
    constexpr int KK = D / 16, NT = D / 8;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ float s_m[RW][RM], s_l[RW][RM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    RowTile t;
    if (!find_tile(a, blockIdx.x, ROWS8 ? 8 : RM, a.causal, t)) return;   // the whole cluster alike
    const int hk = blockIdx.y, rank = blockIdx.z % cluster, split = blockIdx.z / cluster;
    const int n_rows = min(ROWS8 ? 8 : RM, t.nq * a.G - t.row0);

    // keys of the tile: steps [s0, s1) of this split
    const int most = keys_seen(a, t, (t.row0 + n_rows - 1) / a.G);
    const int n_steps = (most + KS - 1) / KS, per = (n_steps + a.splits - 1) / a.splits;
    const int s0 = min(n_steps, split * per), s1 = min(n_steps, s0 + per);
    const int first = s0 + rank * RW + warp, stride = cluster * RW;

    const uint32_t ring = smem_u32(dyn) + warp * C::WARP;
    constexpr int U = KS / 16;   // a page holds whole blocks of 16 keys
    auto pages_of = [&](int step, int (&pg)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            pg[u] = -1;
            const int pos = step * KS + 16 * u;
            if (PAGED && step < s1 && pos < t.nk) pg[u] = a.c.table[(int64_t)t.b * a.c.max_pages + (pos >> a.c.page_shift)];
        }
    };
    auto issue = [&](int step, int slot, const int (&pg)[U]) {
        if (step < s1) {
            const uint32_t dk = ring + slot * C::STAGE, dv = dk + KS * RB;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pos0 = step * KS + 16 * u;
                const char *sk, *sv;
                int64_t st, row0 = 0;
                bool on = true;
                if (PAGED) {
                    on = pg[u] >= 0 && pg[u] < a.c.num_pages;
                    row0 = on ? (((int64_t)pg[u] * a.c.H + hk) << a.c.page_shift) + (pos0 & (a.c.page_size - 1)) : 0;
                    sk = a.c.k + row0 * RB, sv = a.c.v + row0 * RB, st = RB;
                } else {
                    sk = a.k.p + (t.k0 + pos0) * a.k.st + hk * a.k.sh;
                    sv = a.v.p + (t.k0 + pos0) * a.v.st + hk * a.v.sh;
                    st = 0;
                }
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) {
                    const int x = lane + 32 * i, r = x / CH, c = x % CH;
                    const bool ok = on && pos0 + r < t.nk;
                    const uint32_t pk = CH > 4 ? c ^ ((r & 1) << 2) : c;
                    const uint32_t pv = CH > 4 ? c ^ (((r >> 1) & 3) << 1) : c ^ (((r >> 1) & 1) << 1);
                    const int64_t ok_r = ok ? r : 0;   // an address inside the tensors also where nothing is read
                    const char* ak = PAGED ? sk + ok_r * st : (ok ? sk + r * a.k.st : a.k.p);
                    const char* av = PAGED ? sv + ok_r * st : (ok ? sv + r * a.v.st : a.v.p);
                    cp16(dk + (16 * u + r) * RB + pk * 16, ak + (ok ? c * 16 : 0), ok);
                    cp16(dv + (16 * u + r) * RB + pv * 16, av + (ok ? c * 16 : 0), ok);
                }
                if (E8 && lane < 2) cp16(dk + 2 * KS * RB + lane * KS + 16 * u, (lane ? a.c.vs : a.c.ks) + row0, on);
            }
        }
        cp_async_commit();
    };
    int pg[U];
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
        pages_of(first + s * stride, pg);
        issue(first + s * stride, s, pg);
    }
    pages_of(first + (NS - 1) * stride, pg);

    // queries as fragments: element pair i of k-step kk of lane t4 is d = 16-byte chunk
    // (t4 + 4 h) of the row, elements 4 i + {0, 1} and {2, 3}
    uint32_t qa[KK][NR][2];
    float rs[NR];       // factor of the row's scores: softmax scale, log2 e and 2^(Q's exponent)
    int seen[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = g + 8 * r;
        const bool on = row < n_rows;
        const int rr = t.row0 + (on ? row : 0);
        seen[r] = on ? keys_seen(a, t, rr / a.G) : 0;
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q.p + (t.q0 + rr / a.G) * a.q.st +
                                                                        (int64_t)(hk * a.G + rr % a.G) * a.q.sh);
        float mul = 1.0f;
        rs[r] = a.scale_log2;
        if (E8) {
            float mx = 0.f;
            if (on)
                for (int i = t4 * (D / 4); i < (t4 + 1) * (D / 4); i += 4) {
                    const float4 x = load4f(q + i);
                    mx = fmax3(fmax3(mx, fabsf(x.x), fabsf(x.y)), fabsf(x.z), fabsf(x.w));
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // exponent e of the maximum (2^e <= mx < 2^(e+1)); Q' = Q 2^(14 - e)
            const int e = mx > 0.f ? (int)(__float_as_uint(mx) >> 23) - 127 : 14, up = min(14 - e, 120);
            mul = pow2i(up);
            rs[r] = a.scale_log2 * pow2i(-up);
        }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int h = kk / (EC / 4), i = kk % (EC / 4), d = (t4 + 4 * h) * EC + 4 * i;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on) x = load4f(q + d);
            if (E8) {
                qa[kk][r][0] = pack_f16(x.x * mul, x.y * mul);
                qa[kk][r][1] = pack_f16(x.z * mul, x.w * mul);
            } else {
                qa[kk][r][0] = pack_bf16(x.x, x.y);
                qa[kk][r][1] = pack_bf16(x.z, x.w);
            }
        }
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) m[r] = -INFINITY, l[r] = 0.f;
    constexpr float W0 = E8 ? 12.0f : 0.0f;   // fp16 weights are kept at 2^12 times their value

    int slot = 0, fill = NS - 1;
    for (int step = first; step < s1; step += stride) {
        issue(step + (NS - 1) * stride, fill, pg);
        pages_of(step + NS * stride, pg);
        fill = fill + 1 == NS ? 0 : fill + 1;
        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t bk = ring + slot * C::STAGE, bv = bk + KS * RB;
        slot = slot + 1 == NS ? 0 : slot + 1;

        float s[KS / 8][4];
#pragma unroll
        for (int n = 0; n < KS / 8; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            const int r = 8 * n + g;
#pragma unroll
            for (int h = 0; h < CH / 4; ++h) {
                const int c = t4 + 4 * h;
                const uint4 w = lds128(bk + r * RB + (CH > 4 ? c ^ ((r & 1) << 2) : c) * 16);
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < EC / 4; ++i) {
                    const int kk = h * (EC / 4) + i;
                    const uint32_t b0 = E8 ? widen<false>(x[i]) : x[2 * i % 4], b1 = E8 ? widen<true>(x[i]) : x[(2 * i + 1) % 4];
                    mma16816<E8>(s[n], qa[kk][0][0], ROWS8 ? 0u : qa[kk][NR - 1][0], qa[kk][0][1], ROWS8 ? 0u : qa[kk][NR - 1][1], b0, b1);
                }
            }
        }
        // scores in log2 units, with the value scale's exponent added
        float inv[KS / 8][2];   // 2^-e of the keys
        float mx[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) mx[r] = -INFINITY;
#pragma unroll
        for (int n = 0; n < KS / 8; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int key = 8 * n + 2 * t4 + j;
                float f = 1.0f, ev = 0.0f;
                if (E8) {
                    f = scale_of((uint8_t)lds_u8(bk + 2 * KS * RB + key));
                    const int vb = (int)lds_u8(bk + 2 * KS * RB + KS + key);
                    ev = (float)(vb - 127);
                    // 2^(127 - vb); vb up to 246 from vdm_cache_write, beyond 253 the sum loses denormals
                    inv[n][j] = __uint_as_float((uint32_t)max(1, 254 - vb) << 23);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float& x = s[n][2 * r + j];
                    x = E8 ? fmaf(x, rs[r] * f, ev) : x * rs[r];
                    if (step * KS + key >= seen[r]) x = -INFINITY;
                    mx[r] = fmaxf(mx[r], x);
                }
            }
        bool raise = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            raise = raise || mx[r] > m[r] + 3.0f;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float mn = fmaxf(m[r], mx[r]);
                const float f = mn == -INFINITY ? 1.0f : exp2f(m[r] - mn);
                m[r] = mn;
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < NT; ++i) o[i][2 * r] *= f, o[i][2 * r + 1] *= f;
            }
        }
        uint32_t p[KS / 8][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float ref = (m[r] == -INFINITY ? 0.f : m[r]) - W0;
#pragma unroll
            for (int n = 0; n < KS / 8; ++n) {
                const float w0 = ex2(s[n][2 * r] - ref), w1 = ex2(s[n][2 * r + 1] - ref);
                if (E8) l[r] = fmaf(w0, inv[n][0], fmaf(w1, inv[n][1], l[r]));
                else l[r] += w0 + w1;
                p[n][r] = E8 ? pack_f16(w0, w1) : pack_bf16(w0, w1);
            }
        }
#pragma unroll
        for (int kg = 0; kg < KS / 16; ++kg) {
            const uint32_t a0 = p[2 * kg][0], a1 = ROWS8 ? 0u : p[2 * kg][NR - 1], a2 = p[2 * kg + 1][0], a3 = ROWS8 ? 0u : p[2 * kg + 1][NR - 1];
            const uint32_t rows = bv + (16 * kg + 2 * t4) * RB;   // this lane's rows: +0, +1, +8, +9
            if (E8 && D == 64) {
                // 8 bytes of each row: half of chunk g / 2
                const uint32_t off = (uint32_t)(((g >> 1) ^ ((t4 & 1) << 1)) * 16 + (g & 1) * 8);
                const uint2 x0 = lds64(rows + off), x1 = lds64(rows + RB + off), y0 = lds64(rows + 8 * RB + off), y1 = lds64(rows + 9 * RB + off);
                const uint32_t X0[2] = {x0.x, x0.y}, X1[2] = {x1.x, x1.y}, Y0[2] = {y0.x, y0.y}, Y1[2] = {y1.x, y1.y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t u0 = __byte_perm(X0[i], X1[i], 0x5140), u1 = __byte_perm(X0[i], X1[i], 0x7362);
                    const uint32_t v0 = __byte_perm(Y0[i], Y1[i], 0x5140), v1 = __byte_perm(Y0[i], Y1[i], 0x7362);
                    mma16816<E8>(o[(4 * i) % NT], a0, a1, a2, a3, widen<false>(u0), widen<false>(v0));
                    mma16816<E8>(o[(4 * i + 1) % NT], a0, a1, a2, a3, widen<true>(u0), widen<true>(v0));
                    mma16816<E8>(o[(4 * i + 2) % NT], a0, a1, a2, a3, widen<false>(u1), widen<false>(v1));
                    mma16816<E8>(o[(4 * i + 3) % NT], a0, a1, a2, a3, widen<true>(u1), widen<true>(v1));
                }
            } else {
#pragma unroll
                for (int h = 0; h < CH / 8; ++h) {
                    const uint32_t off = (uint32_t)((g ^ (t4 << 1)) + 8 * h) * 16;   // rows 2 t4 + {0, 1, 8, 9}: (r / 2) % 4 = t4
                    const uint4 x0 = lds128(rows + off), x1 = lds128(rows + RB + off), y0 = lds128(rows + 8 * RB + off),
                                y1 = lds128(rows + 9 * RB + off);
                    const uint32_t X0[4] = {x0.x, x0.y, x0.z, x0.w}, X1[4] = {x1.x, x1.y, x1.z, x1.w}, Y0[4] = {y0.x, y0.y, y0.z, y0.w},
                                   Y1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (E8) {
                            const uint32_t u0 = __byte_perm(X0[i], X1[i], 0x5140), u1 = __byte_perm(X0[i], X1[i], 0x7362);
                            const uint32_t v0 = __byte_perm(Y0[i], Y1[i], 0x5140), v1 = __byte_perm(Y0[i], Y1[i], 0x7362);
                            mma16816<E8>(o[(4 * i) % NT], a0, a1, a2, a3, widen<false>(u0), widen<false>(v0));
                            mma16816<E8>(o[(4 * i + 1) % NT], a0, a1, a2, a3, widen<true>(u0), widen<true>(v0));
                            mma16816<E8>(o[(4 * i + 2) % NT], a0, a1, a2, a3, widen<false>(u1), widen<false>(v1));
                            mma16816<E8>(o[(4 * i + 3) % NT], a0, a1, a2, a3, widen<true>(u1), widen<true>(v1));
                        } else {
                            const int n = 8 * h + 2 * i;
                            mma16816<E8>(o[n % NT], a0, a1, a2, a3, __byte_perm(X0[i], X1[i], 0x5410), __byte_perm(Y0[i], Y1[i], 0x5410));
                            mma16816<E8>(o[(n + 1) % NT], a0, a1, a2, a3, __byte_perm(X0[i], X1[i], 0x7632), __byte_perm(Y0[i], Y1[i], 0x7632));
                        }
                    }
                }
            }
        }
        __syncwarp();   // the next copy into this slot comes after every lane's reads
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warp's rows into its ring, column n-tile i, lane column j: element of the row
    const float w0 = exp2f(-W0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        l[r] *= w0;
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t4 == 0) s_m[warp][g + 8 * r] = m[r], s_l[warp][g + 8 * r] = l[r];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2 * NR; ++e) {
            // column j = 2 t4 + (e & 1) of n-tile i: the dimensions that lane group g = j loaded as i
            const int row = g + 8 * (e >> 1), j = 2 * t4 + (e & 1);
            const int d = E8 ? j * (D / 8) + i : (i / 8) * 64 + j * 8 + i % 8;
            const float x = o[i][e] * w0;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + (row * D + d) * 4), "f"(x) : "memory");
        }
    if (cluster > 1) cluster_sync();
    else __syncthreads();

    // joining: a warp of the cluster per row, parts in order
    for (int row = rank * RW + warp; row < n_rows; row += cluster * RW) {
        float M = -INFINITY;
        for (int k = 0; k < cluster; ++k)
            for (int w = 0; w < RW; ++w) M = fmaxf(M, ld_cluster_f32(mapa(smem_u32(&s_m[w][row]), k)));
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool on = 4 * lane < D;
        for (int k = 0; k < cluster; ++k)
            for (int w = 0; w < RW; ++w) {
                const float pm = ld_cluster_f32(mapa(smem_u32(&s_m[w][row]), k)), pl = ld_cluster_f32(mapa(smem_u32(&s_l[w][row]), k));
                if (pm == -INFINITY && pl == 0.f) continue;   // no key
                const float f = exp2f(pm - ref);
                L = fmaf(f, pl, L);
                if (on) {
                    const float4 y = ld_cluster_f4(mapa(smem_u32(dyn) + w * C::WARP + (row * D + 4 * lane) * 4, k));
                    x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
                }
            }
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        float lse2 = L == 0.f ? -INFINITY : ref + log2f(L);
        const int rr = t.row0 + row, see = keys_seen(a, t, rr / a.G);
        const bool bad = !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY && fabsf(x.w) < INFINITY);
        const int end = min(s1 * KS, most);
        if (see < end && __any_sync(0xffffffffu, bad))
            lse2 = repair_row<typename std::conditional<E8, uint8_t, __nv_bfloat16>::type, D, PAGED>(a, t, hk, rr, s0 * KS, min(see, end), x);
        const int64_t tok = t.q0 + rr / a.G;
        const int h = hk * a.G + rr % a.G;
        if (a.splits > 1) {
            const int64_t prow = ((int64_t)split * a.Tq + tok) * a.Hq + h;
            if (on) store4(a.part_o + prow * D + 4 * lane, x);
            if (lane == 0) a.part_lse[prow] = lse2;
        } else {
            if (on) store4(reinterpret_cast<__nv_bfloat16*>(a.out.p + tok * a.out.st + h * a.out.sh) + 4 * lane, x);
            if (lane == 0 && a.lse) a.lse[tok * a.Hq + h] = lse2 * kLn2;
        }
    }
    if (cluster > 1) cluster_sync();   // no block leaves while another reads its shared memory
}

template <int D, int SRC, bool ROWS8>
vdm_status launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = attention_rows_kernel<D, SRC, ROWS8>;
    constexpr int M = ROWS8 ? 8 : RM;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), Cfg<D, SRC>::SMEM, true));
    const int64_t tiles = (a.Tq * a.G + (a.B < a.Tq ? a.B : a.Tq) * (int64_t)(M - 1)) / M;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles, a.Hk, a.splits * a.cluster);
    cfg.blockDim = dim3(RW * 32);
    cfg.dynamicSmemBytes = Cfg<D, SRC>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 1, at.val.clusterDim.y = 1, at.val.clusterDim.z = a.cluster;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    VDM_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, a, a.cluster));
    VDM_TRY(check_launch("attention_rows_kernel"));
    return a.splits > 1 ? launch_combine(a, VDM_BF16, s) : VDM_OK;
}

template <int SRC>
vdm_status launch_d(const AttnArgs& a, cudaStream_t s) {
    const bool r8 = rows_tile(a.G, a.Tq, a.B) == 8;
    if (a.D == 64) return r8 ? launch<64, SRC, true>(a, s) : launch<64, SRC, false>(a, s);
    return r8 ? launch<128, SRC, true>(a, s) : launch<128, SRC, false>(a, s);
}

}  // namespace

vdm_status launch_attention_rows(const AttnArgs& a, cudaStream_t s) {
    if (a.paged ? a.c.num_pages == 0 || a.c.max_pages == 0 : a.Tk == 0) return launch_attention_simt(a, VDM_BF16, s);   // no keys at all
    if (!a.paged) return launch_d<kPacked>(a, s);
    return a.c.dtype == VDM_CACHE_E4M3 ? launch_d<kPagedE4m3>(a, s) : launch_d<kPagedBf16>(a, s);
}

}  // namespace vdm
