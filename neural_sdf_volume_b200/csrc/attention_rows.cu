// Attention of few query rows to many keys (single tokens, short chunks): bf16 queries over
// packed or paged bf16 or paged 8-bit keys and values.  Bound by memory: every key and value is
// read once per 16 rows, and nothing else of size is moved.
//
// A row is (token, query head of the group); a tile is up to 16 rows of one sequence and key
// head.  The tile's keys are shared out over the warps of a cluster of blocks (and, beyond
// eight blocks, over grid z with partial results in the workspace): warp w takes steps w, w + n, ...
// of KS keys.  Each warp keeps a ring of steps in shared memory of its own, filled by 16-byte
// asynchronous copies (no barrier between warps until the end), and runs the softmax's running
// maximum and sum on its keys alone:
//   S^T = K Q^T    mma.sync m16n8k16, 16 keys as M and 8 rows of the tile as N.  A contraction's
//                  order is free, so lane t of a key's four takes 16 contiguous bytes of it and Q is
//                  laid out to match: K goes from shared memory into fragments without a transposition.
//   O^T += V^T P^T the weights' 8 x 8 blocks are transposed in registers (movmatrix); lane g takes 16
//                  contiguous bytes (dimensions, as M) of the four keys it needs, paired by byte
//                  permutations.
// mma.sync, not tcgen05: with 1 to 16 rows the tensor work is 1/8 of a tile's and hidden behind the
// loads, and operands in registers skip the staging that widening 8-bit codes in shared memory
// would take.
//
// 8-bit codes are widened to fp16 (exact).  Q is scaled per row by a power of two so that
// its largest element is in [2^14, 2^15): what of a bf16 row fp16 cannot hold lies below 2^-38 of
// that.  A key's scale goes into its score.  A value's scale 2^e goes into the exponent of its weight,
// w = 2^(s + e - M), with M the running maximum of s + e: a row's largest product w v sets the
// reference of the product whatever the scales of its keys are; a value row of zeros has no
// product, so that its e (0, as written) must not set M and counts as -100.  w is rounded to fp16 at 2^12 times
// its value: off by 2^-11 of itself at most down to w = 2^-26, below that by 2^-37.
// The sum l has nothing to do with the values: it adds 2^(s - R), with R a reference of the scores.  While all value
// exponents are within 24 of one E0, R = M - E0 - 12 and a term is w 2^(E0 - e); what is lost where w flushes to zero
// lies below 2^-42 of the largest term.  A step with other exponents computes its terms from the scores, against an R of
// their own (M and R may lie 219 apart, more than float32's exponents hold below one reference), and takes its largest
// e as E0; while R stays more than 60 from M - E0 - 12, so do the steps after it.  Against a sum of w 2^-e alone, which lost
// keys 138 below M, this costs 2 to 5 % (a second exponential in every step 8 to 34 %).
// bf16 values: e = 0 and w is rounded to bf16.
// The reference follows the maximum when that has grown by more than 2^3.
//
// Masked keys: rows of V that no row of the tile sees are read as zeros.  Rows that
// only its later queries see lose their non-finite elements in shared memory; see odd_only.
//
// Measured: 48 sequences of 300 to 16000 tokens, one query token each, 32/8 heads of 128, 8-bit (801 MB): 146 us,
// 5.5 TB/s, 84 % of the copy rate; with queries as M and keys as N, half of each product empty, and the keys'
// scales unpacked by every lane, 239 us.  One sequence of 700 tokens, 8 heads of 64: 6.2 us, which is loads that wait
// for one another (offsets, page, keys: 1.1 + 1.0 + 0.7 us) and 2.1 us of joining.
#include <type_traits>

#include "attention_join.cuh"

namespace vdm {
namespace {

using namespace ptx;

enum Source : int { kPacked = 0, kPagedBf16 = 1, kPagedE4m3 = 2 };

template <int D, int SRC> struct Cfg {
    static constexpr bool E8 = SRC == kPagedE4m3;
    static constexpr int RB = E8 ? D : 2 * D;               // bytes of a row
    static constexpr int KS = RB > 128 ? 16 : 32;           // keys of a step
    static constexpr int STAGE = 2 * KS * RB + (E8 ? 2 * KS : 0);
    static constexpr int NS = RB > 64 ? 2 : 4;              // steps in a warp's ring
    static constexpr int PART = RM * D * 4;                 // a warp's O, in its ring at the end
    static constexpr int WARP = NS * STAGE > PART ? NS * STAGE : PART;
    static constexpr int SMEM = RW * WARP;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int W>
__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&v)[W]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2 % W]), "=r"(v[3 % W]) : "r"(a));
}
template <int W>
__device__ __forceinline__ void lds64(uint32_t a, uint32_t (&v)[W]) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
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
// an 8 x 8 block of 16-bit elements transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// four e4m3 codes as two pairs of fp16
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Where chunk c of row r lies in a step's rows.  Keys: the eight lanes of a quarter of a 16-byte load
// read four neighbouring chunks of two rows; values: two chunks of the rows 0, 2, 4, 6.
template <int CH>
__device__ __forceinline__ int swizzle_k(int r, int c) { return CH > 4 ? c ^ ((r & 1) << 2) : c; }
template <int CH>
__device__ __forceinline__ int swizzle_v(int r, int c) { return CH > 4 ? c ^ (((r >> 1) & 3) << 1) : c ^ (((r >> 1) & 1) << 1); }

constexpr float kW0 = 12.0f;   // 8-bit values: fp16 weights are kept at 2^12 times their value, and sums against M - E0 - 12
constexpr int kNear = 24;      // how far from E0 a step's value exponents may lie

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float over_keys(float x) {   // a row's keys are on the lanes of the same t4
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// Non-finite elements of the value rows [r0, r1) of a step become zeros; *s_odd says that there were some.  Out of line, as what follows: few
// calls meet it, and the others' loop is shorter without.
template <bool E8, int CH>
__device__ __noinline__ void make_finite(uint32_t bv, int r0, int r1, int* s_odd) {
    bool odd = false;
#pragma unroll 1
    for (int x = r0 * CH + (threadIdx.x & 31); x < r1 * CH; x += 32) {
        uint4 v = lds128(bv + x * 16);
        if (!any_odd<E8>(v)) continue;
        odd = true;
        v = without_odd<E8>(v);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(bv + x * 16), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
    if (odd) *s_odd = 1;
    __syncwarp();
}

// The sum's terms of a step whose value exponents are not all near E0, or one of whose value rows is zeros: from the
// scores, against their own reference R.
template <int NQ> struct Apart {
    float s[4][NQ][2];               // score + value exponent of the lane's keys 8 k + g; zero rows': with -100 for 0 when done
    float m[NQ][2], l[NQ][2], mx[NQ][2];
    float ev;                        // of the key `lane`, and whether its value row is zeros
    bool none;
    int e0;
    bool far;
};
template <int NQ>
__device__ __noinline__ void sum_apart(Apart<NQ>& x, float (&s_r)[RM]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const float now = x.none ? -100.0f : x.ev, was = (float)(x.e0 - 127);
    const uint32_t top_e = __reduce_max_sync(0xffffffffu, x.none ? 0u : (uint32_t)(x.ev + 127.0f));
    if (top_e) x.e0 = (int)top_e;
    float R[NQ][2], by[NQ][2];
    bool no = false;
    for (int r = 0; r < NQ; ++r)
        for (int j = 0; j < 2; ++j) {
            float sc[4], top = -INFINITY, mx = -INFINITY;
            for (int k = 0; k < 4; ++k) {
                sc[k] = x.s[k][r][j] - __shfl_sync(0xffffffffu, x.ev, 8 * k + g);
                top = fmaxf(top, sc[k]);
                x.s[k][r][j] = sc[k] + __shfl_sync(0xffffffffu, now, 8 * k + g);
                mx = fmaxf(mx, x.s[k][r][j]);
            }
            top = over_keys(top);
            x.mx[r][j] = mx = over_keys(mx);
            // the row's first keys set R, later ones raise it
            const float m = x.m[r][j], R0 = x.far ? s_r[8 * r + 2 * t4 + j] : m - was - kW0;
            const float R1 = m == -INFINITY ? (top == -INFINITY ? 0.f : top) : top > R0 + 16.0f ? top : R0;
            float l = x.l[r][j];
            if (l != 0.f) l *= ex2(R0 - R1);
            for (int k = 0; k < 4; ++k) l += ex2(sc[k] - R1);
            x.l[r][j] = l;
            // against M - E0 - 12 again?
            const float mn = fmaxf(m, mx);
            R[r][j] = R1;
            by[r][j] = mn == -INFINITY ? 0.f : R1 - (mn - (float)(x.e0 - 127) - kW0);
            no = no || fabsf(by[r][j]) > 60.0f;
        }
    __syncwarp();
    x.far = __any_sync(0xffffffffu, no);
    for (int r = 0; r < NQ; ++r)
        for (int j = 0; j < 2; ++j) {
            if (x.far) {
                if (g == 0) s_r[8 * r + 2 * t4 + j] = R[r][j];
            } else if (x.l[r][j] != 0.f) x.l[r][j] *= ex2(by[r][j]);
        }
    __syncwarp();
}

// ROWS8: tiles have at most 8 rows, the other half of the matrix product's rows stays empty
template <int D, int SRC, bool ROWS8>
__global__ void __launch_bounds__(RW * 32, 3) attention_rows_kernel(const __grid_constant__ AttnArgs a, const int cluster) {
    using C = Cfg<D, SRC>;
    constexpr bool E8 = C::E8, PAGED = SRC != kPacked;
    constexpr int RB = C::RB, KS = C::KS, NS = C::NS, CH = RB / 16;   // CH: 16-byte chunks of a row
    constexpr int NQ = ROWS8 ? 1 : 2;                                 // tiles of 8 rows
    constexpr int EC = E8 ? 16 : 8;                                   // elements of a chunk
    constexpr int KK = D / 16;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ float s_m[RW][RM], s_l[RW][RM], s_r[E8 ? RW : 1][RM];   // s_r: R where it is not M - E0
    __shared__ int s_odd[RW];   // whether the warp has made values finite
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    RowTile t;
    if (!find_tile(a, blockIdx.x, ROWS8 ? 8 : RM, a.causal, t)) return;   // the whole cluster alike
    if (cluster > 1) cluster_started();
    const int hk = blockIdx.y, rank = blockIdx.z % cluster, split = blockIdx.z / cluster;
    const int n_rows = min(ROWS8 ? 8 : RM, t.nq * a.G - t.row0);

    // keys of the tile: steps [s0, s1) of this split
    const int most = keys_seen(a, t, (t.row0 + n_rows - 1) / a.G);
    const int n_steps = (most + KS - 1) / KS, per = (n_steps + a.splits - 1) / a.splits;
    const int s0 = min(n_steps, split * per), s1 = min(n_steps, s0 + per);
    const int first = s0 + rank * RW + warp, stride = cluster * RW;

    // Queries, asked for first: row 8 r + g; the pairs of k-step kk of lane t4 are elements 4 i + {0, 1} and
    // {2, 3} of the row's 16-byte (in the keys' type) chunk t4 + 4 h.
    uint2 raw[KK][NQ];
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
        const bool on = g + 8 * r < n_rows;
        const int rr = t.row0 + (on ? g + 8 * r : 0);
        const char* q = a.q.p + (t.q0 + rr / a.G) * a.q.st + (int64_t)(hk * a.G + rr % a.G) * a.q.sh;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int h = kk / (EC / 4), i = kk % (EC / 4);
            raw[kk][r] = on ? *reinterpret_cast<const uint2*>(q + ((t4 + 4 * h) * EC + 4 * i) * 2) : make_uint2(0u, 0u);
        }
    }

    const uint32_t ring = smem_u32(dyn) + warp * C::WARP;
    constexpr int U = KS / 16;   // a page holds whole blocks of 16 keys
    auto pages_of = [&](int step, int (&pg)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            pg[u] = -1;
            const int pos = step * KS + 16 * u;
            if (PAGED && step < s1 && pos < most) pg[u] = a.c.table[(int64_t)t.b * a.c.max_pages + (pos >> a.c.page_shift)];
        }
    };
    auto issue = [&](int step, int slot, const int (&pg)[U]) {
        if (step < s1) {
            const uint32_t dk = ring + slot * C::STAGE, dv = dk + KS * RB;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pos0 = step * KS + 16 * u;
                const char *sk, *sv;
                int64_t row0 = 0;
                bool on = true;
                if (PAGED) {
                    on = pg[u] >= 0 && pg[u] < a.c.num_pages;
                    row0 = on ? (((int64_t)pg[u] * a.c.H + hk) << a.c.page_shift) + (pos0 & (a.c.page_size - 1)) : 0;
                    sk = a.c.k + row0 * RB, sv = a.c.v + row0 * RB;
                } else {
                    sk = a.k.p + (t.k0 + pos0) * a.k.st + hk * a.k.sh;
                    sv = a.v.p + (t.k0 + pos0) * a.v.st + hk * a.v.sh;
                }
                if (on && pos0 + 16 <= most) {
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i) {
                        const int x = lane + 32 * i, r = x / CH, c = x % CH;
                        cp16(dk + (16 * u + r) * RB + swizzle_k<CH>(r, c) * 16, sk + r * (PAGED ? RB : a.k.st) + c * 16, true);
                        cp16(dv + (16 * u + r) * RB + swizzle_v<CH>(r, c) * 16, sv + r * (PAGED ? RB : a.v.st) + c * 16, true);
                    }
                } else {
                    // no page, or no row of the tile sees more: zeros (nothing is read, the address stays inside the tensors)
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i) {
                        const int x = lane + 32 * i, r = x / CH, c = x % CH;
                        const bool ok = on && pos0 + r < most;
                        cp16(dk + (16 * u + r) * RB + swizzle_k<CH>(r, c) * 16, ok ? sk + r * (PAGED ? RB : a.k.st) + c * 16 : PAGED ? a.c.k : a.k.p, ok);
                        cp16(dv + (16 * u + r) * RB + swizzle_v<CH>(r, c) * 16, ok ? sv + r * (PAGED ? RB : a.v.st) + c * 16 : PAGED ? a.c.v : a.v.p, ok);
                    }
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

    // queries as fragments
    uint32_t qb[KK][NQ][2];
    float rs[NQ][2];     // rows 8 r + 2 t4 + j: factor of the scores (softmax scale, log2 e, Q's exponent)
    int seen[NQ][2];     // and the keys that the row sees
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
        float mul = 1.0f, back = a.scale_log2;
        if (E8) {
            uint32_t mx = 0;   // largest magnitude, bits of a bf16 in either half
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) mx = __vmaxu2(mx, __vmaxu2(raw[kk][r].x & 0x7fff7fffu, raw[kk][r].y & 0x7fff7fffu));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // exponent e of the maximum (2^e <= it < 2^(e+1); infinities and NaN: 128); Q' = Q 2^(14 - e)
            const uint32_t top = max(mx << 16, mx & 0xffff0000u);
            const int e = top ? (int)(top >> 23) - 127 : 14, up = min(14 - e, 120);
            mul = pow2i(up);
            back *= pow2i(-up);
        }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const uint2 x = raw[kk][r];
            qb[kk][r][0] = E8 ? pack_f16(__uint_as_float(x.x << 16) * mul, __uint_as_float(x.x & 0xffff0000u) * mul) : x.x;
            qb[kk][r][1] = E8 ? pack_f16(__uint_as_float(x.y << 16) * mul, __uint_as_float(x.y & 0xffff0000u) * mul) : x.y;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int qr = 8 * r + 2 * t4 + j;
            rs[r][j] = __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + j));
            seen[r][j] = qr < n_rows ? keys_seen(a, t, (t.row0 + qr) / a.G) : 0;
        }
    }
    const int all_see = keys_seen(a, t, t.row0 / a.G);   // keys that every row of the tile sees

    float o[KK][NQ][4];
    float m[NQ][2], l[NQ][2];
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
        m[r][0] = m[r][1] = -INFINITY;
        l[r][0] = l[r][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KK; ++i) o[i][r][0] = o[i][r][1] = o[i][r][2] = o[i][r][3] = 0.f;
    }
    constexpr float W0 = E8 ? kW0 : 0.0f;
    if (lane == 0) s_odd[warp] = 0;
    __syncwarp();
    int e0 = -1;         // E0 as a scale byte; none yet
    bool far = false;    // R is s_r's

    int slot = 0, fill = NS - 1;
    for (int step = first; step < s1; step += stride) {
        issue(step + (NS - 1) * stride, fill, pg);
        pages_of(step + NS * stride, pg);
        fill = fill + 1 == NS ? 0 : fill + 1;
        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t bk = ring + slot * C::STAGE, bv = bk + KS * RB;
        slot = slot + 1 == NS ? 0 : slot + 1;

        if (__builtin_expect(all_see < most && (step + 1) * KS > all_see, 0))   // values that not all rows see
            make_finite<E8, CH>(bv, max(0, all_see - step * KS), min(KS, most - step * KS), &s_odd[warp]);

        // 8-bit, a lane per key: scales; off: its value's exponent is not near E0
        float kf = 0.f, ev_ = 0.f, inv_ = 0.f;
        bool off = false;
        if (E8) {
            static_assert(!E8 || KS == 32, "a lane per key");
            // value scales outside 2^-100 .. 2^119 are not valid; the zeros read for missing pages are among them
            const uint32_t kb = lds_u8(bk + 2 * KS * RB + lane), vb = min(max(lds_u8(bk + 2 * KS * RB + KS + lane), 27u), 246u);
            kf = scale_of((uint8_t)kb);
            ev_ = __uint_as_float(0x4b000000u | vb) - (8388608.0f + 127.0f);   // 2^23 + vb as a float
            const int some = (int)__shfl_sync(0xffffffffu, vb, 0);
            e0 = e0 < 0 ? some : e0;
            off = far || abs((int)vb - e0) > kNear;
            inv_ = __uint_as_float((uint32_t)(127 + e0 - (int)vb) << 23);   // not used where one is off
        }

        // scores: s[u][r][2 half + j] is key 16 u + 8 half + g, row 8 r + 2 t4 + j
        float s[U][NQ][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int r = 0; r < NQ; ++r) s[u][r][0] = s[u][r][1] = s[u][r][2] = s[u][r][3] = 0.f;
            const uint32_t row = bk + (16 * u + g) * RB;
#pragma unroll
            for (int h = 0; h < CH / 4; ++h) {
                const uint32_t at = swizzle_k<CH>(g, t4 + 4 * h) * 16;
                const uint4 w0 = lds128(row + at), w1 = lds128(row + 8 * RB + at);
                const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int i = 0; i < EC / 4; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if (E8) widen(x0[i], a0, a2), widen(x1[i], a1, a3);
                    else a0 = x0[2 * i % 4], a1 = x1[2 * i % 4], a2 = x0[(2 * i + 1) % 4], a3 = x1[(2 * i + 1) % 4];
#pragma unroll
                    for (int r = 0; r < NQ; ++r)
                        mma16816<E8>(s[u][r], a0, a1, a2, a3, qb[h * (EC / 4) + i][r][0], qb[h * (EC / 4) + i][r][1]);
                }
            }
        }
        // in log2 units, with the value scale's exponent added
        float inv[U][2];
        if (E8) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int src = 16 * u + 8 * k + g;
                    const float f = __shfl_sync(0xffffffffu, kf, src), ev = __shfl_sync(0xffffffffu, ev_, src);
                    inv[u][k] = __shfl_sync(0xffffffffu, inv_, src);
#pragma unroll
                    for (int r = 0; r < NQ; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) s[u][r][2 * k + j] = fmaf(s[u][r][2 * k + j], rs[r][j] * f, ev);
                }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][r][e] *= rs[r][e & 1];
        }
        if ((step + 1) * KS > all_see) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < NQ; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (step * KS + 16 * u + 8 * (e >> 1) + g >= seen[r][e & 1]) s[u][r][e] = -INFINITY;
        }
        float mx[NQ][2];
        bool raise = off, apart = false;   // apart: the step's sum from its scores
#pragma unroll
        for (int r = 0; r < NQ; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = fmaxf(s[0][r][j], s[0][r][2 + j]);
#pragma unroll
                for (int u = 1; u < U; ++u) x = fmax3(x, s[u][r][j], s[u][r][2 + j]);
                mx[r][j] = over_keys(x);
                raise = raise || mx[r][j] > m[r][j] + 3.0f;
            }
        if (__any_sync(0xffffffffu, raise)) {
            if (E8) {
                // value rows of zeros (lane: key of the step); rarely more than a look at one chunk
                auto zero = [&](int c) {
                    const uint4 w = lds128(bv + lane * RB + c * 16);
                    return ((w.x | w.y | w.z | w.w) & 0x7f7f7f7fu) == 0u;
                };
                bool none = zero(lane % CH);
                if (__builtin_expect(__any_sync(0xffffffffu, none), 0)) {
                    for (int c = 0; c < CH; ++c) none = none && zero(c);
                    none = none && step * KS + lane < most;
                }
                apart = __any_sync(0xffffffffu, off || none);
                if (__builtin_expect(apart, 0)) {
                    Apart<NQ> x;
#pragma unroll
                    for (int r = 0; r < NQ; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            x.m[r][j] = m[r][j], x.l[r][j] = l[r][j];
#pragma unroll
                            for (int k = 0; k < 4; ++k) x.s[k][r][j] = s[k >> 1][r][2 * (k & 1) + j];
                        }
                    x.ev = ev_, x.none = none, x.e0 = e0, x.far = far;
                    sum_apart(x, s_r[warp % (E8 ? RW : 1)]);
                    e0 = x.e0, far = x.far;
#pragma unroll
                    for (int r = 0; r < NQ; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            l[r][j] = x.l[r][j], mx[r][j] = x.mx[r][j];
#pragma unroll
                            for (int k = 0; k < 4; ++k) s[k >> 1][r][2 * (k & 1) + j] = x.s[k][r][j];
                        }
                }
            }
#pragma unroll
            for (int r = 0; r < NQ; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float mn = fmaxf(m[r][j], mx[r][j]);
                    const float f = mn == -INFINITY ? 1.0f : exp2f(m[r][j] - mn);
                    m[r][j] = mn;
                    if (!E8 || !apart) l[r][j] *= f;
#pragma unroll
                    for (int i = 0; i < KK; ++i) o[i][r][j] *= f, o[i][r][2 + j] *= f;
                }
        }
        uint32_t p[U][NQ][2];   // weights of keys 16 u + 8 half + 2 t4 + {0, 1}, row 8 r + g
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
            float sum0 = E8 ? 0.f : l[r][0], sum1 = E8 ? 0.f : l[r][1];
            const float ref0 = (m[r][0] == -INFINITY ? 0.f : m[r][0]) - W0, ref1 = (m[r][1] == -INFINITY ? 0.f : m[r][1]) - W0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float w0 = ex2(s[u][r][2 * k] - ref0), w1 = ex2(s[u][r][2 * k + 1] - ref1);
                    sum0 = E8 ? fmaf(w0, inv[u][k], sum0) : sum0 + w0;
                    sum1 = E8 ? fmaf(w1, inv[u][k], sum1) : sum1 + w1;
                    p[u][r][k] = transpose8(E8 ? pack_f16(w0, w1) : pack_bf16(w0, w1));
                }
            if (!E8) l[r][0] = sum0, l[r][1] = sum1;
            else if (!apart) l[r][0] += sum0, l[r][1] += sum1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t rows = bv + (16 * u + 2 * t4) * RB;   // this lane's keys: +0, +1, +8, +9
            constexpr int W = E8 && D == 64 ? 2 : 4;             // words of a key that a lane reads at once
#pragma unroll
            for (int h = 0; h < KK * 2 / (W * (E8 ? 4 : 2)); ++h) {
                uint32_t x0[W], x1[W], y0[W], y1[W];
                if constexpr (W == 2) {
                    const uint32_t off = (uint32_t)(swizzle_v<CH>(2 * t4, g >> 1) * 16 + (g & 1) * 8);
                    lds64(rows + off, x0), lds64(rows + RB + off, x1), lds64(rows + 8 * RB + off, y0), lds64(rows + 9 * RB + off, y1);
                } else {
                    const uint32_t off = (uint32_t)swizzle_v<CH>(2 * t4, g + 8 * h) * 16;
                    lds128(rows + off, x0), lds128(rows + RB + off, x1), lds128(rows + 8 * RB + off, y0), lds128(rows + 9 * RB + off, y1);
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (E8) {
                        // elements 4 i .. 4 i + 3, each as a pair of keys
                        uint32_t e0, e1, e2, e3, f0, f1, f2, f3;
                        widen(__byte_perm(x0[i], x1[i], 0x5140), e0, e1);
                        widen(__byte_perm(x0[i], x1[i], 0x7362), e2, e3);
                        widen(__byte_perm(y0[i], y1[i], 0x5140), f0, f1);
                        widen(__byte_perm(y0[i], y1[i], 0x7362), f2, f3);
#pragma unroll
                        for (int r = 0; r < NQ; ++r) {
                            mma16816<E8>(o[(2 * i) % KK][r], e0, e1, f0, f1, p[u][r][0], p[u][r][1]);
                            mma16816<E8>(o[(2 * i + 1) % KK][r], e2, e3, f2, f3, p[u][r][0], p[u][r][1]);
                        }
                    } else {
                        const uint32_t e0 = __byte_perm(x0[i], x1[i], 0x5410), e1 = __byte_perm(x0[i], x1[i], 0x7632);
                        const uint32_t f0 = __byte_perm(y0[i], y1[i], 0x5410), f1 = __byte_perm(y0[i], y1[i], 0x7632);
#pragma unroll
                        for (int r = 0; r < NQ; ++r) mma16816<E8>(o[(4 * h + i) % KK][r], e0, e1, f0, f1, p[u][r][0], p[u][r][1]);
                    }
                }
            }
        }
        __syncwarp();   // the next copy into this slot comes after every lane's reads
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warp's rows into its ring
    const float w0 = pow2i(-(int)W0);
#pragma unroll
    for (int r = 0; r < NQ; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 8 * r + 2 * t4 + j;
            float x = l[r][j];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (E8) x = lg2(x) + (far ? s_r[warp % (E8 ? RW : 1)][row] : m[r][j] - (float)(e0 - 127) - W0);   // -inf of a sum of 0
            if (g == 0) s_m[warp][row] = m[r][j], s_l[warp][row] = x;
#pragma unroll
            for (int i = 0; i < KK; ++i) {
                // elements 2 i and 2 i + 1 of the ones that this lane's group loaded of each key
                const int d = E8 ? g * (D / 8) + 2 * i : (2 * i / 8) * 64 + g * 8 + 2 * i % 8;
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ring + (row * D + d) * 4), "f"(o[i][r][j] * w0), "f"(o[i][r][2 + j] * w0) : "memory");
            }
        }
    join_rows<__nv_bfloat16, typename std::conditional<E8, uint8_t, __nv_bfloat16>::type, D, PAGED, C::WARP, ROWS8 ? 8 : 16, true, E8>(
        a, t, hk, split, rank, cluster, n_rows, max(s0 * KS, all_see), min(s1 * KS, most), s_m, s_l, s_odd, smem_u32(dyn));
}

template <int D, int SRC, bool ROWS8>
vdm_status launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = attention_rows_kernel<D, SRC, ROWS8>;
    constexpr int M = ROWS8 ? 8 : RM;
    static std::atomic<uint64_t> ready{0};
    VDM_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(kern), Cfg<D, SRC>::SMEM));
    const int64_t tiles = row_tiles(a.Tq, a.G, a.B, M);
    VDM_TRY(launch_cluster(kern, dim3((unsigned)tiles, a.Hk, a.splits * a.cluster), RW * 32, Cfg<D, SRC>::SMEM, a.cluster, s, a, a.cluster));
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
