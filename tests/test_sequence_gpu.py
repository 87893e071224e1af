"""Token-sequence operators on the GPU against the float64 oracle.

Tolerances (u = 2^-24 is half a float32 step; a bf16 rounding is off by at most 2^-8
of the value, half of finfo.eps):

* norm + rotation: the sum of squares of D terms (D u, halved by the root), rsqrt, gain and
  two products of the rotation: (D/2 + 16) u of the pair's length, and u of the angle's sine
  and cosine (reduced in float64); with bf16 outputs 2^-8 of the value more.
* attention: a score is a float32 sum of D products, so it is off by at most
  d = (D + 8) u scale sum|q k| (absolute), every weight by the factor 1 + 2 d + 2^-20
  (exponential), sums over n keys by (n + 16) u; each moves the output by that share of
  max|v|.  bf16 calls round the weights once (2^-8 max|v|) and the output (2^-8 |out|), and a
  part of their exponentials may be off by 7.5e-5.
* the log of the sums: d, 2^-20, and n u from the sum (bf16: 7.5e-5 too).
* cache: codes, scales and what is read back are equal, bit for bit.
"""
import numpy as np
import pytest
import torch

import neural_sdf_volume_b200 as vdm
from oracle import sequence as OS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(seed, *shape, dtype="bf16", scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * scale).to(DT[dtype])


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens):
    return ints([0] + list(np.cumsum(lens)))


def np64(x):
    return x.detach().double().cpu().numpy()


def close(got, want, tol, what=""):
    got, want, tol = np64(got) if torch.is_tensor(got) else got, np.asarray(want), np.broadcast_to(tol, np.shape(want))
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(np.isinf(got), np.isinf(want)), what
    fin = np.isfinite(want)
    err = np.abs(got[fin] - want[fin])
    assert (err <= tol[fin]).all(), f"{what}: error {err.max()} at tolerance {tol[fin][np.argmax(err - tol[fin])]}"


# ----------------------------------------------------------------- norm + rotation

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T, Hq, Hk, rot, inter", [
    (1, 8, 8, 64, False), (1, 1, 1, 64, True), (5, 7, 3, 48, False), (5, 7, 3, 48, True), (130, 32, 8, 64, False),
    (33, 5, 0, 2, False), (33, 5, 1, 22, False), (33, 5, 1, 22, True), (9, 6, 2, 0, False), (17, 16, 1, -1, False), (17, 16, 1, -1, True)])
def test_norm_rope(dtype, D, T, Hq, Hk, rot, inter):
    rot = D if rot < 0 else rot
    x = randn(T + D, T, Hq + 2 * Hk + 1, D, dtype=dtype, scale=2.0)      # slices of a fused projection
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk] if Hk else None
    gq, gk = (1 + 0.3 * torch.randn(D, generator=gen(s), device="cuda") for s in (1, 2))
    pos = ints(np.random.default_rng(T).integers(0, 1 << 20, T))
    if T > 2:
        pos[1], pos[2] = 0, 2 ** 31 - 1
    rope = vdm.Rope.make(rot, interleaved=inter, mscale=1.25, factor=8.0, original_length=4096) if rot else None
    before = x.clone()
    qo, ko = vdm.vdm_qk_norm_rope(q, k, pos if rot else None, rope, q_gain=gq, k_gain=gk, eps=1e-5)
    assert torch.equal(x, before)
    f = np64(rope.inv_freq) if rot else None
    for name, got, src, g in (("q", qo, q, gq), ("k", ko, k, gk)):
        if src is None:
            assert got is None
            continue
        want = OS.norm_rope(np64(src), np64(g), 1e-5, np64(pos), f, inter, 1.25)
        size = np.abs(OS.norm_rope(np64(src), np64(g), 1e-5)) * (1.25 if rot else 1.0)
        pair = np.broadcast_to(size.max(-1, keepdims=True) * np.sqrt(2), size.shape)
        tol = (D / 2 + 16 + 8) * U * pair + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
        close(got, want, tol, name)


def test_norm_rope_in_place_without_norm_and_on_one_side():
    x = randn(3, 40, 12, 64)
    q, k = x[:, :8], x[:, 8:]
    pos, rope, g = torch.arange(40, dtype=torch.int32, device="cuda"), vdm.Rope.make(64), torch.ones(64, device="cuda")
    want_q, want_k = vdm.vdm_qk_norm_rope(q, k, pos, rope, q_gain=g)
    got = x.clone()
    vdm.vdm_qk_norm_rope(got[:, :8], got[:, 8:], pos, rope, q_gain=g, q_out=got[:, :8], k_out=got[:, 8:])
    assert torch.equal(got[:, :8], want_q) and torch.equal(got[:, 8:], want_k)
    close(want_k, OS.norm_rope(np64(k), None, 0, np64(pos), np64(rope.inv_freq)), 24 * U * 8 + 2.0 ** -8 * np.abs(np64(want_k)) + 1e-6)
    e, _ = vdm.vdm_qk_norm_rope(x[:0, :8], None, pos[:0], rope)
    assert e.shape == (0, 8, 64)
    z, _ = vdm.vdm_qk_norm_rope(torch.zeros_like(q), None, pos, rope, q_gain=g, eps=0.0)     # 0 / 0 stays what the formula gives
    assert torch.isnan(z).all()


# ----------------------------------------------------------------- attention

def tolerance(q, k, v, want, scale, dtype):
    """Largest allowed |error| of out (array) and lse (number)."""
    D, n = q.shape[-1], max(1, k.shape[0])
    fin = lambda x: np.abs(x[np.isfinite(x)]).max() if np.isfinite(x).any() else 0.0
    d = (D + 8) * U * scale * D * fin(q) * fin(k)
    vmax = fin(v)
    share = 2 * d + 2.0 ** -20 + (n + 16) * U
    ltol = d + 2.0 ** -20 + (n + 16) * U + 1e-5
    if dtype == "bf16":
        share += 2.0 ** -8 + 7.5e-5
        ltol += 7.5e-5
        return share * vmax + 2.0 ** -8 * np.abs(want), ltol
    return share * vmax + U * np.abs(want), ltol


def check_packed(dtype, D, Hq, Hk, nq, nk, causal, seed=0, extra=3, scale=None):
    Tq, Tk = sum(nq) + extra, sum(nk) + extra
    q = randn(seed, Tq, Hq + 1, D, dtype=dtype)[:, :Hq]
    kv = randn(seed + 1, Tk, 2 * Hk, D, dtype=dtype, scale=1.5)
    k, v = kv[:, :Hk], kv[:, Hk:]
    kv[sum(nk):] = float("nan")                  # rows behind the last sequence
    cu_q, cu_k = offsets(nq), offsets(nk)
    out = torch.full((Tq, Hq, D), 7.0, device="cuda", dtype=DT[dtype])
    sc = D ** -0.5 if scale is None else scale
    got, lse = vdm.vdm_attention_packed(q, k, v, cu_q, cu_k, causal=causal, out=out, want_lse=True, scale=scale)
    vdm.vdm_attention_status()
    want, wl = OS.packed(np64(q), np64(k), np64(v), np.cumsum([0] + list(nq)), np.cumsum([0] + list(nk)), causal, sc)
    n = sum(nq)
    assert (out[n:] == 7.0).all()
    tol, ltol = tolerance(np64(q), np64(k)[:max(nk, default=0) or 1], np64(v)[:sum(nk)], want[:n], sc, dtype)
    close(got[:n], want[:n], tol, "out")
    close(lse[:n], wl[:n], ltol + 4 * U * np.abs(np.where(np.isfinite(wl[:n]), wl[:n], 0)), "lse")
    return q, k, v, cu_q, cu_k, got, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq, Hk, lens", [
    (1, 1, [1]), (8, 8, [0, 1, 63, 64, 0, 65, 129]), (6, 2, [130, 1, 0, 200]), (15, 3, [37, 300]), (16, 1, [257, 16, 8, 1]), (7, 7, [511, 513])])
def test_packed_self_attention(dtype, D, causal, Hq, Hk, lens):
    check_packed(dtype, D, Hq, Hk, lens, lens, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq, Hk, nq, nk", [
    (8, 2, [5, 0, 140, 1], [0, 40, 12, 700]),           # no keys, no queries, more queries than keys, one query
    (4, 4, [1, 1, 1], [1, 1000, 129]), (12, 4, [300], [1500]), (32, 8, [33, 2], [4100, 128])])
def test_packed_queries_and_keys_of_different_lengths(dtype, D, causal, Hq, Hk, nq, nk):
    check_packed(dtype, D, Hq, Hk, nq, nk, causal)


def test_packed_is_the_same_for_many_small_sequences():
    lens = [i % 7 for i in range(150)]                  # more sequences than a warp has lanes, empty ones among them
    check_packed("bf16", 64, 4, 2, lens, lens, True)
    check_packed("f32", 64, 4, 2, lens, lens, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_large_logits_and_scale(dtype):
    check_packed(dtype, 64, 2, 1, [70, 300], [70, 300], True, seed=5, scale=3.0)
    check_packed(dtype, 64, 2, 1, [70, 300], [70, 300], False, seed=6, scale=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_packed_unseen_keys_have_no_influence(dtype, D, bad):
    """Causal: rows before token j equal those of a run without the bad token's values; later rows meet them."""
    n, j = 300, 171
    q, k, v = (randn(s, n, 4, D, dtype=dtype) for s in (1, 2, 3))
    want = vdm.vdm_attention_packed(q, k, v, offsets([n]))
    for where in (k, v):
        x = where.clone()
        x[j] = bad
        a = [q, x if where is k else k, x if where is v else v]
        got = vdm.vdm_attention_packed(*a, offsets([n]))
        oracle, _ = OS.attention(np64(q), np64(a[1]), np64(a[2]), True, D ** -0.5) if where is v else (None, None)
        tol, _ = tolerance(np64(q), np64(k), np64(v), np64(want), D ** -0.5, dtype)
        close(got[:j], np64(want)[:j], 2 * tol[:j], "rows that do not see it")
        if where is v:
            assert np.array_equal(np.isnan(np64(got)[j:]), np.isnan(oracle[j:]))
        else:
            assert not torch.isfinite(got[j:]).all()


def test_packed_masks_by_keys_of_minus_infinity():
    """A key row of -inf against positive queries has score -inf: weight 0, like a removed key; all of them: an empty row."""
    q, k, v = torch.ones(40, 2, 64, device="cuda"), randn(2, 40, 2, 64, dtype="f32"), randn(3, 40, 2, 64, dtype="f32")
    for dt in (torch.float32, torch.bfloat16):
        kk = k.to(dt).clone()
        kk[10:25] = float("-inf")
        keep = torch.tensor([i for i in range(40) if not 10 <= i < 25], device="cuda")
        a = vdm.vdm_attention_packed(q.to(dt), kk, v.to(dt), offsets([40]), causal=False)
        b = vdm.vdm_attention_packed(q.to(dt), kk[keep], v.to(dt)[keep], offsets([40]), offsets([25]), causal=False)
        close(a, np64(b), 2.0 ** -6 if dt is torch.bfloat16 else 1e-5)
        kk[:] = float("-inf")
        o, l = vdm.vdm_attention_packed(q.to(dt), kk, v.to(dt), offsets([40]), causal=False, want_lse=True)
        assert (o == 0).all() and torch.isneginf(l).all()


# ----------------------------------------------------------------- cache

def make_table(rng, need, width, pages, bad=()):
    """Pages of each sequence in random order, -1 behind them."""
    order = rng.permutation(pages)
    t, at = np.full((len(need), width), -1, np.int32), 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    for b, j, x in bad:
        t[b, j] = x
    return t


class Cached:
    """Random sequences in a cache, and the rows they stand for in float64."""

    def __init__(self, kind, H, D, page, total, seed=0, spare=2, bad=(), width=None):
        rng = np.random.default_rng(seed)
        need = [-(-t // page) for t in total]
        self.width = max([1, *need]) if width is None else width
        P = sum(need) + spare
        self.tab = make_table(rng, need, self.width, P, bad)
        self.total, self.page, self.H, self.D, self.kind, self.P = total, page, H, D, kind, P
        self.cache = vdm.KVCache.create(P, page, H, D, kind)
        self.rows = {}
        for n in "kv":
            pages = getattr(self.cache, n)
            if kind == "e4m3":
                codes = rng.integers(0, 256, tuple(pages.shape)).astype(np.uint8)
                codes[(codes & 127) == 127] = 0
                scale = rng.integers(116, 121, tuple(pages.shape[:3])).astype(np.uint8)
                # unused rows hold NaN
                used = np.zeros(tuple(pages.shape[:3]), bool)
                for b, t in enumerate(total):
                    for p in range(t):
                        if 0 <= p // page < self.width and 0 <= self.tab[b, p // page] < P:
                            used[self.tab[b, p // page], :, p % page] = True
                codes[~used] = 127
                pages.copy_(torch.from_numpy(codes))
                getattr(self.cache, n + "_scale").copy_(torch.from_numpy(scale))
                self.rows[n] = OS.dequantise(codes, scale)
            else:
                x = torch.from_numpy(rng.normal(size=tuple(pages.shape))).to(pages.dtype)
                used = torch.zeros(pages.shape[:3], dtype=torch.bool)
                for b, t in enumerate(total):
                    for p in range(t):
                        if 0 <= p // page < self.width and 0 <= self.tab[b, p // page] < P:
                            used[self.tab[b, p // page], :, p % page] = True
                x[~used] = float("nan")
                pages.copy_(x)
                self.rows[n] = np64(pages)
        self.table, self.kv_len = ints(self.tab), ints(total)

    def sequence(self, n, b):
        """Rows of sequence b [tokens, H, D]; zeros where there is no page."""
        t = max(0, min(self.total[b], self.width * self.page))
        out = np.zeros((t, self.H, self.D))
        for p in range(t):
            pg = self.tab[b, p // self.page]
            if 0 <= pg < self.P:
                out[p] = self.rows[n][pg, :, p % self.page]
        return out


@pytest.mark.parametrize("dtype, kind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("H, D, page, new, total", [
    (8, 64, 16, [1, 1, 1], [1, 16, 17]), (3, 128, 32, [5, 0, 40, 31], [5, 7, 100, 32]), (1, 64, 256, [300], [300]),
    (5, 128, 128, [0, 3, 0], [0, 130, 9])])
def test_cache_write(dtype, kind, H, D, page, new, total):
    c = Cached(kind, H, D, page, total, seed=1)
    T = sum(new) + 2
    x = randn(1, T, 2 * H, D, dtype=dtype, scale=30.0)
    x *= torch.exp2(torch.randint(-20, 20, (T, 2 * H, 1), generator=gen(3), device="cuda").float()).to(x.dtype)
    if T > 4:
        x[1, 0] = 0
        x[2, 0, 5], x[2, 0, 6] = float("nan"), float("inf")
        x[3, 0] = float("nan")
        x[0, 0, :] = 448.0
    k, v = x[:, :H], x[:, H:]
    before = [t.clone() for t in (c.cache.k, c.cache.v)]
    vdm.vdm_cache_write(c.cache, k, v, offsets(new), c.kv_len, c.table)
    want = [b.clone().cpu() for b in before]
    sc = [None, None]
    if kind == "e4m3":
        ref = Cached(kind, H, D, page, total, seed=1).cache
        sc = [ref.k_scale.cpu(), ref.v_scale.cpu()]
    at = 0
    for b, n in enumerate(new):
        for i in range(n):
            p = total[b] - n + i
            if p >= 0:
                pg, r = c.tab[b, p // page], p % page
                for w, s, src in zip(want, sc, (k, v)):
                    row = src[at + i]
                    if kind == "e4m3":
                        codes, scale = OS.quantise(np64(row))
                        w[pg, :, r], s[pg, :, r] = torch.from_numpy(codes), torch.from_numpy(scale)
                    else:
                        w[pg, :, r] = row.cpu()
        at += n
    for got, w in zip((c.cache.k, c.cache.v), want):
        if kind == "e4m3":       # a NaN's sign is not defined
            g, w = got.cpu(), w
            nan = (w & 127) == 127
            assert torch.equal((g & 127) == 127, nan) and torch.equal(g[~nan], w[~nan])
        else:
            assert torch.equal(got.cpu().view(torch.int16 if kind == "bf16" else torch.int32), w.view(torch.int16 if kind == "bf16" else torch.int32))
    if kind == "e4m3":
        assert torch.equal(c.cache.k_scale.cpu(), sc[0]) and torch.equal(c.cache.v_scale.cpu(), sc[1])


@pytest.mark.parametrize("dtype, kind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("H, D, page, total", [(8, 64, 16, [1, 0, 16, 33]), (3, 128, 64, [200, 64]), (1, 64, 256, [300, 5])])
def test_cache_read(dtype, kind, H, D, page, total):
    c = Cached(kind, H, D, page, total, seed=2)
    n = sum(total)
    out = tuple(torch.full((n + 2, 2 * H, D), 9.0, device="cuda", dtype=DT[dtype])[:, ::2] for _ in "kv")
    k, v = vdm.vdm_cache_read(c.cache, c.kv_len, c.table, offsets(total), out=out)
    for got, name in ((k, "k"), (v, "v")):
        want = torch.from_numpy(np.concatenate([c.sequence(name, b) for b in range(len(total))])).to(DT[dtype])
        assert torch.equal(got[:n].cpu(), want) and (got[n:] == 9.0).all()
    a, b = vdm.vdm_cache_read(c.cache, c.kv_len, c.table, offsets(total), total=n)
    assert a.dtype is (torch.bfloat16 if kind == "e4m3" else DT[kind]) and torch.equal(a.double(), k[:n].double() if a.dtype is k.dtype else a.double())


def test_cache_bad_pages_lengths_and_short_outputs():
    """Table entries that are no page read as zeros and drop writes; lengths beyond the table are clamped; rows that no position goes to stay."""
    H, D, page = 2, 64, 16
    c = Cached("bf16", H, D, page, [40, 40, 20], seed=3, bad=[(0, 1, -7), (1, 0, 1 << 30), (1, 2, 10 ** 9)])
    k, v = vdm.vdm_cache_read(c.cache, c.kv_len, c.table, offsets([40, 40, 20]), total=100)
    assert torch.equal(k.double().cpu(), torch.from_numpy(np.concatenate([c.sequence("k", b) for b in range(3)])))
    assert (k[16:32] == 0).all() and (k[40:56] == 0).all()
    # clamped lengths: 3 pages of 16 at most
    out = tuple(torch.full((200, H, D), 9.0, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    vdm.vdm_cache_read(c.cache, ints([1000, -5, 20]), c.table, ints([0, 100, 150, 155]), out=out)
    assert (out[0][48:150] == 9.0).all() and (out[0][155:] == 9.0).all()
    assert torch.equal(out[0][150:155].double().cpu(), torch.from_numpy(c.sequence("k", 2)[:5]))
    before = c.cache.k.clone()
    new = randn(4, 30, H, D)
    # sequence 0: positions -3 .. 6 (the first three do not exist); 1: page 0 is none; 2: beyond the table
    vdm.vdm_cache_write(c.cache, new, new, offsets([10, 10, 10]), ints([7, 10, 60]), c.table)
    changed = (c.cache.k.view(torch.int16) != before.view(torch.int16)).any(-1).any(1)
    want = torch.zeros_like(changed)
    want[c.tab[0, 0], :7] = True
    assert torch.equal(changed, want)
    assert torch.equal(c.cache.k[c.tab[0, 0], :, :7].transpose(0, 1), new[3:10])
    # offsets that decrease or leave the tensor: nothing out of range is touched
    vdm.vdm_cache_write(c.cache, new, new, ints([0, 500, 20, 40]), ints([20, 20, 20]), c.table)
    vdm.vdm_cache_read(c.cache, c.kv_len, c.table, ints([-5, 500, 20, 40]), total=30)
    torch.cuda.synchronize()


# ----------------------------------------------------------------- attention over the cache

def check_paged(dtype, kind, D, Hq, Hk, page, new, total, causal=True, seed=0, bad=(), width=None):
    c = Cached(kind, Hk, D, page, total, seed=seed, bad=bad, width=width)
    T = sum(new) + 2
    q = randn(seed + 1, T, Hq, D, dtype=dtype)
    out = torch.full((T, Hq, D), 7.0, device="cuda", dtype=DT[dtype])
    got, lse = vdm.vdm_attention_paged(q, c.cache, offsets(new), c.kv_len, c.table, causal=causal, out=out, want_lse=True)
    vdm.vdm_attention_status()
    at = 0
    for b, n in enumerate(new):
        k, v = c.sequence("k", b), c.sequence("v", b)
        want, wl = OS.attention(np64(q)[at:at + n], k, v, causal, D ** -0.5)
        tol, ltol = tolerance(np64(q), k if len(k) else np.zeros((1, 1, D)), v if len(v) else np.zeros((1, 1, D)), want, D ** -0.5, dtype)
        close(got[at:at + n], want, tol, f"out of sequence {b}")
        close(lse[at:at + n], wl, ltol + 4 * U * np.abs(np.where(np.isfinite(wl), wl, 0)), f"lse of sequence {b}")
        at += n
    assert (out[at:] == 7.0).all()


KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")]


@pytest.mark.parametrize("dtype, kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq, Hk, page, total", [
    (8, 8, 16, [1, 15, 16, 17, 0, 700]), (32, 8, 64, [1, 300, 2050]), (16, 1, 32, [33, 5000]), (15, 3, 128, [129, 1]), (24, 2, 256, [255, 257])])
def test_paged_one_token(dtype, kind, D, Hq, Hk, page, total):
    check_paged(dtype, kind, D, Hq, Hk, page, [1] * len(total), total)


@pytest.mark.parametrize("dtype, kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq, Hk, page, new, total", [
    (8, 8, 16, [3, 0, 40, 1], [3, 9, 100, 77]), (12, 4, 64, [130, 17], [1000, 17]), (32, 8, 32, [64, 5], [64, 2500]),
    (6, 2, 128, [10, 9], [4, 0])])                    # more new tokens than positions: rows without keys
def test_paged_chunk(dtype, kind, D, causal, Hq, Hk, page, new, total):
    check_paged(dtype, kind, D, Hq, Hk, page, new, total, causal)


@pytest.mark.parametrize("dtype, kind", KINDS)
def test_paged_bad_pages_read_as_zeros(dtype, kind):
    check_paged(dtype, kind, 64, 8, 2, 16, [1, 70], [100, 200], bad=[(0, 2, -1), (1, 5, 10 ** 9), (1, 12, -2 ** 31)])


@pytest.mark.parametrize("dtype, kind", [("bf16", "e4m3"), ("f32", "f32")])
def test_paged_length_beyond_the_table_and_shared_pages(dtype, kind):
    c = Cached(kind, 2, 64, 16, [64, 64], seed=4)
    c.tab[1, :2] = c.tab[0, :2]                       # a shared prefix
    c.table = ints(c.tab)
    q = randn(5, 2, 8, 64, dtype=dtype)
    got = vdm.vdm_attention_paged(q, c.cache, offsets([1, 1]), ints([64, 2 ** 31 - 1]), c.table)
    for b in range(2):
        k, v = c.sequence("k", b), c.sequence("v", b)
        want, _ = OS.attention(np64(q)[b:b + 1], k, v, True, 0.125)
        close(got[b:b + 1], want, tolerance(np64(q), k, v, want, 0.125, dtype)[0])


# ----------------------------------------------------------------- together, streams, graphs

def test_chunks_and_steps_equal_the_whole_prompt():
    """A sequence fed in chunks and single tokens through norm + rotation, cache and paged attention equals packed attention over the whole."""
    Hq, Hk, D, n = 8, 2, 64, 333
    qkv = randn(1, n, Hq + 2 * Hk, D)
    gq, gk, rope = torch.ones(D, device="cuda"), torch.full((D,), 1.5, device="cuda"), vdm.Rope.make(48, factor=4.0, original_length=256)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, k = vdm.vdm_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], pos, rope, q_gain=gq, k_gain=gk)
    v = qkv[:, Hq + Hk:]
    whole = vdm.vdm_attention_packed(q, k, v, offsets([n]))
    cache = vdm.KVCache.create(30, 16, Hk, D)
    table = ints(np.random.default_rng(0).permutation(30)[None, :21])
    done, outs = 0, []
    for step in (100, 1, 130, 1, 1, 100):
        s = slice(done, done + step)
        qs, ks = vdm.vdm_qk_norm_rope(qkv[s, :Hq], qkv[s, Hq:Hq + Hk], pos[s], rope, q_gain=gq, k_gain=gk)
        assert torch.equal(qs, q[s]) and torch.equal(ks, k[s])
        done += step
        vdm.vdm_cache_write(cache, ks, v[s], offsets([step]), ints([done]), table)
        outs.append(vdm.vdm_attention_paged(qs, cache, offsets([step]), ints([done]), table))
    got = torch.cat(outs)
    tol, _ = tolerance(np64(q), np64(k), np64(v), np64(whole), D ** -0.5, "bf16")
    close(got, np64(whole), 2 * tol)
    kk, vv = vdm.vdm_cache_read(cache, ints([n]), table, offsets([n]), total=n)
    assert torch.equal(kk, k) and torch.equal(vv, v)


def test_stored_vecset_decodes_as_the_dense_one():
    """vdm_precompute_kv -> cache -> cache read -> vdm_decode_dense: bit-identical for bf16 pages, near for 8-bit ones."""
    import workloads as W
    spec = W.DecoderSpec(C=128, H=2, F=256, N=300, query_ln=True, dtype="bf16")
    d = W.make_decoder(spec, seed=0, key=2)
    dec = vdm.Decoder.from_numpy(d["weights"], spec.C, spec.H, spec.F, spec.query_ln, spec.dtype)
    K, V = vdm.vdm_precompute_kv(dec, torch.from_numpy(d["z"]).cuda())
    want = vdm.vdm_decode_dense(dec, K, V, grid_R=8)
    table = ints(np.random.default_rng(1).permutation(12)[None, :10])
    for kind in ("bf16", "e4m3"):
        cache = vdm.KVCache.create(12, 32, spec.H, 64, kind)
        vdm.vdm_cache_write(cache, K[0].transpose(0, 1), V[0].transpose(0, 1), offsets([300]), ints([300]), table)
        K2, V2 = torch.empty_like(K), torch.empty_like(V)
        vdm.vdm_cache_read(cache, ints([300]), table, offsets([300]), out=(K2[0].transpose(0, 1), V2[0].transpose(0, 1)))
        if kind == "bf16":
            assert torch.equal(K2, K) and torch.equal(V2, V)
            assert torch.equal(vdm.vdm_decode_dense(dec, K2, V2, grid_R=8), want)
        else:
            codes, scales = OS.quantise(np64(K[0]))
            assert np.array_equal(np64(K2[0]), OS.dequantise(codes, scales))


def test_other_stream_and_two_calls_at_once():
    q, k, v = (randn(s, 700, 8, 64) for s in (1, 2, 3))
    cu = offsets([700])
    want = vdm.vdm_attention_packed(q, k, v, cu)
    c = Cached("e4m3", 8, 64, 16, [3000], seed=6)
    step = randn(4, 1, 8, 64)
    wp = vdm.vdm_attention_paged(step, c.cache, offsets([1]), c.kv_len, c.table)
    one = offsets([1])
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((vdm.vdm_attention_packed(q, k, v, cu, stream=a), vdm.vdm_attention_paged(step, c.cache, one, c.kv_len, c.table, stream=b)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want) and torch.equal(y, wp)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_captured_step_replays_with_new_inputs():
    """Norm + rotation, cache write and paged attention in one graph; replayed as the sequence grows."""
    Hq, Hk, D, page = 8, 2, 64, 16
    cache = vdm.KVCache.create(40, page, Hk, D, "e4m3")
    table = ints(np.arange(40).reshape(2, 20))
    x = randn(1, 6, 2, Hq + 2 * Hk, D)                 # six steps of two sequences
    cur, pos, kv_len, cu = torch.empty_like(x[0]), ints([0, 0]), ints([1, 1]), offsets([1, 1])
    rope, g = vdm.Rope.make(64), torch.ones(D, device="cuda")

    def step():
        q, k = vdm.vdm_qk_norm_rope(cur[:, :Hq], cur[:, Hq:Hq + Hk], pos, rope, q_gain=g, k_gain=g)
        vdm.vdm_cache_write(cache, k, cur[:, Hq + Hk:], cu, kv_len, table)
        return vdm.vdm_attention_paged(q, cache, cu, kv_len, table)

    def drive(run):
        cache.k.zero_(), cache.v.zero_()
        outs = []
        for i in range(6):
            cur.copy_(x[i])
            pos.fill_(50 * i)
            kv_len.fill_(50 * i + 1)
            outs.append(run().clone())
        return torch.stack(outs)

    want = drive(step)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(other):                     # a second graph in the same process
        out2 = step()

    def replay(gr, o):
        gr.replay()
        return o

    assert torch.equal(drive(lambda: replay(graph, out)), want)
    assert torch.equal(drive(lambda: replay(other, out2)), want)


def test_results_do_not_change_from_run_to_run():
    c = Cached("bf16", 2, 128, 32, [6000, 900, 77], seed=8)
    q = randn(9, 3, 16, 128)
    first = vdm.vdm_attention_paged(q, c.cache, offsets([1, 1, 1]), c.kv_len, c.table)
    for _ in range(10):
        assert torch.equal(vdm.vdm_attention_paged(q, c.cache, offsets([1, 1, 1]), c.kv_len, c.table), first)


def test_python_checks_on_device_tensors():
    q = randn(1, 8, 8, 64)
    cu = offsets([8])
    bad = [lambda: vdm.vdm_attention_packed(q.half(), q.half(), q.half(), cu), lambda: vdm.vdm_attention_packed(q, q.float(), q, cu),
           lambda: vdm.vdm_attention_packed(q, q, q, cu.long()), lambda: vdm.vdm_attention_packed(q, q[:4], q[:4], cu),
           lambda: vdm.vdm_attention_packed(q, q, q[..., ::2], cu), lambda: vdm.vdm_attention_packed(q, q, q, cu.cpu()),
           lambda: vdm.vdm_attention_packed(q, q, q, cu, out=q[:, :4]),
           lambda: vdm.vdm_qk_norm_rope(q, None, None, vdm.Rope.make(64)), lambda: vdm.vdm_qk_norm_rope(q, q_gain=torch.ones(32, device="cuda")),
           lambda: vdm.vdm_qk_norm_rope(q, None, cu, vdm.Rope.make(64))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(vdm.VdmError) as e:
        vdm.vdm_attention_packed(q.reshape(-1)[4:-60].reshape(-1, 1, 64)[:8], q[:, :1], q[:, :1], cu)    # 8 bytes off
    assert e.value.status == 1 and "16-byte" in str(e.value)
    with pytest.raises(vdm.VdmError):
        vdm.vdm_attention_packed(q[:1].expand(8, 8, 64), q, q, cu)                                       # rows overlap
