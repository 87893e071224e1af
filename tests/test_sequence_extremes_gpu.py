"""Token-sequence operators on the GPU at the far ends of what their contract allows.
Tolerances are those of test_sequence_gpu.py and test_sequence_routes_gpu.py; what is added stands at its place."""
import numpy as np
import pytest
import torch

import neural_sdf_volume_b200 as vdm
import test_sequence_gpu as S
from oracle import sequence as OS
from test_sequence_gpu import U, close, ints, np64, offsets, randn
from test_sequence_routes_gpu import weighted_tolerance

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- value scales of an 8-bit cache

def scaled(H, D, page, total, sv, seed=20, zero=()):
    """A cache whose value rows have the scale bytes sv [tokens, H] (one sequence); the rows `zero` are zeros as written."""
    c = S.Cached("e4m3", H, D, page, [total], seed=seed)
    c.cache.k_scale.fill_(117)
    for p in range(total):
        c.cache.v_scale[c.tab[0, p // page], :, p % page] = torch.from_numpy(np.asarray(sv[p], np.uint8)).cuda()
    for p in zero:
        c.cache.v[c.tab[0, p // page], :, p % page] = 0
        c.cache.v_scale[c.tab[0, p // page], :, p % page] = 127
    c.rows["k"], c.rows["v"] = (OS.dequantise(t.cpu().numpy(), s.cpu().numpy()) for t, s in
                                ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)))
    return c


def check_scaled(c, q, new=1, scale=None):
    """Weights are fp16 at 2^12 times their share of 2^M, M at most the largest of score + value exponent: a rounding moves
    a weight by 2^-11 of itself, or by 2^-37 of 2^M where that is more; codes are at most 448.  M, up to 220 beside the
    score, is rounded once a part, and so is a score + value exponent that a sum's term is taken back from: factors of
    1 + 220 ln 2 u of a weight and 1 + (2 * 120 + 2 |score|) ln 2 u of a term, the second's |score| in d."""
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    k, v = c.sequence("k", 0), c.sequence("v", 0)
    got, lse = vdm.vdm_attention_paged(q, c.cache, offsets([new]), c.kv_len, c.table, want_lse=True, scale=sc)
    want, wl = OS.attention(np64(q), k, v, True, sc)
    G = q.shape[1] // k.shape[1]
    e = np.stack([c.cache.v_scale[c.tab[0, p // c.page], :, p % c.page].cpu().numpy() for p in range(len(k))]).astype(float) - 127
    e[(v == 0).all(-1)] = -100
    n = len(k)
    for i in range(new):
        m = n - new + i + 1
        tol = weighted_tolerance(np64(q)[i:i + 1], k[:m], v[:m], sc, 2.0 ** -11 + 160 * U)
        s = np.einsum("hd,khd->kh", np64(q)[i], np.repeat(k[:m], G, 1)) * sc
        top = np.exp(s + np.repeat(e[:m], G, 1) * np.log(2) - wl[i]).max(0)          # [Hq], 2^M over the row's sum
        close(got[i:i + 1], want[i:i + 1], tol + m * 448 * 2.0 ** -37 * top[None, :, None], f"row {i}")
    d = (q.shape[-1] + 8) * U * sc * np.einsum("qhd,khd->qhk", np.abs(np64(q)), np.abs(np.repeat(k, G, 1))).max()
    close(lse, wl, 2 * d + 170 * U + 2.0 ** -20 + (n + 16) * U + 4 * U * np.abs(np.where(np.isfinite(wl), wl, 0)), "lse")
    return got, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("a, b", [(27, 246), (246, 27), (57, 197), (27, 27), (246, 246)])
@pytest.mark.parametrize("ahead", [0.0, 8.0, -8.0])
def test_two_keys_at_both_ends_of_the_value_scales(D, a, b, ahead):
    """Both count in the sum, whatever their values' scales are: equal scores, or either key ahead."""
    c = scaled(2, D, 16, 2, [[a, a], [b, b]])
    c.cache.k.zero_()
    c.cache.k[c.tab[0, 0], :, 0, 0] = 0x38                           # 1.0, at scale 2^-10
    c.rows["k"] = OS.dequantise(c.cache.k.cpu().numpy(), c.cache.k_scale.cpu().numpy())
    q = torch.zeros(1, 8, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = ahead * 2.0 ** 10
    got, lse = check_scaled(c, q, scale=1.0)
    if ahead == 0.0:
        close(lse, np.full((1, 8), np.log(2)), 2.0 ** -20)


@pytest.mark.parametrize("D, Hq, Hk", [(64, 8, 2), (128, 8, 2), (128, 16, 1)])
@pytest.mark.parametrize("total, new", [(33, 1), (900, 1), (900, 5), (20001, 1)])     # a step, warps, a cluster's rows, parts
def test_value_scales_over_their_whole_range(D, Hq, Hk, total, new):
    sv = np.random.default_rng(total).integers(27, 245, (total, Hk))
    c = scaled(Hk, D, 64, total, sv)
    q = randn(21, new, Hq, D)
    _, lse = check_scaled(c, q, new)
    c.cache.v_scale.fill_(127)                                       # the sums have nothing to do with the values
    _, near = vdm.vdm_attention_paged(q, c.cache, offsets([new]), c.kv_len, c.table, want_lse=True)
    close(lse, np64(near), (2 * 170 + 2 * (total + 16)) * U + 2.0 ** -19 + 2 * U * np.abs(np64(near)).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-45, -60, -95])
@pytest.mark.parametrize("zero", [[0], list(range(40)), [450], list(range(0, 900, 2))])
def test_zero_value_rows_beside_small_ones(D, e, zero):
    """A row of zeros has the scale 2^0 whatever its neighbours' are; it must not push their weights below fp16."""
    sv = np.full((900, 2), 127 + e)
    check_scaled(scaled(2, D, 16, 900, sv, zero=zero), randn(22, 1, 8, D))


def test_sums_when_scores_rise_and_fall_by_hundreds():
    """Scores from far below to far above the first keys': the reference of the sum follows."""
    for order in (1, -1):
        c = scaled(1, 64, 16, 600, np.random.default_rng(3).integers(60, 190, (600, 1)))
        c.cache.k.zero_()
        for p in range(600):
            c.cache.k[c.tab[0, p // 16], 0, p % 16, 0] = int(OS.e4m3_encode(float((p - 300) * order) / 1.5))
        c.rows["k"] = OS.dequantise(c.cache.k.cpu().numpy(), c.cache.k_scale.cpu().numpy())
        q = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
        q[0, :, 0] = torch.tensor([2.0 ** 10, 2.0 ** 11, -2.0 ** 11, 1.0])
        check_scaled(c, q, scale=1.0)


# ----------------------------------------------------------------- layouts

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [20, 1500])
def test_keys_and_values_in_different_orders(D, n):
    """Head-major keys beside token-major values and the other way: the same kernel, the same bits."""
    q, k, v = randn(1, n, 8, D), randn(2, n, 2, D), randn(3, n, 2, D)
    hm = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    want = vdm.vdm_attention_packed(q, k, v, offsets([n]))
    assert torch.equal(vdm.vdm_attention_packed(q, hm(k), v, offsets([n])), want)
    assert torch.equal(vdm.vdm_attention_packed(q, k, hm(v), offsets([n])), want)


# ----------------------------------------------------------------- offsets

def inside(shape, dtype):
    """A tensor in the middle of a larger one, and whether what surrounds it is as it was."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * 65536,), 7.0, device="cuda", dtype=dtype)
    return whole[65536:65536 + n].view(shape), lambda: bool((whole[:65536] == 7.0).all() and (whole[65536 + n:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", [[0, 40, 20], [10, 5, 20], [40, 60, 0, 40], [0, 30, 60, 0, 0], [-9, 500, 3, -1, 70, 64], [900, 0, 900, 0, 900]])
@pytest.mark.parametrize("keys", [64, 3000, 40000])                  # one part of the keys, or several
def test_offsets_that_decrease_touch_nothing_outside(dtype, cu, keys):
    """What they mean is not specified; memory around the tensors stays as it was, and what is written is an average of values."""
    T, B = 64, len(cu) - 1
    q = randn(1, T, 8, 64, dtype=dtype)
    out, untouched = inside((T, 8, 64), S.DT[dtype])
    k, v = randn(2, keys, 2, 64, dtype=dtype), randn(3, keys, 2, 64, dtype=dtype)
    top = float(v.abs().max())
    vdm.vdm_attention_packed(q, k, v, ints(cu), ints([x * keys // 64 for x in cu]), causal=False, out=out)
    vdm.vdm_attention_packed(q, k, v, ints(cu), ints([0, keys] * B)[:B + 1].contiguous(), causal=True, out=out)
    vdm.vdm_attention_status()
    assert untouched() and (((out.abs() <= top * 1.01) | (out == 7.0)).all())
    c = S.Cached("e4m3", 2, 64, 16, [min(keys, 3000)] * B, seed=2)
    vdm.vdm_attention_paged(q, c.cache, ints(cu), c.kv_len, c.table, out=out)
    vdm.vdm_attention_status()
    (rk, ku), (rv, vu) = inside((T, 2, 64), S.DT[dtype]), inside((T, 2, 64), S.DT[dtype])
    vdm.vdm_cache_read(c.cache, c.kv_len, c.table, ints(cu), out=(rk, rv))
    vdm.vdm_cache_write(c.cache, rk, rv, ints(cu), c.kv_len, c.table)
    torch.cuda.synchronize()
    assert untouched() and ku() and vu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens, keys", [([40, 50], 60), ([3, 1], 30000), ([1], 40000)])
def test_batches_of_fixed_size_repeat_the_last_offset(dtype, lens, keys):
    """Unused entries change nothing, whatever the route."""
    q, kv = randn(1, sum(lens) + 3, 8, 64, dtype=dtype), randn(2, keys * len(lens), 4, 64, dtype=dtype)
    cu, ck = [0, *np.cumsum(lens).tolist()], [keys * i for i in range(len(lens) + 1)]
    k, v, n = kv[:, :2], kv[:, 2:], sum(lens)
    want = vdm.vdm_attention_packed(q, k, v, ints(cu), ints(ck), causal=False)
    for extra in (1, 40):
        got = vdm.vdm_attention_packed(q, k, v, ints(cu + cu[-1:] * extra), ints(ck + ck[-1:] * extra), causal=False)
        tol, _ = S.tolerance(np64(q), np64(k), np64(v), np64(want), 0.125, dtype)
        close(got[:n], np64(want)[:n], 2 * tol[:n])


# ----------------------------------------------------------------- calls that give up

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind, new, total", [("packed", 2000, 2000), ("bf16", 520, 5000), ("e4m3", 520, 5000)])
def test_a_call_that_gives_up_leaves_nan(D, kind, new, total):
    """A withheld signal: every row of out and lse says that it is no result, also where parts of the keys are joined."""
    q = randn(1, new + 3, 8, D)
    out = torch.full((new + 3, 8, D), 7.0, device="cuda", dtype=torch.bfloat16)
    if kind == "packed":
        k, v = randn(2, total, 2, D), randn(3, total, 2, D)
        call = lambda: vdm.vdm_attention_packed(q, k, v, offsets([new]), offsets([total]), want_lse=True, out=out)
    else:
        c = S.Cached(kind, 2, D, 32, [total], seed=1)
        call = lambda: vdm.vdm_attention_paged(q, c.cache, offsets([new]), c.kv_len, c.table, want_lse=True, out=out)
    want, wl = (x.clone() for x in call())
    vdm.vdm_attention_status()
    vdm.vdm_debug_inject(1, 20_000_000)            # cycles of a wait, about 10 ms
    try:
        got, lse = call()
        with pytest.raises(vdm.VdmError) as e:
            vdm.vdm_attention_status()
        assert e.value.status == 5
        assert torch.isnan(got[:new]).all() and torch.isnan(lse[:new]).all() and (got[new:] == 7.0).all()
    finally:
        vdm.vdm_debug_inject(0, 0)
    got, lse = call()
    vdm.vdm_attention_status()
    assert torch.equal(got, want) and torch.equal(lse[:new], wl[:new])


# ----------------------------------------------------------------- smallest calls, and types and strides at their edges

@pytest.mark.parametrize("dtype, kind", S.KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pages, width", [(0, 3), (4, 0), (0, 0)])
@pytest.mark.parametrize("new", [1, 300])
def test_no_pages_at_all(dtype, kind, D, pages, width, new):
    """A cache without pages, a table without columns: rows without keys; nothing read, nothing written."""
    c = vdm.KVCache.create(pages, 16, 2, D, kind)
    table, cu = torch.zeros(1, width, dtype=torch.int32, device="cuda"), offsets([new])
    q, out = randn(1, new + 1, 4, D, dtype=dtype), torch.full((new + 1, 4, D), 7.0, device="cuda", dtype=S.DT[dtype])
    got, lse = vdm.vdm_attention_paged(q, c, cu, ints([width * 16]), table, out=out, want_lse=True, causal=False)
    vdm.vdm_attention_status()
    if width == 0:
        assert (got[:new] == 0).all() and torch.isneginf(lse[:new]).all()
    else:                                            # positions without a page are zeros: weights, but no values
        assert (got[:new] == 0).all()
    assert (out[new:] == 7.0).all()
    x = randn(2, new, 2, D, dtype=dtype)
    vdm.vdm_cache_write(c, x, x, cu, ints([width * 16]), table)
    k, v = (torch.full_like(x, 5.0) for _ in "kv")
    vdm.vdm_cache_read(c, ints([min(new, width * 16)]), table, cu, out=(k, v))
    n = min(new, width * 16)
    assert (k[:n] == 0).all() and (v[:n] == 0).all() and (k[n:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 700])
def test_queries_without_keys(dtype, n):
    q, k = randn(1, n, 4, 64, dtype=dtype), randn(2, 0, 2, 64, dtype=dtype)
    got, lse = vdm.vdm_attention_packed(q, k, k, offsets([n]), ints([0, 0]), want_lse=True)
    assert (got == 0).all() and torch.isneginf(lse).all()
    got, lse = vdm.vdm_attention_packed(q, randn(3, 40, 2, 64, dtype=dtype), randn(4, 40, 2, 64, dtype=dtype), offsets([n]), ints([40, 40]), want_lse=True)
    assert (got == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("dtype", [None, torch.float32, torch.bfloat16])
def test_cache_read_into_tensors_of_its_own(kind, dtype):
    """The tensors that a read allocates hold the cache's rows, keys and values, in the type asked for."""
    if kind != "e4m3" and dtype not in (None, S.DT.get(kind)):
        with pytest.raises(vdm.VdmError):
            vdm.vdm_cache_read(vdm.KVCache.create(1, 16, 2, 64, kind), ints([3]), ints([[0]]), offsets([3]), total=3, dtype=dtype)
        return
    total = [33, 1, 70]
    c = S.Cached(kind, 3, 64, 16, total, seed=9)
    if kind == "e4m3":                               # the codes under their own type
        c.cache = vdm.KVCache(c.cache.k.view(torch.float8_e4m3fn), c.cache.v.view(torch.float8_e4m3fn), c.cache.k_scale, c.cache.v_scale)
    k, v = vdm.vdm_cache_read(c.cache, c.kv_len, c.table, offsets(total), total=sum(total), dtype=dtype)
    want_type = dtype or (torch.bfloat16 if kind == "e4m3" else S.DT[kind])
    for got, n in ((k, "k"), (v, "v")):
        want = torch.from_numpy(np.concatenate([c.sequence(n, b) for b in range(len(total))])).to(want_type)
        assert got.dtype is want_type and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_that_do_not_count(dtype):
    """One token, or one head: its stride may be anything."""
    for T, H in ((1, 4), (6, 1), (1, 1)):
        q, k, v = (randn(s, T, H, 64, dtype=dtype) for s in (1, 2, 3))
        odd = lambda x: x.as_strided(x.shape, (x.stride(0) if T > 1 else 3, x.stride(1) if H > 1 else 5, 1))
        want = vdm.vdm_attention_packed(q, k, v, offsets([T]))
        assert torch.equal(vdm.vdm_attention_packed(odd(q), odd(k), odd(v), offsets([T])), want)
        g = torch.ones(64, device="cuda")
        assert torch.equal(vdm.vdm_qk_norm_rope(odd(q), odd(k), q_gain=g)[0], vdm.vdm_qk_norm_rope(q, k, q_gain=g)[0])
    q, k, v = randn(1, 900, 4, 64), randn(2, 900, 1, 64), randn(3, 900, 1, 64)         # large tiles, one key head
    one = lambda x: x.as_strided(x.shape, (64, 8, 1))
    assert torch.equal(vdm.vdm_attention_packed(q, one(k), one(v), offsets([900])), vdm.vdm_attention_packed(q, k, v, offsets([900])))


@pytest.mark.parametrize("inter", [False, True])
def test_positions_below_zero(inter):
    x, rope = randn(1, 4, 3, 64, dtype="f32"), vdm.Rope.make(64, interleaved=inter)
    pos = ints([-1, -5000, -2 ** 31, 7])
    got, _ = vdm.vdm_qk_norm_rope(x, None, pos, rope)
    want = OS.norm_rope(np64(x), None, 0, np64(pos), np64(rope.inv_freq), inter)
    close(got, want, 24 * U * np.abs(np64(x)).max() * 2)


def test_heads_on_one_side_alone():
    x, rope, pos = randn(1, 5, 4, 64), vdm.Rope.make(64), torch.arange(5, dtype=torch.int32, device="cuda")
    q, k = vdm.vdm_qk_norm_rope(x[:, :0], x, pos, rope)
    assert q.shape == (5, 0, 64) and torch.equal(k, vdm.vdm_qk_norm_rope(x, None, pos, rope)[0])
    q, k = vdm.vdm_qk_norm_rope(x, x[:, :0], pos, rope)
    assert k.shape == (5, 0, 64) and torch.equal(q, vdm.vdm_qk_norm_rope(x, None, pos, rope)[0])
