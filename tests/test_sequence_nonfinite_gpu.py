"""Attention over values with infinities and NaN among them, on every route: what a query sees reaches it as its formula
says (infinity, or NaN where signs mix), what it does not see has no influence, and neither makes a call slow.  Finite
elements at the tolerances of test_sequence_gpu.py."""
import numpy as np
import pytest
import torch

import neural_sdf_volume_b200 as vdm
import test_sequence_gpu as S
from oracle import sequence as OS
from test_sequence_gpu import U, close, np64, offsets, randn

pytestmark = pytest.mark.gpu


def sprinkle(x, share, seed, kinds=(float("nan"), float("inf"), -float("inf"))):
    r = np.random.default_rng(seed)
    hit = torch.from_numpy(r.random(tuple(x.shape)) < share).cuda()
    what = torch.tensor(kinds, device="cuda")[torch.from_numpy(r.integers(0, len(kinds), tuple(x.shape))).cuda()].to(x.dtype)
    return torch.where(hit, what, x)


def same(got, lse, want, wl, q, k, v, scale, dtype):
    tol, ltol = S.tolerance(q, k, v, want, scale, dtype)
    g, fin = np64(got), np.isfinite(want)
    assert np.array_equal(np.isnan(g), np.isnan(want)), "NaN elsewhere"
    assert np.array_equal(g[np.isinf(want)], want[np.isinf(want)]), "infinities"
    tol = np.broadcast_to(tol, want.shape)
    assert (np.abs(g[fin] - want[fin]) <= tol[fin]).all()
    close(lse, wl, ltol + 4 * U * np.abs(np.where(np.isfinite(wl), wl, 0)), "lse")


def check(dtype, D, Hq, Hk, nq, nk, causal, share, seed, **kw):
    q, k = randn(seed, sum(nq), Hq, D, dtype=dtype), randn(seed + 1, sum(nk), Hk, D, dtype=dtype)
    v = sprinkle(randn(seed + 2, sum(nk), Hk, D, dtype=dtype), share, seed, **kw)
    got, lse = vdm.vdm_attention_packed(q, k, v, offsets(nq), offsets(nk), causal=causal, want_lse=True)
    vdm.vdm_attention_status()
    with np.errstate(invalid="ignore"):
        want, wl = OS.packed(np64(q), np64(k), np64(v), np.cumsum([0, *nq]), np.cumsum([0, *nk]), causal, D ** -0.5)
    same(got, lse, want, wl, np64(q), np64(k), np64(v), D ** -0.5, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("share", [3e-5, 2e-4, 0.02])
@pytest.mark.parametrize("Hq, Hk, nq, nk", [
    (8, 2, [700, 517], [700, 517]), (3, 3, [641, 130], [641, 130]), (5, 1, [900], [300]), (2, 2, [600], [1100])])
def test_large_tiles(D, causal, share, Hq, Hk, nq, nk):
    check("bf16", D, Hq, Hk, nq, nk, causal, share, seed=int(D + 100 * Hq + 1e5 * share))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", [float("nan"), float("inf"), -float("inf")])
def test_large_tiles_one_kind(D, kind):
    check("bf16", D, 4, 4, [800], [800], True, 1e-3, seed=D, kinds=(kind,))
    check("bf16", D, 4, 4, [800], [800], True, 1.1, seed=D, kinds=(kind,))          # all of them


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq, Hk, nq, nk", [(8, 2, [3, 1, 5], [90, 40, 77]), (4, 4, [16, 9], [16, 200]), (16, 1, [2], [3000]), (2, 2, [7], [4])])
def test_few_rows(dtype, D, Hq, Hk, nq, nk):
    for causal in (True, False):
        for share in (1e-3, 0.05):
            check(dtype, D, Hq, Hk, nq, nk, causal, share, seed=D + Hq)


@pytest.mark.parametrize("dtype, kind", S.KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new, total", [([300, 33], [700, 400]), ([5, 3, 1], [500, 3, 90]), ([8], [20001]), ([520], [5000])])
def test_paged(dtype, kind, D, new, total):
    """(8 rows over 20001 keys: several blocks of a cluster, and parts of the keys.)"""
    c = S.Cached(kind, 2, D, 32, total, seed=4)
    if kind == "e4m3":
        hit = torch.from_numpy(np.random.default_rng(7).random(tuple(c.cache.v.shape)) < 1e-3).cuda()
        c.cache.v[hit] = 255
        c.rows["v"] = OS.dequantise(c.cache.v.cpu().numpy(), c.cache.v_scale.cpu().numpy())
    else:
        c.cache.v = sprinkle(c.cache.v, 1e-3, 7)
        c.rows["v"] = np64(c.cache.v)
    q = randn(5, sum(new), 8, D, dtype=dtype)
    got, lse = vdm.vdm_attention_paged(q, c.cache, offsets(new), c.kv_len, c.table, want_lse=True)
    vdm.vdm_attention_status()
    at = 0
    for b, n in enumerate(new):
        k, v, rows = c.sequence("k", b), c.sequence("v", b), slice(at, at + n)
        with np.errstate(invalid="ignore"):
            want, wl = OS.attention(np64(q)[rows], k, v, True, D ** -0.5)
        same(got[rows], lse[rows], want, wl, np64(q), k, v, D ** -0.5, dtype)
        at += n


def milliseconds(f):
    f()
    best = 1e9
    for _ in range(3):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", ["first value", "one query", "a channel", "everywhere", "infinite"])
def test_non_finite_values_do_not_make_a_prompt_slow(D, where):
    """A prompt of 16384 tokens: within four times its own time and half a millisecond, where a row's keys one by one would be
    hundreds of times as long."""
    n = 16384
    q, k, v = randn(1, n, 8, D), randn(2, n, 2, D), randn(3, n, 2, D)
    cu = offsets([n])
    want = vdm.vdm_attention_packed(q, k, v, cu)
    plain = milliseconds(lambda: vdm.vdm_attention_packed(q, k, v, cu))
    if where == "first value":
        v[0, 0, 5] = float("nan")
    elif where == "one query":
        q[700] = float("nan")
    elif where == "a channel":
        v[:, 1, 3] = float("nan")
    else:
        v[:] = float("nan") if where == "everywhere" else float("inf")
    got = vdm.vdm_attention_packed(q, k, v, cu)
    vdm.vdm_attention_status()
    assert milliseconds(lambda: vdm.vdm_attention_packed(q, k, v, cu)) <= 4 * plain + 0.5
    bad = torch.zeros_like(want, dtype=torch.bool)
    if where == "first value":
        bad[:, :4, 5] = True
    elif where == "one query":
        bad[700] = True
    elif where == "a channel":
        bad[:, 4:, 3] = True
    else:
        bad[:] = True
    assert torch.equal(got[~bad], want[~bad])
    assert (torch.isinf if where == "infinite" else torch.isnan)(got[bad]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_non_finite_values_do_not_make_a_step_slow(kind):
    """Three new tokens over 30000: the same."""
    c = S.Cached(kind, 2, 128, 64, [30000], seed=1)
    q = randn(2, 3, 8, 128)
    f = lambda: vdm.vdm_attention_paged(q, c.cache, offsets([3]), c.kv_len, c.table)
    plain = milliseconds(f)
    c.cache.v.fill_(float("nan") if kind == "bf16" else 127)
    assert torch.isnan(f()).all()
    assert milliseconds(f) <= 4 * plain + 0.5
