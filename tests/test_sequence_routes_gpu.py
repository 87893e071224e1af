"""Token-sequence operators on the GPU at the sizes that lead to each kernel - large tiles on the
tensor cores, few rows, float32 - and at what is hard on each: non-finite values in unseen
places, layouts, page sizes, scales from end to end of their range, many sequences, caches
beyond 32-bit offsets, split keys.  Tolerances are those of test_sequence_gpu.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import neural_sdf_volume_b200 as vdm
import test_sequence_gpu as S
from oracle import sequence as OS
from test_sequence_gpu import U, close, ints, np64, offsets, randn

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- large tiles

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq, Hk, nq, nk", [
    (8, 2, [1300, 517], None), (4, 4, [2049], None), (3, 1, [700, 0, 1025, 130], None),
    (8, 2, [900, 300], [2100, 1]), (4, 2, [1500], [640])])            # more queries than keys: rows without any
def test_packed_large(D, causal, Hq, Hk, nq, nk):
    S.check_packed("bf16", D, Hq, Hk, nq, nk or nq, causal, seed=D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_paged_large(D, kind, page):
    S.check_paged("bf16", kind, D, 8, 2, page, [400, 33, 700], [1500, 601, 700], seed=page)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq, Hk", [(8, 8), (8, 2)])
def test_packed_large_unseen_values_have_no_influence(D, bad, Hq, Hk):
    """Causal: rows before token j equal those of a run without the bad value, bit for bit where no tile holds it."""
    n, j = 1400, 777
    q, k, v = randn(1, n, Hq, D), randn(2, n, Hk, D), randn(3, n, Hk, D)
    want = vdm.vdm_attention_packed(q, k, v, offsets([n]))
    tol, _ = S.tolerance(np64(q), np64(k), np64(v), np64(want), D ** -0.5, "bf16")
    for where in ("k", "v"):
        x = (k if where == "k" else v).clone()
        x[j, 0, 5] = bad
        got = vdm.vdm_attention_packed(q, x if where == "k" else k, x if where == "v" else v, offsets([n]))
        close(got[:j], np64(want)[:j], 2 * tol[:j], f"rows that do not see the {where}")
        G = Hq // Hk
        if where == "v":                                            # later rows of that head: this dimension alone
            assert not torch.isfinite(got[j:, :G, 5]).any() and torch.isfinite(got[j:, :G, 6]).all()
        close(got[j:, G:], np64(want)[j:, G:], 2 * tol[j:, G:], "other heads")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [600, 9])                           # large tiles, few rows
def test_paged_unseen_values_have_no_influence(kind, new):
    total = 1000
    c = S.Cached(kind, 2, 64, 16, [total], seed=3)
    q = randn(4, new, 8, 64)
    args = (offsets([new]), c.kv_len, c.table)
    want = vdm.vdm_attention_paged(q, c.cache, *args)
    p = total - 4                                                   # seen by the last four queries
    pg, r = c.tab[0, p // 16], p % 16
    c.cache.v[pg, 1, r, 7] = 127 if kind == "e4m3" else float("nan")
    got = vdm.vdm_attention_paged(q, c.cache, *args)
    tol, _ = S.tolerance(np64(q), c.sequence("k", 0), c.sequence("v", 0), np64(want), 0.125, "bf16")
    close(got[:-4], np64(want)[:-4], 2 * tol[:-4])
    assert torch.isnan(got[-4:, 4:, 7]).all() and torch.isfinite(got[-4:, :4]).all()


@pytest.mark.parametrize("n", [30, 1300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_all_keys_of_minus_infinity(n, dtype):
    """Scores of -inf everywhere: empty rows, whatever the kernel."""
    q, v = torch.ones(n, 4, 64, device="cuda", dtype=S.DT[dtype]), randn(1, n, 4, 64, dtype=dtype)
    k = torch.full_like(q, float("-inf"))
    o, l = vdm.vdm_attention_packed(q, k, v, offsets([n]), causal=False, want_lse=True)
    assert (o == 0).all() and torch.isneginf(l).all()
    k[: n // 2] = 0.25                                              # the other half counts alone
    o = vdm.vdm_attention_packed(q, k, v, offsets([n]), causal=False)
    want = np64(v)[: n // 2].mean(0)[None].repeat(n, 0)
    close(o, want, S.tolerance(np64(q), np64(k)[: n // 2], np64(v), want, 0.125, dtype)[0])


def test_packed_more_row_tiles_than_a_grid_dimension():
    """8.5 million queries of one sequence over 64 keys without a preference: every row is the mean of the values."""
    n = 8_500_000
    q, k, v = torch.ones(n, 1, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(64, 1, 64, device="cuda", dtype=torch.bfloat16), randn(1, 64, 1, 64)
    o = vdm.vdm_attention_packed(q, k, v, ints([0, n]), ints([0, 64]), causal=False)
    vdm.vdm_attention_status()
    assert torch.equal(o, o[:1].expand_as(o))
    close(o[:1], np64(v).mean(0)[None], 2.0 ** -8 * np.abs(np64(v)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [20, 1100])
def test_layouts_give_the_same_result(dtype, n):
    """Head-major tensors, slices of a projection and an output view: bit-identical; keys and values laid out differently: near."""
    Hq, Hk, D = 8, 2, 64
    q, k, v = randn(1, n, Hq, D, dtype=dtype), randn(2, n, Hk, D, dtype=dtype), randn(3, n, Hk, D, dtype=dtype)
    cu = offsets([n // 3, n - n // 3])
    want = vdm.vdm_attention_packed(q, k, v, cu)
    hm = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.empty(n, Hq + 3, D, device="cuda", dtype=q.dtype)
    out = wide[:, 1:1 + Hq]
    vdm.vdm_attention_packed(hm(q), hm(k), hm(v), cu, out=out)
    assert torch.equal(out, want)
    fused = torch.cat((q, k, v), 1)
    assert torch.equal(vdm.vdm_attention_packed(fused[:, :Hq], fused[:, Hq:Hq + Hk], fused[:, Hq + Hk:], cu), want)
    tol, _ = S.tolerance(np64(q), np64(k), np64(v), np64(want), D ** -0.5, dtype)
    close(vdm.vdm_attention_packed(q, hm(k), v, cu), np64(want), 2 * tol)


# ----------------------------------------------------------------- few rows

def weighted_tolerance(q, k, v, scale, bits):
    """2^-8 (bf16 output) + weights' rounding and twice the score's error, of sum p |v| / sum p."""
    H, G = k.shape[1], q.shape[1] // k.shape[1]
    s = np.einsum("qhd,khd->hqk", q, np.repeat(k, G, 1)) * scale
    d = (q.shape[-1] + 8) * U * scale * np.einsum("qhd,khd->hqk", np.abs(q), np.abs(np.repeat(k, G, 1))).max()
    p = np.exp(s - s.max(-1, keepdims=True))
    return (2.0 ** -8 + bits + 2 * d + (k.shape[0] + 16) * U) * np.einsum("hqk,khd->qhd", p / p.sum(-1, keepdims=True), np.abs(np.repeat(v, G, 1)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scales", ["smallest", "largest", "sink", "any"])
def test_paged_one_token_value_scales_from_end_to_end(D, scales):
    """8-bit values whose scales lie anywhere in 2^-100 .. 2^119, also where the heaviest keys have the smallest."""
    rng = np.random.default_rng(5)
    n, page, H = 900, 16, 2
    c = S.Cached("e4m3", H, D, page, [n], seed=6)
    sv = {"smallest": np.full((c.P, H, page), 27), "largest": np.full((c.P, H, page), 244),
          "sink": np.full((c.P, H, page), 130), "any": rng.integers(60, 190, (c.P, H, page))}[scales].astype(np.uint8)
    sk = np.full((c.P, H, page), 117, np.uint8)
    codes = np64(c.cache.k.view(torch.float8_e4m3fn))
    if scales == "sink":                                            # the first key: score far above the others', values 2^-60 of theirs
        sv[c.tab[0, 0], :, 0] = 70
    c.cache.v_scale.copy_(torch.from_numpy(sv)), c.cache.k_scale.copy_(torch.from_numpy(sk))
    q = randn(7, 1, 8, D)
    if scales == "sink":
        key = codes[c.tab[0, 0], :, 0] * 2.0 ** -10
        q = torch.from_numpy(np.repeat(key, 4, 0)[None] * (30.0 / (np.repeat(key, 4, 0) ** 2).sum(-1) / D ** -0.5)[None, :, None]).cuda().to(torch.bfloat16)
    c.rows["k"], c.rows["v"] = (OS.dequantise(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)))
    k, v = c.sequence("k", 0), c.sequence("v", 0)
    got, lse = vdm.vdm_attention_paged(q, c.cache, offsets([1]), c.kv_len, c.table, want_lse=True)
    want, wl = OS.attention(np64(q), k, v, True, D ** -0.5)
    close(got, want, weighted_tolerance(np64(q), k, v, D ** -0.5, 2.0 ** -11))
    close(lse, wl, 1e-4 + 4 * U * np.abs(wl))


@pytest.mark.parametrize("dtype, kind", S.KINDS)
@pytest.mark.parametrize("mag", [2.0 ** -70, 2.0 ** 60])
def test_paged_one_token_query_magnitudes(dtype, kind, mag):
    """Queries far from 1 (the kernel of 8-bit caches scales them into fp16): tiny ones weigh all keys alike."""
    c = S.Cached(kind, 2, 64, 16, [300], seed=8)
    q = randn(9, 1, 4, 64, dtype=dtype) * mag
    scale = 0.125 / mag if mag > 1 else 0.125
    got = vdm.vdm_attention_paged(q, c.cache, offsets([1]), c.kv_len, c.table, scale=scale)
    k, v = c.sequence("k", 0), c.sequence("v", 0)
    want, _ = OS.attention(np64(q), k, v, True, scale)
    close(got, want, S.tolerance(np64(q), k, v, want, scale, dtype)[0])


@pytest.mark.parametrize("dtype, kind", S.KINDS)
@pytest.mark.parametrize("D, Hq, Hk", [(64, 4, 4), (128, 16, 1), (128, 6, 2)])
def test_paged_one_token_of_a_long_context(dtype, kind, D, Hq, Hk):
    """Keys split over blocks and over launches' parts; a workspace of the user's own, and one too small."""
    total = [20001]
    c = S.Cached(kind, Hk, D, 64, total, seed=10)
    q = randn(11, 1, Hq, D, dtype=dtype)
    args = (q, c.cache, offsets([1]), c.kv_len, c.table)
    got, lse = vdm.vdm_attention_paged(*args, want_lse=True)
    k, v = c.sequence("k", 0), c.sequence("v", 0)
    want, wl = OS.attention(np64(q), k, v, True, D ** -0.5)
    tol, ltol = S.tolerance(np64(q), k, v, want, D ** -0.5, dtype)
    close(got, want, tol)
    close(lse, wl, ltol + 4 * U * np.abs(wl))
    n = vdm.vdm_attention_workspace_size(Hq, Hk, D, dtype, 1, 1, c.width * 64)
    assert n > 0
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    assert torch.equal(vdm.vdm_attention_paged(*args, workspace=ws), got)
    with pytest.raises(vdm.VdmError):
        vdm.vdm_attention_paged(*args, workspace=ws[:-1])


@pytest.mark.parametrize("dtype, kind", S.KINDS)
def test_paged_many_sequences(dtype, kind):
    """Hundreds of sequences, empty ones and chunks among single tokens."""
    rng = np.random.default_rng(12)
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 1, 3], 400)]
    total = [n + int(x) for n, x in zip(new, rng.integers(0, 40, 400))]
    S.check_paged(dtype, kind, 64, 4, 2, 16, new, total, seed=13)


def test_packed_many_long_and_empty_sequences():
    lens = [0, 300, 0, 0, 900] + [0] * 30 + [200, 1, 0]              # more than 32: found by the search
    S.check_packed("bf16", 128, 4, 2, lens, lens, True)
    S.check_packed("f32", 64, 4, 4, lens, lens, False)
    S.check_packed("bf16", 64, 2, 2, [0] * 1100 + [70] + [0] * 1100, [0] * 1100 + [70] + [0] * 1100, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 9, 16, 17])
def test_packed_few_queries_of_every_group_size(dtype, G):
    S.check_packed(dtype, 64, 2 * G, 2, [1, 2, 0, 1], [200, 70, 5, 33], True, seed=G)


# ----------------------------------------------------------------- norm + rotation, cache

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, T, Hq, Hk, rot, inter", [
    (64, 3001, 3, 1, 64, True), (64, 3001, 3, 1, 40, False), (128, 1203, 9, 2, 128, False), (128, 1203, 9, 2, 20, False),
    (64, 601, 1, 0, 6, True), (128, 700, 41, 7, 0, False), (128, 2, 41, 7, 96, False), (64, 1500, 16, 16, 64, False)])
def test_norm_rope_many_tokens(dtype, D, T, Hq, Hk, rot, inter):
    S.test_norm_rope(dtype, D, T, Hq, Hk, rot, inter)


def test_norm_rope_one_side_without_gain_keeps_its_values():
    """Elements that are neither normalised nor rotated pass through as they are, infinities too; NaN stays NaN."""
    x = randn(1, 900, 6, 64)
    x[3, 4, 50], x[7, 5, 63] = float("nan"), float("inf")
    rope, pos = vdm.Rope.make(32), torch.arange(900, dtype=torch.int32, device="cuda")
    _, k = vdm.vdm_qk_norm_rope(x[:, :4], x[:, 4:], pos, rope, q_gain=torch.ones(64, device="cuda"))
    assert torch.allclose(k[..., 32:], x[:, 4:, 32:], rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype, kind", S.KINDS)
@pytest.mark.parametrize("H, D", [(9, 64), (33, 128), (1, 128)])
def test_cache_many_heads_and_sequences(dtype, kind, H, D):
    rng = np.random.default_rng(H)
    new = [int(x) for x in rng.choice([0, 1, 2, 9], 70)]
    total = [n + int(x) for n, x in zip(new, rng.integers(0, 20, 70))]
    S.test_cache_write(dtype, kind, H, D, 16, new, total)
    S.test_cache_read(dtype, kind, H, D, 16, total)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_cache_beyond_32_bit_offsets(kind):
    """Pages behind 4 GiB of keys: write, read and both attention kernels."""
    H, D, page = 8, 128, 256
    P = (5 << 30) // (H * page * D * (2 if kind == "bf16" else 1))
    t = torch.bfloat16 if kind == "bf16" else torch.uint8
    k, v = (torch.empty((P, H, page, D), device="cuda", dtype=t) for _ in "kv")
    sc = [torch.full((P, H, page), 127, device="cuda", dtype=torch.uint8) for _ in "kv"] if kind == "e4m3" else [None, None]
    cache = vdm.KVCache(k, v, *sc)
    table = ints([[P - 1, 0, P - 2, 1]])
    n = 900
    x = randn(1, n, 2 * H, D)
    vdm.vdm_cache_write(cache, x[:, :H], x[:, H:], offsets([n]), ints([n]), table)
    rk, rv = vdm.vdm_cache_read(cache, ints([n]), table, offsets([n]), total=n)
    if kind == "bf16":
        assert torch.equal(rk, x[:, :H]) and torch.equal(rv, x[:, H:])
    else:
        codes, s = OS.quantise(np64(x[800:, :H]))
        assert np.array_equal(np64(rk[800:]), OS.dequantise(codes, s))
    q = randn(2, n, H, D)
    whole = vdm.vdm_attention_paged(q, cache, offsets([n]), ints([n]), table)
    near = vdm.vdm_attention_packed(q, rk, rv, offsets([n]))
    tol, _ = S.tolerance(np64(q), np64(rk), np64(rv), np64(near), D ** -0.5, "bf16")
    close(whole, np64(near), 2 * tol)
    one = vdm.vdm_attention_paged(q[-1:], cache, offsets([1]), ints([n]), table)
    close(one, np64(near)[-1:], 2 * tol[-1:])


# ----------------------------------------------------------------- failure detection, graphs, gradients

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["packed", "bf16", "e4m3"])
def test_withheld_signal_times_out_and_later_calls_run(D, kind):
    """A tensor-core attention whose scores are never announced gives up its waits; the status says so once."""
    n = 2000                                       # enough for the tensor-core kernel
    q = randn(1, n, 8, D)
    if kind == "packed":
        k, v = randn(2, n, 2, D), randn(3, n, 2, D)
        call = lambda: vdm.vdm_attention_packed(q, k, v, offsets([n]))
    else:
        c = S.Cached(kind, 2, D, 32, [n], seed=1)
        call = lambda: vdm.vdm_attention_paged(q, c.cache, offsets([n]), c.kv_len, c.table)
    want = call()
    vdm.vdm_attention_status()
    vdm.vdm_debug_inject(1, 20_000_000)            # cycles of a wait, about 10 ms
    try:
        call()
        with pytest.raises(vdm.VdmError) as e:
            vdm.vdm_attention_status()
        assert e.value.status == 5 and "bounded wait" in str(e.value)
    finally:
        vdm.vdm_debug_inject(0, 0)
    vdm.vdm_attention_status()
    assert torch.equal(call(), want)
    vdm.vdm_attention_status()


def test_first_calls_of_a_process_may_be_captured():
    """A fresh process whose first call of each operator is inside a capture."""
    code = """
import torch, neural_sdf_volume_b200 as vdm
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device='cuda')
n = 1500
q, k = torch.randn(n, 8, 128, device='cuda').bfloat16(), torch.randn(n, 2, 128, device='cuda').bfloat16()
qf, kf, cu, one, ln, table = q.float(), k.float(), i32([0, n]), i32([0, 1]), i32([n]), i32([list(range(50))])
cache, rope, pos, g1 = vdm.KVCache.create(64, 32, 2, 128, 'e4m3'), vdm.Rope.make(64), torch.arange(n, dtype=torch.int32, device='cuda'), torch.ones(128, device='cuda')
torch.cuda.synchronize()
for f in (lambda: vdm.vdm_qk_norm_rope(q, k, pos, rope, q_gain=g1)[0], lambda: vdm.vdm_cache_write(cache, k, k, cu, ln, table),
          lambda: vdm.vdm_cache_read(cache, ln, table, cu, total=n)[0], lambda: vdm.vdm_attention_packed(q, k, k, cu),
          lambda: vdm.vdm_attention_paged(q[:1], cache, one, ln, table), lambda: vdm.vdm_attention_packed(qf, kf, kf, cu)):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = f()
    g.replay()
    torch.cuda.synchronize()
    w = f()
    assert o is None or torch.equal(o, w)
vdm.vdm_attention_status()
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_graphs_and_an_eager_call_at_once():
    """Captured calls keep workspaces of their own: two graphs replayed on two streams beside an eager call."""
    c = S.Cached("e4m3", 1, 128, 64, [20000], seed=14)
    q = [randn(s, 1, 16, 128) for s in (1, 2, 3)]
    args = (c.cache, offsets([1]), c.kv_len, c.table)
    want = [vdm.vdm_attention_paged(x, *args) for x in q]
    torch.cuda.synchronize()
    graphs = []
    for x in q[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = vdm.vdm_attention_paged(x, *args)
        graphs.append((g, o))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(a):
            graphs[0][0].replay()
        with torch.cuda.stream(b):
            graphs[1][0].replay()
        eager = vdm.vdm_attention_paged(q[2], *args)
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], want[0]) and torch.equal(graphs[1][1], want[1]) and torch.equal(eager, want[2])


def test_tensors_that_require_gradients_are_refused():
    q = randn(1, 4, 2, 64).requires_grad_()
    cu = offsets([4])
    with pytest.raises(ValueError, match="gradient"):
        vdm.vdm_attention_packed(q, q, q, cu)
    with pytest.raises(ValueError, match="gradient"):
        vdm.vdm_qk_norm_rope(q.detach(), q_gain=torch.ones(64, device="cuda", requires_grad=True))
    with torch.no_grad():
        vdm.vdm_attention_packed(q, q, q, cu)
