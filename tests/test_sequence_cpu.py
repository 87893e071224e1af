"""Token-sequence operators without a GPU: the oracle against closed forms, the
rotary table, and every refusal of the C entry points (fake pointers: nothing is
launched) and of the Python ones."""
import ctypes as C

import numpy as np
import pytest
import torch

import neural_sdf_volume_b200 as vdm
from oracle import sequence as OS

lib = vdm._lib
P = 0x10000


# ----------------------------------------------------------------- oracle

def test_oracle_codes_equal_torch_conversion():
    x = np.concatenate([np.linspace(-460, 460, 4001), np.linspace(-0.05, 0.05, 2001), OS.E4M3[:127], -OS.E4M3[:127],
                        (OS.E4M3[1:127] + OS.E4M3[:126]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OS.e4m3_encode(x.astype(np.float64)), want)
    assert np.array_equal(OS.e4m3_decode(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("m, e", [(448.0, 0), (448.0001, 1), (224.0, -1), (3.5, -7), (3.51, -6), (0.0, 0), (1e-40, -100), (3.4e38, 119)])
def test_oracle_row_scale(m, e):
    codes, s = OS.quantise_row([m, -m / 3, 0.0])
    assert s == e + 127
    back = OS.dequantise(codes[None], np.array([s]))[0]
    if e > -100:
        assert abs(back[0] - m) <= max(2.0 ** -4 * m, m - 448 * 2.0 ** e)


def test_oracle_special_values():
    codes, s = OS.quantise_row([np.nan, np.inf, 1.0, -np.inf])
    assert (codes[[0, 1, 3]] & 127 == 127).all() and s == 127 - 8 and OS.e4m3_decode(codes[2]) == 256


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(5, 1, 4))
    o, l = OS.attention(np.zeros((3, 2, 4)), rng.normal(size=(5, 1, 4)), v, False, 0.5)
    assert np.allclose(o, v.mean(0)) and np.allclose(l, np.log(5))          # zero queries: the mean
    o, l = OS.attention(rng.normal(size=(5, 2, 4)), rng.normal(size=(5, 1, 4)), v, True, 0.5)
    assert np.allclose(o[0], v[0])                                         # the first query sees the first key
    o, l = OS.attention(rng.normal(size=(7, 2, 4)), rng.normal(size=(5, 1, 4)), v, True, 0.5)
    assert (o[:2] == 0).all() and np.isneginf(l[:2]).all() and np.allclose(o[2], v[0])


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_rotation_is_relative_and_keeps_length(inter):
    rng = np.random.default_rng(1)
    f = vdm.rope_frequencies(8)
    q, k = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))
    dot = lambda i, j: float((OS.norm_rope(q, positions=[i], inv_freq=f, interleaved=inter) *
                              OS.norm_rope(k, positions=[j], inv_freq=f, interleaved=inter)).sum())
    assert np.isclose(dot(3, 11), dot(103, 111))
    assert np.isclose((OS.norm_rope(q, positions=[77], inv_freq=f, interleaved=inter) ** 2).sum(), (q ** 2).sum())


def test_rope_frequencies():
    f = vdm.rope_frequencies(64)
    assert f.dtype == np.float64 and np.allclose(f, 10000.0 ** (-np.arange(32) / 32))
    assert np.allclose(vdm.rope_frequencies(64, factor=4.0), f / 4)
    g = vdm.rope_frequencies(64, factor=8.0, original_length=4096)
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    assert (g <= f + 1e-15).all() and (g >= f / 8 - 1e-15).all() and (np.diff(g) < 0).all()
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, base=0), dict(rot_dim=64, factor=0),
                dict(rot_dim=64, original_length=100, slow_turns=5, fast_turns=5)):
        with pytest.raises(ValueError):
            vdm.rope_frequencies(**bad)


# ----------------------------------------------------------------- C refusals (nothing is launched)

def H(data=P, st=512, sh=64):
    return vdm.CHeads(data, st, sh)


def rope_call(dt=1, T=4, Hq=8, Hk=8, D=64, q=None, k=None, eps=1e-6, rope=None, pos=P):
    q, k = q or H(), k or H()
    return lib.vdm_qk_norm_rope(dt, T, Hq, Hk, D, q, k, None, None, eps, rope, pos, q, k, None)


@pytest.mark.parametrize("status, kw", [
    (1, dict(dt=2)), (2, dict(D=96)), (1, dict(T=-1)), (2, dict(T=1 << 31)), (1, dict(Hq=0, Hk=0)), (1, dict(Hq=-1)),
    (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (1, dict(q=H(0))), (1, dict(k=H(P + 2))), (1, dict(q=H(sh=65))),
    (1, dict(q=H(st=516))), (1, dict(q=H(st=0))), (1, dict(q=H(st=64))), (1, dict(q=H(sh=0))), (1, dict(q=H(st=504))),
    (2, dict(rope=vdm.CRope(130, 0, P, 1.0))), (2, dict(rope=vdm.CRope(66, 0, P, 1.0))), (2, dict(rope=vdm.CRope(3, 0, P, 1.0))),
    (1, dict(rope=vdm.CRope(64, 2, P, 1.0))), (1, dict(rope=vdm.CRope(64, 0, 0, 1.0))), (1, dict(rope=vdm.CRope(64, 0, P, float("inf")))),
    (1, dict(rope=vdm.CRope(64, 0, P, 1.0), pos=None)),
    (0, dict(T=0)),
])
def test_norm_rope_refusals(status, kw):
    assert rope_call(**kw) == status, lib.vdm_last_error()


def cache(dt=2, pages=4, page=16, Hh=8, D=64, k=P, v=P, ks=P, vs=P):
    return vdm.CKvCache(dt, pages, page, Hh, D, k, v, ks, vs)


BAD_CACHES = [(1, dict(dt=3)), (2, dict(D=32)), (2, dict(page=8)), (2, dict(page=48)), (2, dict(page=512)), (1, dict(Hh=0)),
              (1, dict(pages=-1)), (1, dict(k=0)), (1, dict(v=P + 8)), (1, dict(ks=0)), (1, dict(vs=0))]
BAD_CACHES += [(1, dict(ks=P + 8)), (1, dict(vs=P + 1))]             # scales are fetched 16 bytes at a time


@pytest.mark.parametrize("status, kw", BAD_CACHES)
def test_cache_refusals(status, kw):
    c = cache(**kw)
    assert lib.vdm_cache_write(c, 1, H(), H(), 4, P, P, P, 4, 2, None) == status
    assert lib.vdm_cache_read(c, 1, P, P, 4, P, 2, 4, H(), H(), None) == status
    a = vdm.CAttention(8, 8, 64, 1, 1, 0.125)
    assert lib.vdm_attention_paged(a, H(), c, P, P, P, 4, 2, 4, H(), None, None, 0, None) == status


def test_cache_call_refusals():
    w = lambda c=None, dt=1, k=None, v=None, T=4, cu=P, ln=P, tab=P, mp=4, B=2: \
        lib.vdm_cache_write(c or cache(), dt, k or H(), v or H(), T, cu, ln, tab, mp, B, None)
    assert w(dt=5) == 1
    assert w(c=cache(dt=0)) == 2 and w(c=cache(dt=1), dt=0) == 2         # neither 8-bit nor the tensors' type
    assert w(T=-1) == 1 and w(B=-1) == 1 and w(mp=-1) == 1
    assert w(cu=None) == 1 and w(ln=None) == 1 and w(tab=None) == 1
    assert w(k=H(0)) == 1 and w(v=H(st=60)) == 1
    assert w(mp=1 << 28) == 2                                          # positions beyond 32 bits
    assert w(mp=(1 << 27) - 1) == 2                                    # and so near that a tile would be
    assert w(T=0) == 0 and w(B=0, tab=None) == 0 and w(mp=0, tab=None) == 0
    assert lib.vdm_cache_read(cache(), 1, P, P, 4, None, 2, 4, H(), H(), None) == 1
    assert lib.vdm_cache_read(None, 1, P, P, 4, P, 2, 4, H(), H(), None) == 1


def attn(Hq=8, Hk=8, D=64, dt=1, causal=1, scale=0.125):
    return vdm.CAttention(Hq, Hk, D, dt, causal, scale)


@pytest.mark.parametrize("status, kw", [
    (1, dict(Hq=7, Hk=2)), (1, dict(Hq=0)), (1, dict(Hk=0)), (2, dict(D=256)), (1, dict(dt=7)), (1, dict(causal=2)),
    (1, dict(scale=0.0)), (1, dict(scale=-1.0)), (1, dict(scale=float("nan"))), (1, dict(scale=float("inf")))])
def test_attention_parameter_refusals(status, kw):
    n = C.c_size_t(0)
    a = attn(**kw)
    assert lib.vdm_attention_workspace_size(a, 2, 4, 64, n) == status
    assert lib.vdm_attention_packed(a, H(), H(), H(), P, P, 2, 4, 4, H(), None, P, 1 << 40, None) == status
    assert lib.vdm_attention_paged(a, H(), cache(), P, P, P, 4, 2, 4, H(), None, P, 1 << 40, None) == status


def test_attention_call_refusals():
    f = lambda a=None, q=None, k=None, v=None, cq=P, ck=P, B=2, Tq=4, Tk=4, o=None, ws=P, nb=1 << 40: \
        lib.vdm_attention_packed(a or attn(), q or H(), k or H(), v or H(), cq, ck, B, Tq, Tk, o or H(), None, ws, nb, None)
    assert f(cq=None) == 1 and f(ck=None) == 1 and f(q=H(0)) == 1 and f(k=H(0)) == 1 and f(v=H(P + 1)) == 1
    assert f(o=H(0)) == 1 and f(o=H(st=0)) == 1 and f(k=H(st=0)) == 1
    assert f(Tq=-1) == 1 and f(Tk=-1) == 1 and f(B=-1) == 1 and f(Tq=1 << 31) == 2 and f(Tk=1 << 31) == 2
    assert f(Tk=0x7fffffff) == 2 and f(Tq=0x7fffffff) == 2
    assert f(Tq=0) == 0 and f(B=0) == 0
    assert f(a=attn(Hq=64, Hk=1), q=H(st=4096), o=H(st=4096), Tq=1 << 26, B=1) == 2    # rows beyond 32 bits
    assert lib.vdm_attention_packed(None, H(), H(), H(), P, P, 2, 4, 4, H(), None, P, 1 << 40, None) == 1
    # a split over long keys needs a workspace, 256-byte aligned
    n = C.c_size_t(0)
    assert lib.vdm_attention_workspace_size(attn(), 1, 1, 100000, n) == 0 and n.value > 0
    assert f(B=1, Tq=1, Tk=100000, ws=None) == 3 and f(B=1, Tq=1, Tk=100000, nb=n.value - 1) == 3
    assert f(B=1, Tq=1, Tk=100000, ws=P + 16) == 1
    # the cache's heads are the call's
    g = lambda a: lib.vdm_attention_paged(a, H(), cache(), P, P, P, 4, 2, 4, H(), None, P, 1 << 40, None)
    assert g(attn(Hq=8, Hk=4)) == 1 and g(attn(D=128)) == 1
    assert b"cache" in lib.vdm_last_error()
    assert lib.vdm_attention_paged(attn(dt=0), H(), cache(dt=1), P, P, P, 4, 2, 4, H(), None, P, 1 << 40, None) == 2


# ----------------------------------------------------------------- Python refusals

def test_python_refuses_host_tensors_and_bad_tables():
    t = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: vdm.vdm_qk_norm_rope(t), lambda: vdm.vdm_attention_packed(t, t, t, i),
                 lambda: vdm.vdm_cache_write(vdm.KVCache.create(2, 16, 8, 64, device="cpu"), t, t, i, i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        vdm.KVCache.create(2, 24, 8, 64, device="cpu")
    with pytest.raises(ValueError):
        vdm.KVCache.create(2, 16, 8, 64, dtype="fp8", device="cpu")
    c = vdm.KVCache.create(2, 16, 8, 64, dtype="e4m3", device="cpu")
    s = c.cstruct()
    assert (s.dtype, s.num_pages, s.page_size, s.H, s.D) == (2, 2, 16, 8, 64) and (c.k_scale == 127).all()
    for bad in (vdm.KVCache(c.k, c.v), vdm.KVCache(c.k, c.v[:1], c.k_scale, c.v_scale), vdm.KVCache(c.k.int(), c.v.int()),
                vdm.KVCache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            bad.cstruct()
