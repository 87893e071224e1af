"""Token-sequence calls without a GPU: what their Python side hands to the library."""
import ctypes as C
import importlib.util
import os
import types

import pytest
import torch

import neural_sdf_volume_b200 as vdm


# ----------------------------------------------------------------- status of a device that is not the current one

class FakeCuda:
    """Two devices, 0 current, each with a default stream (handle 0) and one of its own."""

    def __init__(self, monkeypatch, error):
        self.current, self.asked = 0, []

        class on:
            def __init__(ctx, dev):
                ctx.dev = torch.device(dev).index

            def __enter__(ctx):
                ctx.was, self.current = self.current, ctx.dev

            def __exit__(ctx, *a):
                self.current = ctx.was

        def status(handle):                      # as the library: the default stream is the current device's
            self.asked.append((self.current, handle))
            return 5 if error == (handle - 1 if handle else self.current) else 0

        monkeypatch.setattr(torch.cuda, "device", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: self.stream(self.current if d is None else torch.device(d).index, 0))
        monkeypatch.setattr(vdm, "_lib", types.SimpleNamespace(vdm_attention_status=status, vdm_last_error=lambda: b"expired",
                                                              vdm_status_string=lambda s: b"timeout"))

    def stream(self, dev, handle):
        return types.SimpleNamespace(device=torch.device("cuda", dev), cuda_stream=handle)


def test_status_is_of_the_streams_device(monkeypatch):
    f = FakeCuda(monkeypatch, error=1)
    vdm.vdm_attention_status()                                   # device 0: fine
    for call in (lambda: vdm.vdm_attention_status(f.stream(1, 0)), lambda: vdm.vdm_attention_status(device="cuda:1"),
                 lambda: vdm.vdm_attention_status(f.stream(1, 2))):
        with pytest.raises(vdm.VdmError) as e:
            call()
        assert e.value.status == 5 and f.asked[-1][0] == 1 and f.current == 0
    with pytest.raises(ValueError):
        vdm.vdm_attention_status(f.stream(0, 0), device="cuda:1")


# ----------------------------------------------------------------- workspace

@pytest.mark.parametrize("Hq, Hk, D, dtype, B, T", [(4, 1, 128, "f32", 1, 3155), (2, 2, 128, "f32", 11, 6711), (8, 1, 64, "f32", 1, 10048),
                                                    (8, 8, 64, "bf16", 6, 9000), (32, 8, 128, "bf16", 1, 1)])
def test_workspace_is_enough_for_either_mask(Hq, Hk, D, dtype, B, T):
    """A causal self-attention may split its keys further than one without a mask."""
    need = []
    for causal in (0, 1):
        n = C.c_size_t(0)
        vdm._check(vdm._lib.vdm_attention_workspace_size(vdm.CAttention(Hq, Hk, D, 0 if dtype == "f32" else 1, causal, 1.0), B, T, T, n))
        need.append(n.value)
        assert vdm.vdm_attention_workspace_size(Hq, Hk, D, dtype, B, T, T, causal=bool(causal)) == n.value
    assert vdm.vdm_attention_workspace_size(Hq, Hk, D, dtype, B, T, T) == max(need)


# ----------------------------------------------------------------- build

@pytest.fixture
def builder(monkeypatch, tmp_path):
    """The build with its tools replaced by one that writes what it is asked for; `fail`: words of a command that fails."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(os.path.dirname(vdm.__file__), "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    for name, path in (("LIB", "libvdm.so"), ("SEQ", "_seq.so"), ("BUILD", "_build")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    b.ran, b.fail = [], None

    def run(cmd, **kw):
        b.ran.append(" ".join(cmd))
        bad = b.fail is not None and b.fail in b.ran[-1]
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w"):
                pass
        return types.SimpleNamespace(returncode=int(bad), stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    return b


def test_c_library_is_built_without_torch(builder, monkeypatch):
    monkeypatch.setattr(builder, "_binding_versions", lambda: None)
    assert builder.build() == builder.LIB and os.path.exists(builder.LIB) and not os.path.exists(builder.SEQ)
    assert not any("seq_binding" in c for c in builder.ran)
    n = len(builder.ran)
    builder.build()
    assert len(builder.ran) == n                                 # nothing left to do


def test_c_library_stands_when_the_binding_fails(builder):
    builder.fail = "seq_binding.cpp"
    with pytest.raises(RuntimeError, match="seq_binding"):
        builder.build()
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.SEQ)


def test_binding_is_built_again_for_another_torch(builder, monkeypatch):
    builder.build()
    n = len(builder.ran)
    builder.build()
    assert os.path.exists(builder.SEQ) and len(builder.ran) == n
    monkeypatch.setattr(builder, "_binding_versions", lambda: "torch 99, python 4")
    builder.build()
    assert any("seq_binding" in c for c in builder.ran[n:])


# ----------------------------------------------------------------- gradients

def test_cache_that_requires_gradients_is_refused():
    c = vdm.KVCache.create(2, 16, 8, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    out = (torch.zeros(1, 8, 64, dtype=torch.bfloat16),) * 2
    c.v.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        vdm.vdm_cache_read(c, i[:1], i[None], i, out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):          # as far as a host tensor gets
        vdm.vdm_cache_read(c, i[:1], i[None], i, out=out)
    c.v = c.v.detach()
    with torch.autograd.forward_ad.dual_level():
        c.k = torch.autograd.forward_ad.make_dual(c.k, torch.ones_like(c.k))
        with pytest.raises(ValueError, match="tangent"):
            vdm.vdm_cache_read(c, i[:1], i[None], i, out=out)


# ----------------------------------------------------------------- caches

def test_both_readers_of_a_cache_refuse_the_same():
    """KVCache.cstruct and the native calls check a cache each for itself."""
    g = vdm.KVCache.create(4, 16, 2, 64, dtype="e4m3", device="cpu")
    b = vdm.KVCache.create(4, 16, 2, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    out = (torch.zeros(1, 2, 64, dtype=torch.bfloat16),) * 2
    native = lambda c: vdm.vdm_cache_read(c, i[:1], i[None], i, out=out)
    for good in (g, b, vdm.KVCache(g.k.view(torch.float8_e4m3fn), g.v.view(torch.float8_e4m3fn), g.k_scale, g.v_scale)):
        good.cstruct()
        with pytest.raises(ValueError, match="CUDA"):
            native(good)
    for bad in (vdm.KVCache(g.k, g.v), vdm.KVCache(g.k, g.v, g.k_scale, g.v_scale.int()), vdm.KVCache(g.k, g.v, g.k_scale[:3], g.v_scale),
                vdm.KVCache(g.k, g.v, g.k_scale, g.v_scale.transpose(0, 1).contiguous().transpose(0, 1)), vdm.KVCache(g.k, g.v[:3], g.k_scale, g.v_scale),
                vdm.KVCache(b.k, b.v.float()), vdm.KVCache(b.k.half(), b.v.half()), vdm.KVCache(b.k[0], b.v[0]),
                vdm.KVCache(b.k[..., ::2], b.v[..., ::2]), vdm.KVCache(b.k.transpose(1, 2), b.v.transpose(1, 2))):
        with pytest.raises(ValueError, match="cache"):
            bad.cstruct()
        with pytest.raises(ValueError, match="cache"):
            native(bad)
