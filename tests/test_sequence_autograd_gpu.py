"""Token-sequence calls beside autograd and threads: what would have to be differentiated is refused, whichever tensor asks for it."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import neural_sdf_volume_b200 as vdm
from test_sequence_gpu import Cached, ints, offsets, randn

pytestmark = pytest.mark.gpu


def calls():
    """Name of a tensor -> a call of it, all others plain."""
    q, k, v = (randn(s, 5, 4, 64) for s in (1, 2, 3))
    pos, cu, g = torch.arange(5, dtype=torch.int32, device="cuda"), offsets([5]), torch.ones(64, device="cuda")
    c = Cached("bf16", 4, 64, 16, [5])
    rope = lambda f: vdm.Rope(f)
    f = vdm.Rope.make(64).inv_freq
    paged = lambda x=q, ck=c.cache.k, cv=c.cache.v: vdm.vdm_attention_paged(x, vdm.KVCache(ck, cv), cu, c.kv_len, c.table)
    return {
        "inv_freq": (f, lambda x: vdm.vdm_qk_norm_rope(q, None, pos, rope(x))),
        "norm q": (q, lambda x: vdm.vdm_qk_norm_rope(x, None, pos, rope(f))),
        "norm k": (k, lambda x: vdm.vdm_qk_norm_rope(q, x, pos, rope(f))),
        "gain": (g, lambda x: vdm.vdm_qk_norm_rope(q, k, pos, rope(f), q_gain=x)),
        "packed q": (q, lambda x: vdm.vdm_attention_packed(x, k, v, cu)),
        "packed v": (v, lambda x: vdm.vdm_attention_packed(q, k, x, cu)),
        "paged q": (q, lambda x: paged(x)),
        "cache k": (c.cache.k, lambda x: paged(ck=x)),
        "cache v": (c.cache.v, lambda x: paged(cv=x)),
        "read": (c.cache.k, lambda x: vdm.vdm_cache_read(vdm.KVCache(x, c.cache.v), c.kv_len, c.table, cu, total=5)),
        "write": (k, lambda x: vdm.vdm_cache_write(c.cache, x, v, cu, c.kv_len, c.table)),
        "written": (c.cache.v, lambda x: vdm.vdm_cache_write(vdm.KVCache(c.cache.k, x), k, v, cu, c.kv_len, c.table)),
    }


NAMES = ["inv_freq", "norm q", "norm k", "gain", "packed q", "packed v", "paged q", "cache k", "cache v", "read", "write", "written"]


@pytest.mark.parametrize("name", NAMES)
def test_gradients_are_refused(name):
    x, call = calls()[name]
    call(x)
    y = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(y)
    with torch.no_grad():
        call(y)


@pytest.mark.parametrize("name", NAMES)
def test_tangents_are_refused(name):
    x, call = calls()[name]
    with fw.dual_level():
        y = fw.make_dual(x.clone(), torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            call(y)
        call(fw.unpack_dual(y).primal)


@pytest.mark.parametrize("name", ["norm", "packed", "paged", "write", "read"])
def test_tensors_written_in_place_tell_a_graph_that_kept_them(name):
    """A product that has kept a factor for its backward pass finds it changed, as after torch's own in-place operations."""
    q, k = randn(1, 5, 4, 64), randn(2, 5, 4, 64)
    c = Cached("bf16", 4, 64, 16, [5])
    cu, x = offsets([5]), torch.zeros(5, 4, 64, device="cuda", dtype=torch.bfloat16)
    target, call = {
        "norm": (x, lambda: vdm.vdm_qk_norm_rope(q, k, q_gain=torch.ones(64, device="cuda"), k_out=x)),
        "packed": (x, lambda: vdm.vdm_attention_packed(q, k, k, cu, out=x)),
        "paged": (x, lambda: vdm.vdm_attention_paged(q, c.cache, cu, c.kv_len, c.table, out=x)),
        "write": (c.cache.v, lambda: vdm.vdm_cache_write(c.cache, q, k, cu, c.kv_len, c.table)),
        "read": (x, lambda: vdm.vdm_cache_read(c.cache, c.kv_len, c.table, cu, out=(torch.empty_like(x), x))),
    }[name]
    w = torch.ones((), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = (target * w).sum()
    before = target._version
    call()
    assert target._version > before
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():                     # no versions there
        z = torch.empty_like(x)
        vdm.vdm_attention_packed(q, k, k, cu, out=z)
    vdm.vdm_attention_packed(q, k, k, cu, out=z)


def test_other_threads_run_while_a_launch_waits():
    """More calls than a stream's queue holds, behind a second of other work: a thread that only counts goes on meanwhile."""
    import threading
    import time
    q, cu = randn(1, 5, 4, 64), offsets([5])
    f = lambda: vdm.vdm_attention_packed(q, q, q, cu, out=out)
    out = torch.empty_like(q)
    f()
    torch.cuda.synchronize()
    gap, stop = [0.0], threading.Event()

    def count():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0], last = max(gap[0], now - last), now

    t = threading.Thread(target=count)
    t.start()
    try:
        torch.cuda._sleep(2_000_000_000)             # cycles: a second
        start = time.perf_counter()
        for _ in range(4000):
            f()
        waited = time.perf_counter() - start
    finally:
        stop.set()
        t.join()
    torch.cuda.synchronize()
    assert waited > 0.6, f"the queue held all of them ({waited:.3f} s)"
    assert gap[0] < 0.4, f"held up for {gap[0]:.3f} s"
