"""Cases, plain forms and 64-bit definitions of the library's attention-side operators.

Five operators around a set of latent tokens or a token sequence:

  rope    ``vdm_qk_norm_rope``      RMS norm of every query and key head and the rotary position, one pass
  packed  ``vdm_attention_packed``  attention inside packed sequences, grouped heads, causal or full
  write   ``vdm_cache_write``       new keys and values into a paged cache (8-bit with a scale per row, or as is)
  read    ``vdm_cache_read``        a paged cache's tokens back, in order
  paged   ``vdm_attention_paged``   a chunk of new tokens (or a single one) attending to a paged cache

A case names the operator, its sizes and types, and (``lens``) the number that the
sequence lengths follow from, so that the work of a case is known without its data.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PAD = 3          # pages of a cache that no sequence owns


def _lens(case):
    """(new tokens, tokens in the cache or keys) of every sequence."""
    r = random.Random(case["lens"])
    new = [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]
    old = [case["ctx_hi"]] + [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"] - 1)]
    return new, [n + c for n, c in zip(new, old)]


def listed():
    seq = {"lens": 7, "ctx_lo": 0, "ctx_hi": 0}
    return [
        # one new token of an 8-head, 64-wide block: the smallest call, where its latency counts
        {"name": "rope_one_token", "op": "rope", "T": 1, "Hq": 8, "Hk": 8, "D": 64, "dtype": "bf16",
         "rot": 64, "interleaved": False, "scaled": False, "pos0": 1000},
        # a long prompt with grouped heads: part of the head rotated, interleaved pairs, far positions, long-context scaling
        {"name": "rope_prompt", "op": "rope", "T": 16381, "Hq": 32, "Hk": 8, "D": 128, "dtype": "bf16",
         "rot": 96, "interleaved": True, "scaled": True, "pos0": 120000},
        # self-attention over vecsets of different sizes packed together (the token counts of this library's decoders: up to 4096)
        {"name": "packed_vecsets", "op": "packed", "B": 6, "lo": 256, "hi": 4096, "Hq": 8, "Hk": 8, "D": 64,
         "dtype": "bf16", "causal": False, **seq},
        # prompts of different lengths, causal, four query heads to a key head
        {"name": "packed_prompts", "op": "packed", "B": 5, "lo": 1500, "hi": 4096, "Hq": 32, "Hk": 8, "D": 128,
         "dtype": "bf16", "causal": True, **seq},
        # short float32 sequences, odd lengths
        {"name": "packed_f32", "op": "packed", "B": 4, "lo": 1, "hi": 1027, "Hq": 8, "Hk": 4, "D": 64,
         "dtype": "f32", "causal": True, **seq},
        # one step's keys and values of 64 sequences, quantised as they are written
        {"name": "write_step", "op": "write", "B": 64, "lo": 1, "hi": 1, "ctx_lo": 1, "ctx_hi": 1500, "lens": 3,
         "Hk": 8, "D": 128, "dtype": "bf16", "cache": "e4m3", "page": 16},
        # whole prompts written into the 8-bit cache
        {"name": "write_prompts", "op": "write", "B": 8, "lo": 700, "hi": 8192, "ctx_lo": 0, "ctx_hi": 900, "lens": 4,
         "Hk": 8, "D": 128, "dtype": "bf16", "cache": "e4m3", "page": 64},
        # the keys and values of one stored vecset read back for the volume decoder
        {"name": "read_vecset", "op": "read", "B": 1, "lo": 4096, "hi": 4096, "ctx_lo": 0, "ctx_hi": 0, "lens": 1,
         "Hk": 8, "D": 64, "dtype": "bf16", "cache": "e4m3", "page": 64},
        # many long contexts read back (a batch that moves to another card)
        {"name": "read_contexts", "op": "read", "B": 8, "lo": 3000, "hi": 16384, "ctx_lo": 0, "ctx_hi": 0, "lens": 2,
         "Hk": 8, "D": 128, "dtype": "bf16", "cache": "e4m3", "page": 32},
        # one sequence, one new token, a short bf16 context: the latency of a single step
        {"name": "paged_one_token", "op": "paged", "B": 1, "lo": 1, "hi": 1, "ctx_lo": 700, "ctx_hi": 700, "lens": 1,
         "Hq": 8, "Hk": 8, "D": 64, "dtype": "bf16", "cache": "bf16", "page": 16, "causal": True},
        # a serving step: 48 sequences, one token each, long ragged contexts in the 8-bit cache
        {"name": "paged_step", "op": "paged", "B": 48, "lo": 1, "hi": 1, "ctx_lo": 300, "ctx_hi": 16000, "lens": 5,
         "Hq": 32, "Hk": 8, "D": 128, "dtype": "bf16", "cache": "e4m3", "page": 64, "causal": True},
        # chunked prefill: 512 new tokens behind a long bf16 context, next to a short chunk
        {"name": "paged_chunk", "op": "paged", "B": 2, "lo": 100, "hi": 512, "ctx_lo": 9000, "ctx_hi": 15000, "lens": 6,
         "Hq": 32, "Hk": 8, "D": 128, "dtype": "bf16", "cache": "bf16", "page": 32, "causal": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = ((8, 8), (4, 4), (32, 8), (16, 1), (12, 4), (6, 2), (15, 3), (7, 7), (24, 2))


def draw(rng):
    """A case of the same ranges; one that would cost more than the largest listed one is drawn again."""
    case = _draw(rng)
    w = work(case)
    if w["flops"] * (24 if case["dtype"] == "f32" else 1) > 3.8e11 or w["bytes"] > 7e8:
        return draw(rng)
    return case


def _draw(rng):
    op = rng.choice(["rope", "packed", "packed", "write", "read", "paged", "paged", "paged"])
    Hq, Hk = rng.choice(HEADS)
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    lens = rng.randrange(1 << 20)
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 16384), "Hq": Hq, "Hk": Hk, "D": D, "dtype": dtype,
                "rot": rng.choice([D, D, D // 2, D // 4 * 3, 22]), "interleaved": rng.random() < 0.5,
                "scaled": rng.random() < 0.4, "pos0": _log(rng, 1, 1 << 20) - 1}
    if op == "packed":
        most = 4096 if dtype == "bf16" else 1100
        hi = _log(rng, 1, most)
        # the padded scores of the plain form stay within those of the largest listed case
        B = min(_log(rng, 1, 24), max(1, (5 * 32 * 4096 * 4096) // (Hq * hi * hi)))
        return {"op": op, "B": B, "lo": rng.randint(0, hi), "hi": hi, "ctx_lo": 0, "ctx_hi": 0, "lens": lens, "Hq": Hq, "Hk": Hk,
                "D": D, "dtype": dtype, "causal": rng.random() < 0.6}
    cache = rng.choice([dtype, "e4m3", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        hi = _log(rng, 1, 8192)
        return {"op": op, "B": min(_log(rng, 1, 64), max(1, 65536 // hi)), "lo": rng.randint(0, hi), "hi": hi, "ctx_lo": 0,
                "ctx_hi": rng.randint(0, 900) if op == "write" else 0, "lens": lens, "Hk": Hk, "D": D, "dtype": dtype, "cache": cache,
                "page": page}
    single = rng.random() < 0.5
    hi = 1 if single else _log(rng, 2, 512)
    ctx = _log(rng, 1, 16000 if dtype == "bf16" else 4000)
    B = min(_log(rng, 1, 48), max(1, 48 * 16000 // (ctx + hi) // (1 if single else 8)))
    B = max(1, min(B, (5 * 32 * 4096 * 4096 // 8) // (Hq * hi * (ctx + hi))))
    return {"op": op, "B": B, "lo": 1 if single else rng.randint(1, hi), "hi": hi, "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx,
            "lens": lens, "Hq": Hq, "Hk": Hk, "D": D, "dtype": dtype, "cache": cache, "page": page,
            "causal": single or rng.random() < 0.8}


def _frequencies(case, device):
    """Angles per position of the rotary pairs; long contexts: slow pairs divided by 8, a ramp in between, fast pairs as they are."""
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device=device)
    f = 10000.0 ** (-i / half)
    if case["scaled"]:
        turns = 4096 * f / 6.283185307179586          # turns of a pair over the context it was made for
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / 8.0 * (1 - keep)
    return f


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(DT[case["dtype"]])

    def offsets(lens):
        return torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=dev)

    op, D = case["op"], case["D"]
    s = {"case": case}
    if op == "rope":
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        qkv = randn(T, Hq + 2 * Hk, D, scale=1.7)      # the fused projection's output: queries, keys, values
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["q_gain"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
        s["k_gain"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
        s["positions"] = torch.arange(case["pos0"], case["pos0"] + T, dtype=torch.int32, device=dev)
        s["inv_freq"] = _frequencies(case, dev)
        s["mscale"] = 1.2 if case["scaled"] else 1.0
        return s
    new, total = _lens(case)
    s["max_new"], s["max_total"], s["T"] = max(new), max(total), sum(new)
    s["cu"] = offsets(new)
    if op == "packed":
        qkv = randn(sum(new), case["Hq"] + 2 * case["Hk"], D, scale=1.2)
        s["q"], s["k"], s["v"] = qkv.split([case["Hq"], case["Hk"], case["Hk"]], 1)
        return s
    B, Hk, page = case["B"], case["Hk"], case["page"]
    width = max(1, -(-max(total) // page))
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + PAD
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(B)], device=dev)[:, None]
    j = torch.arange(width, device=dev)[None]
    s["table"] = torch.where(j < torch.tensor(need, device=dev)[:, None], order[(first + j).clamp(max=n_pages - 1)],
                             torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    shape = (n_pages, Hk, page, D)
    for n in ("k", "v"):
        if case["cache"] == "e4m3":
            s["cache_" + n] = (torch.randn(*shape, generator=g, device=dev) * 110.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["exp_" + n] = torch.randint(118, 122, shape[:3], generator=g, device=dev, dtype=torch.uint8)
        else:
            s["cache_" + n], s["exp_" + n] = torch.randn(*shape, generator=g, device=dev).to(DT[case["cache"]]), None
    if op == "write":
        s["k"], s["v"] = randn(sum(new), Hk, D, scale=1.5), randn(sum(new), Hk, D)
    if op == "read":
        s["out_k"], s["out_v"] = (torch.empty(sum(total), Hk, D, dtype=DT[case["dtype"]], device=dev) for _ in "kv")
    if op == "paged":
        s["q"] = randn(sum(new), case["Hq"], D, scale=1.2)
    return s


# ------------------------------------------------------------------ plain forms

def _rope_plain(s, x, gain):
    c, x = s["case"], x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["mscale"]).float()[:, None], (torch.sin(angle) * s["mscale"]).float()[:, None]
    y, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = y.chunk(2, -1)
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, rest), -1).to(DT[c["dtype"]])


def _gather_rows(x, cu, n):
    """[T, H, D] packed -> [B, n, H, D] float32, rows beyond a sequence zero."""
    i = torch.arange(n, device=x.device)
    at = cu[:-1, None] + i
    rows = x[at.clamp(max=x.shape[0] - 1)].float()
    return torch.where((i < (cu[1:] - cu[:-1])[:, None])[:, :, None, None], rows, torch.zeros((), device=x.device))


def _attend(q, k, v, q_len, k_len, causal):
    """q [B, n, Hk, G, D], k and v [B, m, Hk, D] in float32 -> [B, n, Hk, G, D], log of the sums [B, n, Hk, G]."""
    B, n, Hk, G, D = q.shape
    m = k.shape[1]
    sc = (q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, D) @ k.permute(0, 2, 3, 1)).view(B, Hk, G, n, m) * D ** -0.5
    j, i = torch.arange(m, device=q.device), torch.arange(n, device=q.device)
    seen = (j < k_len[:, None])[:, None, :]
    if causal:
        seen = seen & (j[None, None] <= (k_len - q_len)[:, None, None] + i[:, None])
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros((), device=q.device))
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, G * n, m) @ v.permute(0, 2, 1, 3)).view(B, Hk, G, n, D) / total
    o = torch.where(total > 0, o, torch.zeros((), device=q.device))
    return o.permute(0, 3, 1, 2, 4), (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)


def _pack(x, cu, T):
    """[B, n, ...] -> [T, ...]: the rows of every sequence behind one another."""
    t = torch.arange(T, device=x.device, dtype=cu.dtype)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return x[b, (t - cu[b]).long()]


def _attention_plain(s, k, v, k_len):
    c, cu = s["case"], s["cu"]
    q = _gather_rows(s["q"], cu, s["max_new"]).unflatten(2, (c["Hk"], c["Hq"] // c["Hk"]))
    o, lse = _attend(q, k, v, cu[1:] - cu[:-1], k_len, c["causal"])
    return _pack(o.flatten(2, 3), cu, s["T"]).to(DT[c["dtype"]]), _pack(lse.flatten(2, 3), cu, s["T"])


def _cache_rows(s, n, length):
    """The cache's first `length` tokens of every sequence as float32 [B, length, Hk, D], rows beyond its length zero."""
    page = s["case"]["page"]
    i = torch.arange(length, device="cuda")
    pages = s["table"][:, i // page].clamp(min=0).long()
    x = s["cache_" + n][pages, :, i % page]
    if s["exp_" + n] is not None:
        x = x.view(torch.float8_e4m3fn).float() * torch.exp2(s["exp_" + n][pages, :, i % page].float() - 127)[..., None]
    return torch.where((i < s["kv_len"][:, None])[:, :, None, None], x.float(), torch.zeros((), device="cuda"))


def _slots(s):
    """Page and row in it of every new token: the last ones of their sequences."""
    page, cu = s["case"]["page"], s["cu"]
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = s["kv_len"][b] - (cu[b + 1] - t)
    return s["table"][b, at // page].long(), (at % page).long()


def _write_plain(s, n):
    x, (pages, rows) = s[n], _slots(s)
    if s["exp_" + n] is None:
        s["cache_" + n][pages, :, rows] = x
        return s["cache_" + n]
    x = x.float()
    mantissa, e = torch.frexp(x.abs().amax(-1))                   # the row's largest value is mantissa 2^e, 448 = 0.875 2^9
    e = torch.where(mantissa > 0, torch.where(mantissa <= 0.875, e - 9, e - 8).clamp(-100, 119), torch.zeros((), dtype=e.dtype, device=e.device))
    codes = (x * torch.exp2(-e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["cache_" + n][pages, :, rows] = codes.view(torch.uint8)
    s["exp_" + n][pages, :, rows] = (e + 127).to(torch.uint8)
    return s["cache_" + n].view(torch.float8_e4m3fn), s["exp_" + n]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return _rope_plain(s, s["q"], s["q_gain"]), _rope_plain(s, s["k"], s["k_gain"])
    if c["op"] == "packed":
        cu, n = s["cu"], s["max_new"]
        return _attention_plain(s, _gather_rows(s["k"], cu, n), _gather_rows(s["v"], cu, n), cu[1:] - cu[:-1])
    if c["op"] == "write":
        return _write_plain(s, "k"), _write_plain(s, "v")
    if c["op"] == "read":
        return tuple(_pack(_cache_rows(s, n, s["max_total"]), s["cu"], s["T"]).to(DT[c["dtype"]]) for n in "kv")
    return _attention_plain(s, _cache_rows(s, "k", s["max_total"]), _cache_rows(s, "v", s["max_total"]), s["kv_len"])


def run(state):
    if not own:
        return _run_plain(state)
    import neural_sdf_volume_b200 as vdm
    s, c = state, state["case"]
    if c["op"] == "rope":
        rope = vdm.Rope(s["inv_freq"], c["interleaved"], s["mscale"])
        return vdm.vdm_qk_norm_rope(s["q"], s["k"], s["positions"], rope, q_gain=s["q_gain"], k_gain=s["k_gain"], eps=1e-6)
    if c["op"] == "packed":
        return vdm.vdm_attention_packed(s["q"], s["k"], s["v"], s["cu"], causal=c["causal"], want_lse=True)
    cache = vdm.KVCache(s["cache_k"], s["cache_v"], s["exp_k"], s["exp_v"])
    if c["op"] == "write":
        vdm.vdm_cache_write(cache, s["k"], s["v"], s["cu"], s["kv_len"], s["table"])
        if c["cache"] != "e4m3":
            return s["cache_k"], s["cache_v"]
        return tuple((s["cache_" + n].view(torch.float8_e4m3fn), s["exp_" + n]) for n in "kv")
    if c["op"] == "read":
        return vdm.vdm_cache_read(cache, s["kv_len"], s["table"], s["cu"], out=(s["out_k"], s["out_v"]))
    return vdm.vdm_attention_paged(s["q"], cache, s["cu"], s["kv_len"], s["table"], causal=c["causal"], want_lse=True)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, D, el = case["op"], case["D"], 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * D * el + 4 * case["T"] + 8 * D + 4 * case["rot"], "flops": n * D * 7}
    new, total = _lens(case)
    Hk = case["Hk"]
    row = D + 1 if case.get("cache") == "e4m3" else D * (2 if case.get("cache") == "bf16" else 4)   # a cached row
    if op == "write":
        return {"bytes": 2 * sum(new) * Hk * (D * el + row) + 4 * (sum(new) // case["page"] + 2 * case["B"]), "flops": 2 * sum(new) * Hk * D * 3}
    if op == "read":
        return {"bytes": 2 * sum(total) * Hk * (D * el + row) + 4 * (sum(total) // case["page"] + 2 * case["B"]), "flops": 2 * sum(total) * Hk * D}
    Hq = case["Hq"]
    pairs = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in zip(new, total))
    keys = sum(total) * Hk * 2 * (D * el if op == "packed" else row)
    return {"bytes": keys + sum(new) * Hq * (2 * D * el + 4), "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        z = torch.exp(1j * s["positions"].double()[:, None, None] * s["inv_freq"][None, None]) * s["mscale"]
        out = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            x = x.double()
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["D"] + 1e-6) * gain.double()
            r, h = case["rot"], case["rot"] // 2
            first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, h), slice(h, r))
            w = torch.complex(x[..., first], x[..., second]) * z
            y = x.clone()
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y)
        return tuple(out)
    new, total = _lens(case)

    def cached(n, b):
        """Sequence b's cached rows in order, [tokens, Hk, D]."""
        pages = s["table"][b, :-(-total[b] // case["page"])].long()
        x = s["cache_" + n][pages]
        x = x.view(torch.float8_e4m3fn).double() * 2.0 ** (s["exp_" + n][pages].double()[..., None] - 127) if case["cache"] == "e4m3" else x.double()
        return x.transpose(1, 2).flatten(0, 1)[:total[b]]

    if case["op"] == "read":
        return tuple(torch.cat([cached(n, b) for b in range(case["B"])]) for n in "kv")
    if case["op"] == "write":
        return None          # codes are the definition's own rounding: compared with the plain form's
    outs, sums, G = [], [], case["Hq"] // case["Hk"]
    at = 0
    for b in range(case["B"]):
        n, m = new[b], total[b]
        q = s["q"][at:at + n].double()
        k, v = (s["k"][at:at + n].double(), s["v"][at:at + n].double()) if case["op"] == "packed" else (cached("k", b), cached("v", b))
        at += n
        allowed = torch.ones(n, m, dtype=torch.bool, device="cuda")
        if case["causal"]:
            allowed = allowed.tril(m - n)
        o, l = torch.zeros(n, case["Hq"], case["D"], dtype=torch.float64, device="cuda"), torch.empty(n, case["Hq"], dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            sc = (q[:, h] @ k[:, h // G].T / case["D"] ** 0.5).masked_fill(~allowed, float("-inf"))
            l[:, h] = torch.logsumexp(sc, -1)
            o[:, h] = torch.where(allowed.any(-1, keepdim=True), torch.softmax(sc, -1), torch.zeros((), dtype=torch.float64, device="cuda")) @ v[:, h // G]
        outs.append(o)
        sums.append(l)
    return torch.cat(outs), torch.cat(sums)
