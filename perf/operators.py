"""The operators of decoding on a bounded key/value cache, as a user's program calls them.

Four operators that follow one another in a serving step:

* ``rope``     rotary positions of packed queries and keys, with one position axis (text) or
               several (time, height, width), and the same rotation backwards for gradients;
* ``prefix``   attention of a batch whose sequences all start with the same keys and values;
* ``weights``  the attention weight that each cached key has received, summed over the queries;
* ``evict``    the cache cut down to a budget by that weight.

``own`` False computes them in elementary torch operations (32-bit arithmetic, angles in 64 bits);
``own`` True calls the library.  ``prepare`` makes what the program has in hand before the call.
Lengths follow from the case alone, values from the seed.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of 64 requests: q and k are slices of the fused projection's output,
        # contexts of up to a million tokens.  Latency.
        dict(name="rope_decode", op="rope", tokens=64, h_q=32, h_kv=8, d=128, rot=128, dtype="bf16",
             axes=1, interleaved=False, inverse=False, packed=True, far=1000000),
        # Prompts of images and video: positions in time, height and width, a ragged token count.
        dict(name="rope_video", op="rope", tokens=20011, h_q=32, h_kv=8, d=128, rot=128, dtype="bf16",
             axes=3, interleaved=False, inverse=False, packed=True, far=32768),
        # The gradients of a training step, where only 64 of 96 columns turn, in pairs of neighbours.
        dict(name="rope_backward", op="rope", tokens=16384, h_q=16, h_kv=16, d=96, rot=64, dtype="fp16",
             axes=1, interleaved=True, inverse=True, packed=False, far=8192),
        # A few requests behind a short system prompt.  Latency.
        dict(name="prefix_decode_small", op="prefix", seqs=3, q_lo=1, q_hi=1, prefix=1000, kv_lo=17, kv_hi=255,
             h_q=8, h_kv=8, d=64, dtype="fp16", causal=True, window=0),
        # A decode step of many requests behind one long prompt, each with its own answer so far.
        dict(name="prefix_decode", op="prefix", seqs=64, q_lo=1, q_hi=1, prefix=16384, kv_lo=100, kv_hi=1024,
             h_q=32, h_kv=8, d=128, dtype="bf16", causal=True, window=0),
        # New user turns of ragged length appended to chats that share a prompt.
        dict(name="prefix_extend", op="prefix", seqs=16, q_lo=64, q_hi=436, prefix=8192, kv_lo=436, kv_hi=2048,
             h_q=32, h_kv=8, d=128, dtype="bf16", causal=True, window=0),
        # The running weights of a decode step over ragged caches.
        dict(name="weights_decode", op="weights", seqs=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=8192,
             h_q=32, h_kv=8, d=128, dtype="bf16", causal=True, window=0, prev=True),
        # The weights that the last rows of each long prompt give to all of its keys.
        dict(name="weights_window", op="weights", seqs=4, q_lo=32, q_hi=32, kv_lo=12288, kv_hi=32768,
             h_q=32, h_kv=8, d=128, dtype="fp16", causal=True, window=0, prev=False),
        # Every row of whole prompts.
        dict(name="weights_prompt", op="weights", seqs=4, q_lo=4096, q_hi=4096, kv_lo=4096, kv_hi=4096,
             h_q=32, h_kv=32, d=128, dtype="bf16", causal=True, window=0, prev=False),
        # A few short caches.  Latency.
        dict(name="evict_small", op="evict", seqs=8, kv_lo=100, kv_hi=436, budget=128, sink=4, recent=32,
             h_kv=4, d=64, dtype="fp16"),
        # A batch of decoding requests, each cut to a quarter.
        dict(name="evict_batch", op="evict", seqs=64, kv_lo=4096, kv_hi=8192, budget=2048, sink=4, recent=256,
             h_kv=8, d=128, dtype="bf16"),
        # One very long prompt.
        dict(name="evict_long", op="evict", seqs=1, kv_lo=131071, kv_hi=131071, budget=16384, sink=16, recent=1024,
             h_kv=8, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefix", "weights", "evict"])
    h_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 8) if g * h_kv <= 32])
    d = rng.choice([64, 96, 128])
    if op == "rope":
        axes = rng.choice([1, 2, 3])
        rot = rng.choice([r for r in (32, 64, 96, 128) if r <= d])
        return dict(op=op, tokens=_log(rng, 1, 20011), h_q=h_kv * group, h_kv=h_kv, d=d, rot=rot,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), axes=axes, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, packed=rng.random() < 0.5, far=_log(rng, 1000, 1000000))
    if op == "prefix":
        if rng.random() < 0.5:
            seqs, q_hi, prefix = _log(rng, 1, 64), 1, _log(rng, 128, 16384)
        else:
            seqs, q_hi, prefix = _log(rng, 1, 16), _log(rng, 2, 400), _log(rng, 128, 8192)
        kv_hi = _log(rng, q_hi + 16, 1024)
        return dict(op=op, seqs=seqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, prefix=prefix, kv_lo=max(q_hi, kv_hi // 5),
                    kv_hi=kv_hi, h_q=h_kv * group, h_kv=h_kv, d=d, dtype=rng.choice(["bf16", "fp16"]), causal=True,
                    window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]))
    if op == "weights":
        kind = rng.choice(["decode", "window", "prompt"])
        if kind == "decode":
            seqs, q_hi, kv_hi = _log(rng, 1, 64), 1, _log(rng, 32, 8192)
        elif kind == "window":
            seqs, q_hi = _log(rng, 1, 4), _log(rng, 8, 128)
            kv_hi = _log(rng, 200, 32768)
        else:
            seqs, q_hi = _log(rng, 1, 4), _log(rng, 128, 4096)
            kv_hi = q_hi
        return dict(op=op, seqs=seqs, q_lo=q_hi if kind == "prompt" else max(1, q_hi // 2), q_hi=q_hi,
                    kv_lo=kv_hi if kind == "prompt" else max(q_hi, kv_hi // 4), kv_hi=kv_hi, h_q=h_kv * group,
                    h_kv=h_kv, d=d, dtype=rng.choice(["bf16", "fp16"]), causal=True,
                    window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]), prev=rng.random() < 0.5)
    seqs = _log(rng, 1, 64)
    kv_hi = _log(rng, 64, min(131071, 64 * 8192 // seqs))
    budget = max(8, int(kv_hi * rng.uniform(0.05, 0.6)))
    return dict(op=op, seqs=seqs, kv_lo=max(1, kv_hi // 3), kv_hi=kv_hi, budget=budget, sink=min(4, budget // 4),
                recent=budget // 8, h_kv=h_kv, d=d, dtype=rng.choice(["bf16", "fp16", "fp32"]))


def _lens(n, lo, hi):
    """n ragged lengths from lo to hi, both among them where there are two or more."""
    if n == 1:
        return [hi]
    mix = [(i * 7919) % n if math.gcd(7919, n) == 1 else i for i in range(n)]
    return [lo + (hi - lo) * m // (n - 1) for m in mix]


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _pairs(q_lens, kv_lens, prefix, causal, window):
    """Visible (row, key) pairs of one head."""
    n = 0
    for ql, kl in zip(q_lens, kv_lens):
        for i in range(ql):
            diag = i + prefix + kl - ql
            hi = min(prefix + kl, diag + 1) if causal else prefix + kl
            lo = max(0, diag - window + 1) if window > 0 else 0
            n += max(0, hi - lo)
    return n


def _sections(axes, rot):
    half = rot // 2
    if axes == 1:
        return (half,)
    if axes == 2:
        return (half // 2, half - half // 2)
    first = half // 4
    second = (half - first) // 2
    return (first, second, half - first - second)


def work(case):
    c = case
    op, es = c["op"], SIZE[c["dtype"]]
    if op == "rope":
        n = c["tokens"] * (c["h_q"] + c["h_kv"])
        return {"bytes": 2 * n * c["d"] * es + 4 * c["tokens"] * c["axes"], "flops": 3 * n * c["rot"]}
    kv = _lens(c["seqs"], c["kv_lo"], c["kv_hi"])
    if op == "evict":
        kept = sum(min(c["budget"], x) for x in kv)
        h = c["h_kv"]
        return {"bytes": 4 * h * sum(kv) + kept * h * (4 * c["d"] * es + 8), "flops": 4 * h * sum(kv)}
    q = _lens(c["seqs"], c["q_lo"], c["q_hi"])
    rows = sum(q) * c["h_q"]
    if op == "prefix":
        pairs = _pairs(q, kv, c["prefix"], c["causal"], c["window"])
        keys = (c["prefix"] + sum(kv)) * c["h_kv"]
        return {"bytes": 2 * keys * c["d"] * es + rows * (2 * c["d"] * es + 4), "flops": 4 * c["d"] * pairs * c["h_q"]}
    pairs = _pairs(q, kv, 0, c["causal"], c["window"])
    keys = sum(kv) * c["h_kv"]
    return {"bytes": keys * (c["d"] * es + (8 if c["prev"] else 4)) + rows * (c["d"] * es + 4),
            "flops": 2 * c["d"] * pairs * c["h_q"]}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    s = dict(case=c)
    if c["op"] == "rope":
        t, hq, hk, d = c["tokens"], c["h_q"], c["h_kv"], c["d"]
        if c["packed"]:
            qkv = normal(t, hq + 2 * hk, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(t, hq, d), normal(t, hk, d)
        at = torch.arange(t, device=DEV)
        start = torch.randint(0, c["far"], (c["axes"], 1), generator=g, device=DEV)
        if c["axes"] == 1:  # sequences of 512 tokens, each with a start of its own
            start = torch.randint(0, c["far"], (t // 512 + 1,), generator=g, device=DEV)
            pos = (start[at // 512] + at % 512).view(1, t)
        else:  # frames of 24 x 32 patches (the last axes are height and width)
            grid = torch.stack([at // 768, at // 32 % 24, at % 32])[3 - c["axes"]:]
            pos = grid + start
        s["positions"] = pos.to(torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        s["sections"] = _sections(c["axes"], c["rot"])
        ax = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        s["axis_of"] = torch.tensor(ax, device=DEV)
        return s
    kv = _lens(c["seqs"], c["kv_lo"], c["kv_hi"])
    total_kv = sum(kv)
    s["cu_kv"], s["max_kv"] = ints(_cu(kv)), max(kv)
    if c["op"] == "evict":
        h, d = c["h_kv"], c["d"]
        s["k"], s["v"] = normal(total_kv, h, d), normal(total_kv, h, d)
        # weights as attention leaves them: heavy-tailed, many of them nothing at all
        u = torch.rand(h, total_kv, generator=g, device=DEV)
        w = torch.exp(4.0 * torch.randn(h, total_kv, generator=g, device=DEV)) * 1e-3
        s["weights"] = torch.where(u < 0.2, torch.zeros_like(w), w)
        s["total_out"] = sum(min(c["budget"], x) for x in kv)
        return s
    q = _lens(c["seqs"], c["q_lo"], c["q_hi"])
    total_q, hq, hk, d = sum(q), c["h_q"], c["h_kv"], c["d"]
    s["cu_q"], s["max_q"] = ints(_cu(q)), max(q)
    s["scale"] = d ** -0.5
    s["q"], s["k"] = normal(total_q, hq, d), normal(total_kv, hk, d)
    if c["op"] == "prefix":
        s["v"] = normal(total_kv, hk, d)
        s["kp"], s["vp"] = normal(c["prefix"], hk, d), normal(c["prefix"], hk, d)
    else:
        logit, _, rows = _own_logits(s)
        lse = torch.logsumexp(logit, dim=-1)  # [seqs, h_kv, max_q, group]
        s["lse"] = lse.permute(1, 3, 0, 2).reshape(hq, -1)[:, rows].contiguous()
        del logit, lse
        s["prev"] = torch.rand(hk, total_kv, generator=g, device=DEV) if c["prev"] else None
    return s


# ------------------------------------------------------------------------------ plain forms
def _padded(x, cu, most):
    """[total, ...] packed rows as [seqs, most, ...], zero behind each sequence, and which rows are real."""
    at = cu[:-1, None].long() + torch.arange(most, device=x.device)
    real = at < cu[1:, None]
    y = x[at.clamp(max=max(0, x.shape[0] - 1))].float()
    return y * real.view(*real.shape, *([1] * (x.dim() - 1))), real


def _visible(s, first, n, shift):
    """[seqs, max_q, n]: whether a row sees key first + j, counted from the sequence's first key; shift keys come before its own."""
    c = s["case"]
    cu_q, cu_kv = s["cu_q"].long(), s["cu_kv"].long()
    q_len, kv_len = (cu_q[1:] - cu_q[:-1]).view(-1, 1, 1), (cu_kv[1:] - cu_kv[:-1]).view(-1, 1, 1)
    i = torch.arange(s["max_q"], device=DEV).view(1, -1, 1)
    j = first + torch.arange(n, device=DEV).view(1, 1, -1)
    diag = i + shift + kv_len - q_len
    ok = (i < q_len) & (j < shift + kv_len)
    if c["causal"]:
        ok = ok & (j <= diag)
    if c["window"] > 0:
        ok = ok & (j > diag - c["window"])
    return ok


def _rows(q, s):
    """q as [seqs, h_kv, max_q * group, d], and the padded row of every real one."""
    c = s["case"]
    hk, group, d = c["h_kv"], c["h_q"] // c["h_kv"], c["d"]
    y, real = _padded(q, s["cu_q"], s["max_q"])
    n, m = real.shape
    y = y.view(n, m, hk, group, d).permute(0, 2, 1, 3, 4).reshape(n, hk, m * group, d)
    return y, real.reshape(-1).nonzero().view(-1)


def _own_logits(s, shift=0):
    """Logits of each sequence's own keys [seqs, h_kv, max_q, group, max_kv], -inf where masked; its mask and the real rows."""
    c = s["case"]
    group = c["h_q"] // c["h_kv"]
    q, rows = _rows(s["q"], s)
    k, _ = _padded(s["k"], s["cu_kv"], s["max_kv"])
    n, m = k.shape[0], s["max_q"]
    x = (q @ k.permute(0, 2, 3, 1)).view(n, c["h_kv"], m, group, -1) * s["scale"]
    ok = _visible(s, shift, s["max_kv"], shift).view(n, 1, m, 1, -1)
    return x.masked_fill(~ok, -math.inf), ok, rows


def _plain_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    angle = s["positions"].double()[s["axis_of"]].t() * s["inv_freq"].double()  # [tokens, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float()
        r = y[..., :c["rot"]]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, y[..., c["rot"]:]], dim=-1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_prefix(s):
    c = s["case"]
    hk, group, d, n, m, p = c["h_kv"], c["h_q"] // c["h_kv"], c["d"], c["seqs"], s["max_q"], c["prefix"]
    x, _, rows = _own_logits(s, p)
    q, _ = _rows(s["q"], s)
    flat = q.permute(1, 0, 2, 3).reshape(hk, n * m * group, d)
    y = (flat @ s["kp"].float().permute(1, 2, 0)).view(hk, n, m, group, p).transpose(0, 1) * s["scale"]
    y = y.masked_fill(~_visible(s, 0, p, p).view(n, 1, m, 1, p), -math.inf)
    top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x, y = (x - top).exp(), (y - top).exp()
    total = x.sum(-1) + y.sum(-1)
    v, _ = _padded(s["v"], s["cu_kv"], s["max_kv"])
    o = x.view(n, hk, m * group, -1) @ v.transpose(1, 2)
    o = o + (y.transpose(0, 1).reshape(hk, n * m * group, p) @ s["vp"].float().transpose(0, 1)).view(hk, n, m * group, d).transpose(0, 1)
    o = o.view(n, hk, m, group, d) / total.clamp(min=1e-30)[..., None]
    out = o.permute(0, 2, 1, 3, 4).reshape(n * m, hk * group, d)[rows].to(s["q"].dtype)
    lse = (top[..., 0] + total.log()).permute(1, 3, 0, 2).reshape(hk * group, -1)[:, rows]
    return {"out": out, "lse": lse.contiguous()}


def _plain_weights(s):
    c = s["case"]
    x, ok, rows = _own_logits(s)
    n, m, group = c["seqs"], s["max_q"], c["h_q"] // c["h_kv"]
    lse = torch.zeros(c["h_q"], n * m, device=DEV)
    lse[:, rows] = s["lse"]
    lse = lse.view(c["h_kv"], group, n, m).permute(2, 0, 3, 1)[..., None]
    w = (x - lse).exp().sum((2, 3))  # [seqs, h_kv, max_kv]
    at = torch.arange(s["max_kv"], device=DEV) < (s["cu_kv"][1:] - s["cu_kv"][:-1])[:, None]
    w = w.transpose(0, 1).reshape(c["h_kv"], -1)[:, at.reshape(-1)]
    return {"weights": w if s["prev"] is None else s["prev"] + w}


def _plain_evict(s):
    c = s["case"]
    h, n, most = c["h_kv"], c["seqs"], s["max_kv"]
    cu = s["cu_kv"].long()
    size = (cu[1:] - cu[:-1])[:, None]
    keep = size.clamp(max=c["budget"])
    j = torch.arange(most, device=DEV)
    w, _ = _padded(s["weights"].t(), s["cu_kv"], most)  # [seqs, most, h]
    w = w.permute(2, 0, 1)
    # the first `sink` and the last `recent` keys stay; what is behind the end never does
    safe = (j < c["sink"]) | (j >= size - c["recent"])
    w = torch.where(safe, torch.full_like(w, math.inf), w)
    w = torch.where(j < size, w, torch.full_like(w, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, (j < keep).expand(h, n, most))
    index = kept.nonzero()[:, 2].view(h, -1)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), keep[:, 0])
    at = cu[seq] + index  # [h, total_out]: packed key
    heads = torch.arange(h, device=DEV)[:, None]
    cu_out = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), keep[:, 0].cumsum(0)])
    return {"k": s["k"][at, heads].transpose(0, 1).contiguous(), "v": s["v"][at, heads].transpose(0, 1).contiguous(),
            "weights": s["weights"][heads, at], "index": index.int(), "cu": cu_out.int()}


# ------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rope": _plain_rope, "prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict}[op](s)
    import variable_length_flash_gb300 as vlf
    if op == "rope":
        q, k = vlf.vlf_rope(s["q"], s["k"], s["positions"], s["inv_freq"], sections=s["sections"],
                            interleaved=c["interleaved"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if op == "prefix":
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["cu_q"], s["cu_kv"],
                                                  s["max_q"], s["max_kv"], scale=s["scale"], causal=c["causal"],
                                                  window=c["window"])
        return {"out": out, "lse": lse}
    if op == "weights":
        return {"weights": vlf.vlf_attn_key_weights(s["q"], s["k"], s["lse"], s["cu_q"], s["cu_kv"], s["max_q"],
                                                    s["max_kv"], scale=s["scale"], causal=c["causal"],
                                                    window=c["window"], prev=s["prev"])}
    k, v, w, index, cu = vlf.vlf_cache_evict(s["k"], s["v"], s["weights"], s["cu_kv"], c["budget"], sink=c["sink"],
                                             recent=c["recent"], max_seqlen_kv=s["max_kv"], total_out=s["total_out"])
    return {"k": k, "v": v, "weights": w, "index": index, "cu": cu}


# ------------------------------------------------------------------------------ in 64 bits
def _mask64(ql, keys, own_keys, causal, window):
    """[ql, keys] for a sequence whose last own_keys keys are its own: row i stands at key i + keys - ql."""
    at = torch.arange(ql, device=DEV)[:, None] + (keys - ql)
    j = torch.arange(keys, device=DEV)[None]
    ok = torch.ones(ql, keys, dtype=torch.bool, device=DEV)
    if causal:
        ok &= j <= at
    if window > 0:
        ok &= j > at - window
    return ok


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        half, sign = c["rot"] // 2, -1.0 if c["inverse"] else 1.0
        turns = torch.empty(c["tokens"], half, dtype=torch.float64, device=DEV)
        first = 0
        for a, n in enumerate(s["sections"]):
            turns[:, first:first + n] = torch.outer(s["positions"][a].double(), s["inv_freq"][first:first + n].double())
            first += n
        z = torch.polar(torch.ones_like(turns), sign * turns)[:, None]
        got = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            if c["interleaved"]:
                lo, hi = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
            else:
                lo, hi = x[..., :half], x[..., half:c["rot"]]
            y = torch.complex(lo.contiguous(), hi.contiguous()) * z
            lo.copy_(y.real), hi.copy_(y.imag)
            got[name] = x
        return got
    cu_kv = s["cu_kv"].tolist()
    if c["op"] == "evict":
        ks, vs, ws, ix = [], [], [], []
        for a, b in zip(cu_kv[:-1], cu_kv[1:]):
            n = min(c["budget"], b - a)
            w = s["weights"][:, a:b].double().clone()
            w[:, :c["sink"]] = math.inf
            w[:, max(0, b - a - c["recent"]):] = math.inf
            at = torch.argsort(-w, dim=1, stable=True)[:, :n].sort(dim=1).values  # [h, n]
            ix.append(at)
            ws.append(torch.gather(s["weights"][:, a:b].double(), 1, at))
            for got, x in ((ks, s["k"]), (vs, s["v"])):
                rows = at.t()[..., None].expand(-1, -1, c["d"])
                got.append(torch.gather(x[a:b].double(), 0, rows))
        cu = torch.tensor(_cu([x.shape[1] for x in ix]), dtype=torch.int32, device=DEV)
        return {"k": torch.cat(ks), "v": torch.cat(vs), "weights": torch.cat(ws, 1), "index": torch.cat(ix, 1).int(), "cu": cu}
    cu_q = s["cu_q"].tolist()
    group = c["h_q"] // c["h_kv"]
    if c["op"] == "prefix":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[1], s["q"].shape[0], dtype=torch.float64, device=DEV)
        kp, vp = s["kp"].double(), s["vp"].double()
        for n in range(c["seqs"]):
            a, b = cu_q[n], cu_q[n + 1]
            k = torch.cat([kp, s["k"][cu_kv[n]:cu_kv[n + 1]].double()])
            v = torch.cat([vp, s["v"][cu_kv[n]:cu_kv[n + 1]].double()])
            ok = _mask64(b - a, k.shape[0], cu_kv[n + 1] - cu_kv[n], c["causal"], c["window"])
            for g in range(c["h_kv"]):
                hs = slice(g * group, (g + 1) * group)
                x = torch.einsum("ihd,jd->hij", s["q"][a:b, hs].double(), k[:, g]) * s["scale"]
                x = x.masked_fill(~ok, -math.inf)
                top = torch.logsumexp(x, -1)
                lse[hs, a:b] = top
                # (a row that sees no key: no weights, no output)
                p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top))[..., None])
                out[a:b, hs] = torch.einsum("hij,jd->ihd", p, v[:, g])
        return {"out": out, "lse": lse}
    got = torch.zeros(c["h_kv"], cu_kv[-1], dtype=torch.float64, device=DEV)
    for n in range(c["seqs"]):
        a, b = cu_q[n], cu_q[n + 1]
        ok = _mask64(b - a, cu_kv[n + 1] - cu_kv[n], 0, c["causal"], c["window"])
        for h in range(c["h_q"]):
            x = s["q"][a:b, h].double() @ s["k"][cu_kv[n]:cu_kv[n + 1], h // group].double().t()
            p = torch.exp(x * s["scale"] - s["lse"][h, a:b].double()[:, None])
            got[h // group, cu_kv[n]:cu_kv[n + 1]] += torch.where(ok, p, torch.zeros_like(p)).sum(0)
    return {"weights": got if s["prev"] is None else s["prev"].double() + got}
