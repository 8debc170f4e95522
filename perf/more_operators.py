"""The operators of serving from a cache of pages held in 8 bits, as a user's program calls them.

A serving step runs them one after another:

* ``norm``     root-mean-square norm of each head of the queries and keys with the rotary positions
               in the same pass, and its gradients for training;
* ``fork``     the page tables of the next step: sequences that go on, fork, end or begin, the pages
               that they need, and the copies of the pages that they no longer share;
* ``write``    new keys and values rounded into their pages: e4m3 with one scale for each page and head;
* ``attend``   attention of new queries over those pages;
* ``compact``  the pages in use moved to the front of the pool.

``own`` False computes them in elementary torch operations (32-bit arithmetic, angles in 64 bits);
``own`` True calls the library.  ``prepare`` makes what the program has in hand before the call.
Lengths follow from the case alone, values and the pages' order from the seed.  The cache of one layer
is ``[pages, heads, page size, head_dim]`` for keys and for values, scales fp32 ``[pages, heads]``; it
is returned as it is held (an e4m3 tensor and its scales).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of 64 requests: q and k are slices of the fused projection's output.  Latency.
        dict(name="norm_decode", op="norm", tokens=64, h_q=32, h_kv=8, d=128, rot=128, dtype="bf16", axes=1,
             interleaved=False, backward=False, packed=True, far=1000000),
        # Prompts of images and video: positions in time, height and width, a ragged token count.
        dict(name="norm_video", op="norm", tokens=20011, h_q=32, h_kv=8, d=128, rot=128, dtype="bf16", axes=3,
             interleaved=False, backward=False, packed=True, far=32768),
        # The gradients of a training step, where only 64 of 96 columns turn, in pairs of neighbours.
        dict(name="norm_backward", op="norm", tokens=16384, h_q=16, h_kv=16, d=96, rot=64, dtype="fp16", axes=1,
             interleaved=True, backward=True, packed=False, far=8192),
        # One token of each of 64 requests goes into the last page of its cache.  Latency.
        dict(name="write_decode", op="write", seqs=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=8192, page=64, h_kv=8,
             d=128, dtype="bf16"),
        # Whole prompts of ragged length.
        dict(name="write_prompt", op="write", seqs=16, q_lo=128, q_hi=8192, kv_lo=128, kv_hi=8192, page=64, h_kv=8,
             d=128, dtype="bf16"),
        # A few requests with short contexts, small pages.  Latency.
        dict(name="attend_decode_small", op="attend", seqs=3, q_lo=1, q_hi=1, kv_lo=17, kv_hi=1000, page=16, h_q=8,
             h_kv=8, d=64, dtype="fp16", causal=True, window=0),
        # A decode step of many requests with ragged contexts.
        dict(name="attend_decode", op="attend", seqs=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=16384, page=64, h_q=32,
             h_kv=8, d=128, dtype="bf16", causal=True, window=0),
        # New user turns of ragged length appended to chats.
        dict(name="attend_extend", op="attend", seqs=16, q_lo=64, q_hi=436, kv_lo=436, kv_hi=8192, page=128, h_q=32,
             h_kv=8, d=128, dtype="bf16", causal=True, window=0),
        # Beam search: 8 requests with 4 beams each, half of which are dropped for copies of the others.  Latency.
        dict(name="fork_beams", op="fork", groups=8, width=4, kv_lo=100, kv_hi=1024, page=64, spare=64, grow=1, h_kv=8,
             d=128),
        # Sampled answers of many requests in small pages: some end, the best go on more than once.
        dict(name="fork_batch", op="fork", groups=64, width=4, kv_lo=1000, kv_hi=16384, page=16, spare=8192, grow=16,
             h_kv=8, d=128),
        # A small pool after a few requests have ended.  Latency.
        dict(name="compact_small", op="compact", seqs=8, kv_lo=100, kv_hi=1024, page=64, used=0.6, h_kv=8, d=128),
        # A pool half of whose pages are free, cut down so that its memory can be given back.
        dict(name="compact_pool", op="compact", seqs=64, kv_lo=1000, kv_hi=16384, page=64, used=0.5, h_kv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "attend", "fork", "compact"])
    h_kv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 96, 128])
    if op == "norm":
        group = rng.choice([g for g in (1, 2, 3, 4, 8) if g * h_kv <= 32])
        backward = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 16384 if backward else 20011), h_q=h_kv * group, h_kv=h_kv, d=d,
                    rot=rng.choice([r for r in (32, 64, 96, 128) if r <= d]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, backward=backward,
                    packed=rng.random() < 0.5, far=_log(rng, 1000, 1000000))
    page = rng.choice([16, 32, 64, 128])
    if op == "write":
        seqs = _log(rng, 1, 64)
        q_hi = 1 if rng.random() < 0.4 else _log(rng, 2, min(8192, 16 * 4096 // seqs))
        return dict(op=op, seqs=seqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=q_hi, kv_hi=max(q_hi, _log(rng, 32, 8192)),
                    page=page, h_kv=h_kv, d=d, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "attend":
        d = rng.choice([64, 128])
        group = rng.choice([g for g in (1, 2, 3, 4, 8) if g * h_kv <= 32])
        if rng.random() < 0.6:  # decode, one token or a few drafted ones
            seqs, q_hi, kv_hi = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4]), _log(rng, 32, 16384)
        else:
            seqs, q_hi, kv_hi = _log(rng, 1, 16), _log(rng, 5, 400), _log(rng, 400, 8192)
        return dict(op=op, seqs=seqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=max(q_hi, kv_hi // 8), kv_hi=kv_hi,
                    page=page, h_q=h_kv * group, h_kv=h_kv, d=d, dtype=rng.choice(["bf16", "fp16"]), causal=True,
                    window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]))
    if op == "fork":
        groups = _log(rng, 1, 64)
        kv_hi = _log(rng, 17, 8192)
        return dict(op=op, groups=groups, width=rng.choice([1, 2, 3, 4]), kv_lo=max(1, kv_hi // 8), kv_hi=kv_hi,
                    page=page, spare=64 + groups * 4 * 8, grow=_log(rng, 1, 64), h_kv=h_kv, d=d)
    seqs = _log(rng, 1, 64)
    kv_hi = _log(rng, 64, 8192)
    return dict(op=op, seqs=seqs, kv_lo=max(1, kv_hi // 8), kv_hi=kv_hi, page=page,
                used=round(rng.uniform(0.2, 0.95), 3), h_kv=h_kv, d=d)


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


def _two_to(e):
    """2^e of whole numbers, to the bit (a power function need not be)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _held(lens, page):
    """Pages that sequences of these lengths hold."""
    return sum(-(-x // page) for x in lens)


def _sections(axes, rot):
    half = rot // 2
    if axes == 1:
        return (half,)
    if axes == 2:
        return (half // 2, half - half // 2)
    first = half // 4
    second = (half - first) // 2
    return (first, second, half - first - second)


def _qkv_lens(c):
    kv = _lens(c["seqs"], c["kv_lo"], c["kv_hi"])
    return [min(a, b) for a, b in zip(_lens(c["seqs"], c["q_lo"], c["q_hi"]), kv)], kv


def _fork_lens(c):
    """The beams' lengths, the lengths that they share from the start, and which beam each of the next ones follows."""
    n, w = c["groups"], c["width"]
    first = _lens(n, c["kv_lo"], c["kv_hi"])
    lens = [x for x in first for _ in range(w)]
    shared = [x // 2 // c["page"] for x in first for _ in range(w)]  # whole pages of the prompt
    parents = []
    for g in range(n):
        for b in range(w):  # the lower half of the beams goes on, twice each; each eighth request has ended
            parents.append(-1 if g % 8 == 7 else g * w + b // 2)
    return lens, shared, parents


def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        es = SIZE[c["dtype"]]
        n = c["tokens"] * (c["h_q"] + c["h_kv"]) * c["d"]
        few = 4 * c["tokens"] * c["axes"] + 2 * c["d"] * es
        if c["backward"]:
            return {"bytes": 3 * n * es + few, "flops": 12 * n}
        return {"bytes": 2 * n * es + few, "flops": 6 * n}
    if op in ("write", "attend"):
        es = SIZE[c["dtype"]]
        q, kv = _qkv_lens(c)
        if op == "write":
            n = sum(q) * c["h_kv"] * c["d"]
            pages = sum((b - 1) // c["page"] - (b - a) // c["page"] + 1 for a, b in zip(q, kv))
            return {"bytes": 2 * n * (es + 1) + pages * (4 + 16 * c["h_kv"]), "flops": 6 * n}
        pairs = keys = 0
        for ql, kl in zip(q, kv):
            lo = kl
            for i in range(ql):
                diag = i + kl - ql
                first = max(0, diag - c["window"] + 1) if c["window"] > 0 else 0
                lo = min(lo, first)
                pairs += diag + 1 - first
            keys += kl - lo
        rows = sum(q) * c["h_q"]
        return {"bytes": 2 * keys * c["h_kv"] * c["d"] + 4 * (2 * c["h_kv"] + 1) * (keys // c["page"]) +
                rows * (2 * c["d"] * es + 4), "flops": 4 * c["d"] * pairs * c["h_q"]}
    page_bytes = 2 * c["h_kv"] * (c["page"] * c["d"] + 4)
    if op == "fork":
        lens, shared, parents = _fork_lens(c)
        kept = [lens[p] for p in parents if p >= 0]
        copies = sum(1 for i, p in enumerate(parents) if p >= 0 and lens[p] % c["page"] and p in parents[:i])
        pool = _fork_pages(c)
        return {"bytes": 4 * (_held(lens, c["page"]) + _held([x + c["grow"] for x in kept], c["page"]) + 2 * pool) +
                copies * 2 * page_bytes, "flops": pool}
    pool, used, moves = _compact_pages(c)
    return {"bytes": 4 * (2 * used + 2 * pool) + moves * 2 * page_bytes, "flops": pool}


def _fork_pages(c):
    lens, shared, _ = _fork_lens(c)
    w = c["width"]
    return _held(lens, c["page"]) - sum(shared) + sum(shared[::w]) + c["spare"]


def _compact_pages(c):
    """Pages of the pool, pages in use, and how many of them are expected behind the others."""
    used = _held(_lens(c["seqs"], c["kv_lo"], c["kv_hi"]), c["page"])
    pool = max(used, int(used / c["used"]))
    return pool, used, used * (pool - used) // pool


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[c["dtype"]])

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def cache(pages):
        """Keys and values of a pool as earlier tokens left them, and the scales of its pages."""
        s = {}
        for x in ("k", "v"):
            bits = torch.randint(0, 256, (pages, c["h_kv"], c["page"], c["d"]), generator=g, device=DEV, dtype=torch.uint8)
            # (0x7f and 0xff are no numbers; each power of two below 448 as often as the next)
            s[x + "_pages"] = torch.where(bits & 0x7f == 0x7f, bits - 8, bits).view(E4M3)
            s[x + "_scale"] = _two_to(torch.randint(-8, -5, (pages, c["h_kv"]), generator=g, device=DEV))
        return s

    def normal_cache(pages):
        """The same with normal values, rounded as ``write`` rounds them."""
        s = {}
        for x in ("k", "v"):
            y = torch.randn((pages, c["h_kv"], c["page"], c["d"]), generator=g, device=DEV)
            scale = _scale_for(y.abs().amax((2, 3)))
            s[x + "_pages"], s[x + "_scale"] = (y / scale[..., None, None]).to(E4M3), scale
            del y
        return s

    def table(lens, pages, most):
        """Sequences in pages of any order: [seqs, most], -1 behind each one's last."""
        n = _held(lens, c["page"])
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int64)[:n].to(torch.int32)
        out = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
        real = torch.arange(most, device=DEV) < ((ints(lens) + c["page"] - 1) // c["page"])[:, None]
        out[real] = order
        return out

    s = dict(case=c)
    if c["op"] == "norm":
        t, hq, hk, d = c["tokens"], c["h_q"], c["h_kv"], c["d"]
        if c["packed"]:
            qkv = normal(t, hq + 2 * hk, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(t, hq, d), normal(t, hk, d)
        s["wq"], s["wk"] = (1 + 0.1 * normal(d).float()).to(s["q"].dtype), (1 + 0.1 * normal(d).float()).to(s["q"].dtype)
        if c["backward"]:
            s["dq"], s["dk"] = normal(t, hq, d), normal(t, hk, d)
        at = torch.arange(t, device=DEV)
        start = torch.randint(0, c["far"], (c["axes"], 1), generator=g, device=DEV)
        if c["axes"] == 1:  # sequences of 512 tokens, each with a start of its own
            start = torch.randint(0, c["far"], (t // 512 + 1,), generator=g, device=DEV)
            pos = (start[at // 512] + at % 512).view(1, t)
        else:  # frames of 24 x 32 patches (the last axes are height and width)
            pos = torch.stack([at // 768, at // 32 % 24, at % 32])[3 - c["axes"]:] + start
        s["positions"] = pos.to(torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        s["sections"] = _sections(c["axes"], c["rot"])
        s["axis_of"] = torch.tensor([a for a, n in enumerate(s["sections"]) for _ in range(n)], device=DEV)
        return s
    if c["op"] == "fork":
        lens, shared, parents = _fork_lens(c)
        w, page, pool = c["width"], c["page"], _fork_pages(c)
        most = max(-(-(x + c["grow"]) // page) for x in lens)
        order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32).tolist()
        rows, at = [], 0
        for i, x in enumerate(lens):
            n, common = -(-x // page), shared[i]
            if i % w:  # the other beams of a request share its first pages
                row = rows[i - i % w][:common] + order[at:at + n - common]
                at += n - common
            else:
                row = order[at:at + n]
                at += n
            rows.append(row + [-1] * (most - n))
        s["table"], s["lens"], s["parents"] = ints(rows), ints(lens), ints(parents)
        s["grow"] = ints([c["grow"] if p >= 0 else 0 for p in parents])
        flat = s["table"].flatten().long()
        s["refs"] = torch.bincount(flat[flat >= 0], minlength=pool).to(torch.int32)
        s.update(cache(pool))
        return s
    if c["op"] == "compact":
        lens = _lens(c["seqs"], c["kv_lo"], c["kv_hi"])
        pool, used, _ = _compact_pages(c)
        s["table"] = table(lens, pool, max(-(-x // c["page"]) for x in lens))
        flat = s["table"].flatten().long()
        s["refs"] = torch.bincount(flat[flat >= 0], minlength=pool).to(torch.int32)
        s.update(cache(pool))
        return s
    q, kv = _qkv_lens(c)
    total, hk, d = sum(q), c["h_kv"], c["d"]
    pool = _held(kv, c["page"]) + 7
    s["table"] = table(kv, pool, max(-(-x // c["page"]) for x in kv))
    s["cu_q"], s["kv_lens"], s["max_q"] = ints(_cu(q)), ints(kv), max(q)
    if c["op"] == "write":
        s.update(cache(pool))
        qkv = normal(total, 4 * hk, d)  # k and v are slices of a fused projection
        s["k"], s["v"] = qkv[:, 2 * hk:3 * hk], qkv[:, 3 * hk:]
        return s
    s.update(normal_cache(pool))
    s["q"], s["scale"], s["max_kv"] = normal(total, c["h_q"], d), d ** -0.5, max(kv)
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    c = s["case"]
    half, d = c["rot"] // 2, c["d"]
    angle = s["positions"].double()[s["axis_of"]].t() * s["inv_freq"].double()  # [tokens, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(y, sin):
        r = y[..., :c["rot"]]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, y[..., c["rot"]:]], dim=-1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s["w" + name].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if not c["backward"]:
            out[name] = turn(x * r * w, sin).to(s[name].dtype)
            continue
        g = turn(s["d" + name].float(), -sin)
        out["dw" + name] = (g * x * r).sum((0, 1)).to(s["w" + name].dtype)
        g = g * w
        out["d" + name] = (g * r - x * (r ** 3) * (g * x).mean(-1, keepdim=True)).to(s[name].dtype)
    return out


def _scale_for(amax):
    """The smallest power of two, 2^-64 at least, times which 448 is not below amax."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-64)
    return _two_to(torch.where(amax > 0, e, torch.full_like(e, -64)))


def _tokens(s):
    """The sequence of each new token, and its place among the sequence's keys."""
    cu = s["cu_q"].long()
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), new)
    return seq, torch.arange(seq.numel(), device=DEV) - cu[seq] + (s["kv_lens"].long() - new)[seq]


def _plain_write(s):
    c = s["case"]
    seq, at = _tokens(s)
    page, slot = s["table"].long()[seq, at // c["page"]], at % c["page"]
    pool, hk = s["k_scale"].shape
    fresh = torch.zeros(pool, dtype=torch.bool, device=DEV)
    fresh[page[slot == 0]] = True
    touched = torch.unique(page)
    for name in ("k", "v"):
        x, pages, scale = s[name].float(), s[name + "_pages"], s[name + "_scale"]
        size = x.abs().amax(-1)
        top = torch.zeros((pool, hk), device=DEV).index_reduce_(
            0, page, torch.where(size.isfinite(), size, torch.zeros_like(size)), "amax")[touched]
        old, to = scale[touched], _scale_for(top)
        new = torch.where(fresh[touched][:, None], to, torch.maximum(old, to))
        rest = pages.view(torch.uint8)[touched].view(E4M3).float() * (old / new)[..., None, None]
        same = (old == new) | fresh[touched][:, None]
        rest = torch.where(same[..., None, None], pages.view(torch.uint8)[touched], rest.to(E4M3).view(torch.uint8))
        pages.view(torch.uint8)[touched] = rest
        scale[touched] = new
        pages.view(torch.uint8)[page, :, slot] = (x / scale[page][..., None]).to(E4M3).view(torch.uint8)
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale")}


def _plain_attend(s):
    c = s["case"]
    hk, d, n, m, most = c["h_kv"], c["d"], c["seqs"], s["max_q"], s["max_kv"]
    group = c["h_q"] // hk
    kv_len = s["kv_lens"].long()
    j = torch.arange(most, device=DEV)

    def keys(name):  # [n, hk, most, d], zero behind the last key
        page = s["table"].long()[:, j // c["page"]].clamp(min=0)
        x = s[name + "_pages"].view(torch.uint8)[page, :, (j % c["page"]).expand(n, most)].view(E4M3).float()
        x = x * s[name + "_scale"][page][..., None]
        return torch.where((j < kv_len[:, None])[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)

    cu = s["cu_q"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(m, device=DEV)
    real = i < q_len[:, None]
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]  # [n, m, h_q, d]
    q = q.view(n, m, hk, group, d).permute(0, 2, 1, 3, 4).reshape(n, hk, m * group, d)
    x = (q @ keys("k").transpose(2, 3)).view(n, hk, m, group, most) * s["scale"]
    diag = (i + (kv_len - q_len)[:, None])[:, None, :, None, None]
    ok = (j < kv_len.view(n, 1, 1, 1, 1)) & real.view(n, 1, m, 1, 1)
    if c["causal"]:
        ok = ok & (j <= diag)
    if c["window"] > 0:
        ok = ok & (j > diag - c["window"])
    x = x.masked_fill(~ok, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = (x - top).exp_()
    total = x.sum(-1)
    o = (x.view(n, hk, m * group, most) @ keys("v")).view(n, hk, m, group, d) / total.clamp(min=1e-30)[..., None]
    out = o.permute(0, 2, 1, 3, 4).reshape(n, m, c["h_q"], d)[real].to(s["q"].dtype)
    lse = (top[..., 0] + total.log()).permute(1, 3, 0, 2).reshape(c["h_q"], n, m)[:, real]
    return {"out": out, "lse": lse.contiguous()}


def _plain_copy(s, src, dst):
    real = src >= 0
    a, b = src[real].long(), dst[real].long()
    for name in ("k", "v"):
        pages = s[name + "_pages"].view(torch.uint8)
        pages[b] = pages[a]
        s[name + "_scale"][b] = s[name + "_scale"][a]
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale")}


def _plain_fork(s):
    c = s["case"]
    page, table, refs = c["page"], s["table"].long(), s["refs"].long()
    pool, most = refs.numel(), table.shape[1]
    j = torch.arange(most, device=DEV)
    lens, parents = s["lens"].long(), s["parents"].long()
    held = j < ((lens + page - 1) // page)[:, None]
    outside = refs - torch.bincount(table[held], minlength=pool)
    size = torch.where(parents >= 0, lens[parents.clamp(min=0)], torch.zeros_like(parents))
    rows = table[parents.clamp(min=0)]
    whole = j < (size // page)[:, None]
    shared = torch.bincount(rows[whole], minlength=pool)
    # a page that a sequence has begun stays with the first one that follows it; the others take copies
    part = size % page != 0
    last = torch.where(part, rows.gather(1, (size // page).clamp(max=most - 1)[:, None])[:, 0], torch.zeros_like(size))
    s_at = torch.arange(parents.numel(), device=DEV)
    first = torch.full((pool,), parents.numel(), device=DEV).index_reduce_(0, last[part], s_at[part], "amin")
    keeps = part & (first[last] == s_at) & (outside[last] == 0) & (shared[last] == 0)
    copies = part & ~keeps
    count = outside + shared + torch.bincount(last[keeps], minlength=pool)
    grown = size + s["grow"].long()
    more = (grown + page - 1) // page - (size + page - 1) // page
    need = more + copies
    free = (count == 0).nonzero()[:, 0]
    begin = need.cumsum(0) - need
    # entry j of a sequence: what it shares, the page that it keeps, or the next of its new ones
    k = j - (size // page)[:, None] - (keeps * 1)[:, None]
    new = (k >= 0) & (j < ((grown + page - 1) // page)[:, None])
    fresh = free[(begin[:, None] + k).clamp(0, max(0, free.numel() - 1))]
    out = torch.where(whole | (keeps[:, None] & (j == (size // page)[:, None])), rows, torch.full_like(rows, -1))
    out = torch.where(new, fresh, out)
    count = count + torch.bincount(fresh[new], minlength=pool)
    none = torch.full_like(parents, -1)
    src = torch.where(copies, last, none).int()
    dst = torch.where(copies, free[begin.clamp(max=max(0, free.numel() - 1))], none).int()
    got = {"table": out.int(), "lens": grown.int(), "refs": count.int(), "src": src, "dst": dst,
           "left": (free.numel() - need.sum()).int().view(1)}
    got.update(_plain_copy(s, src, dst))
    return got


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    pool = refs.numel()
    used = refs > 0
    front = torch.arange(pool, device=DEV) < used.sum()
    src, dst = (used & ~front).nonzero()[:, 0], (~used & front).nonzero()[:, 0]
    to = torch.where(used, torch.arange(pool, device=DEV), torch.full_like(refs, -1).long())
    to[src] = dst
    out = torch.where(table >= 0, to[table.clamp(min=0).long()], torch.full_like(table, -1).long()).int()
    count = torch.where(front & used, refs, torch.zeros_like(refs))
    count[dst] = refs[src]
    pad = torch.full((pool // 2, ), -1, dtype=torch.int32, device=DEV)
    a, b = pad.clone(), pad
    a[:src.numel()], b[:src.numel()] = src.int(), dst.int()
    got = {"table": out, "refs": count, "to": to.int(), "src": a, "dst": b, "used": used.sum().int().view(1)}
    got.update(_plain_copy(s, a, b))
    return got


# ------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "write": _plain_write, "attend": _plain_attend, "fork": _plain_fork,
                "compact": _plain_compact}[op](s)
    import variable_length_flash_gb300 as vlf
    if op == "norm":
        if c["backward"]:
            dq, dk, dwq, dwk = vlf.vlf_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"],
                                                     s["inv_freq"], sections=s["sections"],
                                                     interleaved=c["interleaved"], eps=EPS)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        q, k = vlf.vlf_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                                 sections=s["sections"], interleaved=c["interleaved"], eps=EPS)
        return {"q": q, "k": k}
    pages = [s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale")]
    if op == "write":
        vlf.vlf_pages_write(s["k"], s["v"], *pages, s["table"], s["cu_q"], s["kv_lens"])
        return dict(zip(("k_pages", "v_pages", "k_scale", "v_scale"), pages))
    if op == "attend":
        out, lse = vlf.vlf_attn_varlen_fwd_pages(s["q"], *pages, s["table"], s["cu_q"], s["kv_lens"], s["max_q"],
                                                 scale=s["scale"], causal=c["causal"], window=c["window"])
        return {"out": out, "lse": lse}
    if op == "fork":
        names = ("table", "lens", "refs", "src", "dst", "left")
        got = dict(zip(names, vlf.vlf_pages_fork(s["table"], s["lens"], s["refs"], s["parents"], s["grow"], c["page"])))
    else:
        names = ("table", "refs", "to", "src", "dst", "used")
        got = dict(zip(names, vlf.vlf_pages_compact(s["table"], s["refs"])))
    vlf.vlf_pages_copy(*pages, got["src"], got["dst"])
    got.update(zip(("k_pages", "v_pages", "k_scale", "v_scale"), pages))
    return got


# ------------------------------------------------------------------------------ in 64 bits
def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to the even one (|x| <= 448)."""
    _, e = torch.frexp(x)
    step = ((e.long() - 4).clamp(min=-9) + 1023 << 52).view(torch.float64)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "norm":
        half, d = c["rot"] // 2, c["d"]
        turns = torch.empty(c["tokens"], half, dtype=torch.float64, device=DEV)
        first = 0
        for a, n in enumerate(s["sections"]):
            turns[:, first:first + n] = torch.outer(s["positions"][a].double(), s["inv_freq"][first:first + n].double())
            first += n

        def turn(x, sign):
            z = torch.polar(torch.ones_like(turns), sign * turns)[:, None]
            y = x.clone()
            lo, hi = (y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]) if c["interleaved"] else (y[..., :half], y[..., half:c["rot"]])
            t = torch.complex(lo.contiguous(), hi.contiguous()) * z
            lo.copy_(t.real), hi.copy_(t.imag)
            return y

        got = {}
        for name in ("q", "k"):
            x, w = s[name].double(), s["w" + name].double()
            size = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
            if not c["backward"]:
                got[name] = turn(x / size * w, 1.0)
                continue
            g = turn(s["d" + name].double(), -1.0)
            got["dw" + name] = torch.einsum("thd,thd->d", g, x / size)
            unit = x / size
            got["d" + name] = (g * w - unit * torch.einsum("thd,thd->th", g * w, unit)[..., None] / d) / size
        return got
    page = c["page"]
    if op == "attend":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(c["h_q"], s["q"].shape[0], dtype=torch.float64, device=DEV)
        cu, group = s["cu_q"].tolist(), c["h_q"] // c["h_kv"]
        for n, kl in enumerate(s["kv_lens"].tolist()):
            a, b = cu[n], cu[n + 1]
            ids = s["table"][n, :-(-kl // page)].long()
            k, v = [(s[x + "_pages"][ids].double() * s[x + "_scale"][ids].double()[..., None, None]).transpose(0, 1)
                    .reshape(c["h_kv"], -1, c["d"])[:, :kl] for x in ("k", "v")]
            at = torch.arange(b - a, device=DEV)[:, None] + (kl - (b - a))
            j = torch.arange(kl, device=DEV)[None]
            no = (j > at) if c["causal"] else torch.zeros_like(j > at)
            if c["window"] > 0:
                no = no | (j <= at - c["window"])
            for h in range(c["h_q"]):
                x = (s["q"][a:b, h].double() @ k[h // group].t() * s["scale"]).masked_fill(no, -math.inf)
                lse[h, a:b] = torch.logsumexp(x, -1)
                out[a:b, h] = torch.softmax(x, -1) @ v[h // group]
        return {"out": out, "lse": lse}
    cache = ("k_pages", "v_pages", "k_scale", "v_scale")
    if op == "write":
        got = {x: s[x].double() for x in cache}
        cu, lens, rows = s["cu_q"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
        for n in range(len(lens)):
            first = lens[n] - (cu[n + 1] - cu[n])
            for p in range(first // page, -(-lens[n] // page)):
                a, b = max(first, p * page), min(lens[n], (p + 1) * page)
                t, i = slice(cu[n] + a - first, cu[n] + b - first), rows[n][p]
                for x in ("k", "v"):
                    y = s[x][t].double().transpose(0, 1)  # [heads, tokens, d]
                    top = y.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(top / 448)).clamp(min=-64).long()
                    scale = (e + 1023 << 52).view(torch.float64)
                    # (the logarithm may be off by a little)
                    scale = torch.where(scale * 224 >= top, scale / 2, torch.where(scale * 448 < top, scale * 2, scale))
                    scale = scale.clamp(min=2.0 ** -64)
                    if a > p * page:
                        was = got[x + "_scale"][i].clone()
                        scale = torch.maximum(scale, was)
                        got[x + "_pages"][i] = _e4m3(got[x + "_pages"][i] * (was / scale)[:, None, None])
                    got[x + "_scale"][i] = scale
                    got[x + "_pages"][i][:, a - p * page:b - p * page] = _e4m3(y / scale[:, None, None])
        return got
    table, refs = s["table"].tolist(), s["refs"].tolist()
    if op == "fork":
        lens, parents, grow = s["lens"].tolist(), s["parents"].tolist(), s["grow"].tolist()
        outside = list(refs)
        for row, x in zip(table, lens):
            for p in row[:-(-x // page)]:
                outside[p] -= 1
        count, shared = list(outside), set()
        for p in parents:
            for i in table[p][:lens[p] // page] if p >= 0 else []:
                count[i] += 1
                shared.add(i)
        kept, rows, todo = set(), [], []
        for n, p in enumerate(parents):
            x = lens[p] if p >= 0 else 0
            row, copy = (table[p][:x // page] if p >= 0 else []), None
            if x % page:
                last = table[p][x // page]
                if outside[last] == 0 and last not in shared and last not in kept:
                    kept.add(last)
                    count[last] += 1
                    row = row + [last]
                else:
                    copy = last
            rows.append(row)
            todo.append((copy, -(-(x + grow[n]) // page) - len(row), x + grow[n]))
        free = [i for i, n in enumerate(count) if n == 0]
        src, dst = [], []
        for row, (copy, more, _) in zip(rows, todo):
            src.append(-1 if copy is None else copy)
            dst.append(-1 if copy is None else free[0])
            for i in free[:more]:
                count[i] += 1
            row += free[:more]
            free = free[more:]
        most = len(table[0])
        got = {"table": [r + [-1] * (most - len(r)) for r in rows], "lens": [x for _, _, x in todo], "refs": count,
               "src": src, "dst": dst, "left": [len(free)]}
    else:
        n = sum(1 for x in refs if x > 0)
        src = [i for i in range(n, len(refs)) if refs[i] > 0]
        dst = [i for i in range(n) if refs[i] == 0]
        to = [i if x > 0 else -1 for i, x in enumerate(refs)]
        count = refs[:n] + [0] * (len(refs) - n)
        for a, b in zip(src, dst):
            to[a], count[b] = b, refs[a]
        pad = [-1] * (len(refs) // 2 - len(src))
        got = {"table": [[to[i] if i >= 0 else -1 for i in r] for r in table], "refs": count, "to": to, "src": src + pad,
               "dst": dst + pad, "used": [n]}
    got = {k: torch.tensor(v, dtype=torch.int32, device=DEV) for k, v in got.items()}
    got.update({x: s[x] for x in cache})
    for a, b in zip(got["src"].tolist(), got["dst"].tolist()):
        if a >= 0:
            for x in cache:
                s[x].view(torch.uint8)[b] = s[x].view(torch.uint8)[a]
    return got
