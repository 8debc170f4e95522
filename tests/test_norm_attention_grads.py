"""Gradients of norm, rotary positions and attention together, element by element, against 64-bit ones.

Tolerance.  Each stage adds relative errors to sums of products, so an element is off by a share of what the same chain
gives for absolute values throughout (no term cancels another): that is formed here beside the gradients.  The shares, in
fp32 with products of three tf32 passes: a product's sum 2^-19; logits 2^-19 of sum |q k| scale <= |q| |k| scale, which the
norm holds to 8 times the weights, so weights P to 2 x 2^-16 x max|w|^2; norms, turns and roundings of q, k, v and their
gradients 2^-20 each.  With weights up to 2 they add up to less than 2^-13 + 2^-16; the bound is 2^-12."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf

F64 = torch.float64
EPS = 1e-6


def turned(x, pos, f, absolute=False, back=False):
    """Rotary positions over x [T, H, D], halves as pairs; absolute: with the sizes of sine and cosine, all added."""
    a = pos.double()[:, None] * f.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    h = f.numel()
    l, r, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    if absolute:
        c, s = c.abs(), s.abs()
        return torch.cat([l * c + r * s, l * s + r * c, rest], -1)
    if back:
        s = -s
    return torch.cat([l * c - r * s, l * s + r * c, rest], -1)


def normed(x, w, pos, f):
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return turned(x * r * w, pos, f)


def weights(q, k, scale, window):
    """P [H, Tq, Tk] of one sequence, causal."""
    g = q.shape[1] // k.shape[1]
    s = scale * torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1))
    i, j = torch.arange(q.shape[0])[:, None], torch.arange(k.shape[0])[None]
    ok = (j <= i) & ((j > i - window) if window else torch.ones_like(j <= i))
    return torch.where(ok, s, torch.full_like(s, -np.inf)).softmax(-1)


def attend(q, k, v, cu, window):
    out = []
    for a, b in zip(cu, cu[1:]):
        p = weights(q[a:b], k[a:b], q.shape[2] ** -0.5, window)
        out.append(torch.einsum("hij,jhd->ihd", p, v[a:b].repeat_interleave(q.shape[1] // v.shape[1], 1)))
    return torch.cat(out)


def sizes(x, w, go, pos, f, cu, hq, hkv, window):
    """The gradients' chain over absolute values: of qkv, wq, wk."""
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    yq, yk = normed(q, w[0], pos, f), normed(k, w[1], pos, f)
    g, scale = hq // hkv, q.shape[2] ** -0.5
    aq, ak, av = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    shared = lambda t: t.unflatten(1, (hkv, g)).sum(2)  # noqa: E731
    for a, b in zip(cu, cu[1:]):
        p = weights(yq[a:b], yk[a:b], scale, window)
        kk, vv = (t[a:b].abs().repeat_interleave(g, 1) for t in (yk, v))
        dp = torch.einsum("ihd,jhd->hij", go[a:b].abs(), vv)
        ds = p * (dp + (p * dp).sum(-1, keepdim=True))
        av[a:b] = shared(torch.einsum("hij,ihd->jhd", p, go[a:b].abs()))
        aq[a:b] = scale * torch.einsum("hij,jhd->ihd", ds, kk)
        ak[a:b] = scale * shared(torch.einsum("hij,ihd->jhd", ds, yq[a:b].abs()))
    grads, dws = [], []
    for t, wt, at in ((q, w[0], aq), (k, w[1], ak)):
        r = (t.square().mean(-1, keepdim=True) + EPS).rsqrt()
        gt = turned(at, pos, f, absolute=True)
        dws.append((gt * t.abs() * r).sum((0, 1)))
        gw = gt * wt.abs()
        grads.append(r * gw + t.abs() * r ** 3 * (gw * t.abs()).mean(-1, keepdim=True))
    return torch.cat([*grads, av], 1), *dws


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,rot,lens,window", [(4, 2, 64, 64, [20, 17], 0), (3, 1, 64, 32, [1, 130, 9], 0), (4, 4, 32, 16, [70, 33], 20),
                                                      (2, 2, 64, 64, [257], 0)])
def test_every_element_of_the_gradients(hq, hkv, d, rot, lens, window):
    g = torch.Generator().manual_seed(hq + d + len(lens))
    t = sum(lens)
    x = torch.randn(t, hq + 2 * hkv, d, generator=g) * torch.exp2(torch.randint(-2, 3, (t, 1, 1), generator=g).float())
    w = [1 + 0.2 * torch.randn(d, generator=g).clamp(-4, 4) for _ in range(2)]
    go = torch.randn(t, hq, d, generator=g)
    f = (10000.0 ** (-torch.arange(rot // 2, dtype=F64) / (rot // 2))).float()
    cu = [0] + [int(c) for c in np.cumsum(lens)]
    pos = torch.cat([torch.arange(n) for n in lens]).int()

    qkv, wq, wk = (a.cuda().requires_grad_() for a in (x, *w))
    q, k = vlf.norm_rotary_embedding(qkv[:, :hq], qkv[:, hq:hq + hkv], wq, wk, pos.cuda(), f.cuda(), eps=EPS)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = vlf.varlen_attention(q, k, qkv[:, hq + hkv:], cu_t, cu_t, max(lens), max(lens), causal=True, window=window)
    out.backward(go.cuda())

    def loss(x, wq, wk):
        q, k = normed(x[:, :hq], wq, pos, f), normed(x[:, hq:hq + hkv], wk, pos, f)
        return (attend(q, k, x[:, hq + hkv:], cu, window) * go.double()).sum()

    leaves = [a.double().requires_grad_() for a in (x, *w)]
    loss(*leaves).backward()
    bounds = sizes(x.double(), [a.double() for a in w], go.double(), pos, f, cu, hq, hkv, window)
    for got, want, size in zip((qkv, wq, wk), leaves, bounds):
        off = (got.grad.cpu().double() - want.grad).abs()
        assert (off <= 2.0 ** -12 * size + 1e-30).all(), (off / (2.0 ** -12 * size)).max()
    # the 64-bit gradients are those of the loss: differences in a direction, off by h^2 of a third derivative (which 64 times
    # the chain's absolute values hold, with h at 2^-10 of it) and 2^-50 of the loss's terms over h
    with torch.no_grad():
        for i, size in enumerate(bounds):
            e, h = torch.randn(leaves[i].shape, generator=g, dtype=F64), 2.0 ** -14
            ends = [loss(*[a + s * h * e if n == i else a for n, a in enumerate(leaves)]) for s in (1, -1)]
            num, room = (ends[0] - ends[1]) / (2 * h), (size * e.abs()).sum()
            assert (num - (leaves[i].grad * e).sum()).abs() <= 2.0 ** -14 * room + 2.0 ** -30 * go.abs().sum()


@pytest.mark.gpu
@pytest.mark.parametrize("t,hk", [(5, 0), (0, 2), (0, 0)])
def test_the_weights_of_no_rows_have_no_gradient(t, hk):
    """What the forward takes, the backward takes: keys without heads, calls without tokens."""
    d = 64
    q, k = (torch.randn(t, h, d, device="cuda", requires_grad=True) for h in (2, hk))
    wq, wk = (torch.ones(d, device="cuda", requires_grad=True) for _ in range(2))
    yq, yk = vlf.norm_rotary_embedding(q, k, wq, wk)
    (yq * yq.detach()).sum().add((yk * yk.detach()).sum()).backward()
    assert q.grad.shape == q.shape and k.grad.shape == k.shape
    assert not wk.grad.any() and bool(wq.grad.any()) == (t > 0)
    assert not wq.grad.isnan().any() and vlf.vlf_check_error() == 0
