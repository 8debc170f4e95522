"""The norm of each head with its rotary positions (vlf_norm_rope, norm_rotary_embedding) and its gradients
against the fp64 definition: types, pair layouts, axes, partial rotation, odd widths, strided tokens,
weights of either type or none, in place, gradients against the formula and against differences.

Tolerances.  u is half a step of the type (UNIT), |x|' below the normed value.  The sum of squares of at
most 256 numbers is added in at most 21 steps (16 in a lane, 5 over lanes), all terms positive: 21 2^-24
relative, half of that in r, whose root adds 2^-22; r, w and their product 3 2^-24: below 2^-20 in all.  The
rotation adds 2^-20 (|a| + |b|) (as in test_rope.py).  Forward: u |y| + 2^-19 (|a| + |b|), a and b the
normed pair.  Backward: with G = |g_a| + |g_b| of the pair, g is off by 2^-20 G, each term of
dx = r (g w - n mean(g w n)) by less than 2^-18 of its size, n the normed row without weight: the mean
adds 21 more steps, 2^-19.  dw: the same for each term and 2^-24 of the sum of sizes for each of the n
additions that one chain has."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUBNORMAL = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
EPS = 1e-6


def np64(t):
    return t.detach().cpu().double().numpy()


def mate(a, rot, inter):
    """|a| + |the other of its pair|."""
    b, half = np.zeros_like(a), rot // 2
    if inter:
        b[..., 0:rot:2], b[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
    else:
        b[..., :half], b[..., half:rot] = a[..., half:rot], a[..., :half]
    return np.abs(a) + np.abs(b)


def make(tokens, hq, hk, d, rot, dtype, axes, far, seed, w_dtype=None, size=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(q=(size * r(tokens, hq, d)).to(dtype).cuda(), k=(size * r(tokens, hk, d)).to(dtype).cuda())
    c["wq"], c["wk"] = ((1 + 0.3 * r(d)).to(w_dtype or dtype).cuda() for _ in range(2))
    c["pos"] = torch.randint(min(far, 0), abs(far), (axes, tokens), generator=g, dtype=torch.int32).cuda()
    half = rot // 2
    c["f"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()
    sec = [half // axes] * axes
    sec[-1] += half - sum(sec)
    c["sec"], c["rot"] = sec, rot
    return c


def turn(c):
    return c["pos"].cpu().numpy(), c["f"].cpu().numpy(), c["sec"], c["rot"]


def check_forward(y, x, w, c, inter, eps=EPS):
    a = np64(x)
    wn = np.ones(a.shape[-1]) if w is None else np64(w)
    want = ref.norm_rope(a, wn, eps, *turn(c), inter)
    n = a / np.sqrt((a * a).mean(-1, keepdims=True) + eps) * wn
    tol = UNIT[y.dtype] * np.abs(want) + 2.0 ** -19 * mate(n, c["rot"], inter) + SUBNORMAL[y.dtype]
    assert (np.abs(np64(y) - want) <= tol).all(), np.abs(np64(y) - want).max()


def check_backward(dx, dw, dy, x, w, c, inter, eps=EPS):
    a, g = np64(x), np64(dy)
    wn = np.ones(a.shape[-1]) if w is None else np64(w)
    want, want_w = ref.norm_rope_bwd(g, a, wn, eps, *turn(c), inter)
    r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    n, G = np.abs(a * r), mate(g, c["rot"], inter)
    sizes = r * (G * np.abs(wn) + n * (G * np.abs(wn) * n).mean(-1, keepdims=True))
    tol = UNIT[dx.dtype] * np.abs(want) + 2.0 ** -17 * sizes + SUBNORMAL[dx.dtype]
    assert (np.abs(np64(dx) - want) <= tol).all(), np.abs(np64(dx) - want).max()
    if w is not None:
        chain = a.shape[0] * a.shape[1]
        tol = UNIT[dw.dtype] * np.abs(want_w) + (2.0 ** -18 + chain * 2.0 ** -24) * (G * n).sum((0, 1)) + SUBNORMAL[dw.dtype]
        assert dw.dtype == w.dtype and (np.abs(np64(dw) - want_w) <= tol).all()


CASES = [
    # tokens, hq, hk, d, rot, axes, interleaved, far
    (1, 1, 1, 2, 2, 1, False, 100),
    (1, 1, 1, 1, 0, 1, False, 100),           # one column
    (1, 32, 8, 128, 128, 1, False, 1000000),
    (7, 3, 1, 64, 64, 3, False, 4000),
    (33, 8, 2, 96, 64, 1, True, 131072),      # six lanes of eight have columns
    (65, 4, 4, 80, 48, 2, True, 4000),
    (19, 5, 2, 40, 40, 4, False, 4000),       # half of 20 pairs: no whole 16-byte chunk
    (13, 2, 1, 33, 10, 1, True, 4000),        # odd width, scalar path
    (21, 2, 2, 251, 250, 1, False, 4000),     # more pairs than lanes
    (9, 2, 2, 24, 0, 1, False, 4000),         # nothing turns: an odd number of chunks
    (257, 16, 16, 128, 128, 3, False, 32768),
    (3000, 8, 8, 64, 32, 1, False, 2 ** 31 - 1),
    (50, 2, 2, 256, 256, 2, True, -70000),
    (3, 70, 1, 64, 64, 1, False, 4000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,axes,inter,far", CASES)
def test_forward_and_gradients_match_the_definition(tokens, hq, hk, d, rot, axes, inter, far, dtype):
    w_dtype = torch.float32 if tokens % 2 else None
    c = make(tokens, hq, hk, d, rot, dtype, axes, far, seed=tokens + d, w_dtype=w_dtype)
    args = (c["wq"], c["wk"], c["pos"], c["f"], c["sec"], inter, EPS)
    yq, yk = vlf.vlf_norm_rope(c["q"], c["k"], *args)
    check_forward(yq, c["q"], c["wq"], c, inter)
    check_forward(yk, c["k"], c["wk"], c, inter)
    g = torch.Generator().manual_seed(1)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (yq, yk))
    got = vlf.vlf_norm_rope_bwd(dq, dk, c["q"], c["k"], *args)
    check_backward(got[0], got[2], dq, c["q"], c["wq"], c, inter)
    check_backward(got[1], got[3], dk, c["k"], c["wk"], c, inter)
    # (sums in a fixed order: the same bits again)
    again = vlf.vlf_norm_rope_bwd(dq, dk, c["q"], c["k"], *args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["q", "k", "none"])
def test_weights_that_are_not_there(which):
    c = make(40, 4, 2, 64, 64, torch.bfloat16, 1, 500, seed=2)
    wq, wk = c["wq"] if which == "q" else None, c["wk"] if which == "k" else None
    args = (wq, wk, c["pos"], c["f"], c["sec"], False, EPS)
    yq, yk = vlf.vlf_norm_rope(c["q"], c["k"], *args)
    check_forward(yq, c["q"], wq, c, False), check_forward(yk, c["k"], wk, c, False)
    dq, dk, dwq, dwk = vlf.vlf_norm_rope_bwd(yk.new_ones(yq.shape), yk, c["q"], c["k"], *args)
    assert (dwq is None) == (wq is None) and (dwk is None) == (wk is None)
    check_backward(dq, dwq, torch.ones_like(yq), c["q"], wq, c, False)
    check_backward(dk, dwk, yk, c["k"], wk, c, False)


@pytest.mark.gpu
def test_norm_alone_no_keys_and_no_tokens():
    c = make(11, 3, 1, 128, 0, torch.float16, 1, 10, seed=3)
    y, none = vlf.vlf_norm_rope(c["q"], None, c["wq"], None)
    assert none is None
    check_forward(y, c["q"], c["wq"], c, False)
    dx, dk, dw, dwk = vlf.vlf_norm_rope_bwd(y, None, c["q"], None, c["wq"], None)
    assert dk is None and dwk is None
    check_backward(dx, dw, y, c["q"], c["wq"], c, False)
    e = torch.empty(0, 3, 128, dtype=torch.float16, device="cuda")
    dx, dk, dw, dwk = vlf.vlf_norm_rope_bwd(e, e[:, :1], e, e[:, :1], c["wq"], c["wk"], c["pos"][0, :0], torch.rand(64).cuda())
    assert dx.shape == e.shape and not dw.any() and not dwk.any()
    assert vlf.vlf_norm_rope(e, None, None, None)[0].shape == e.shape


@pytest.mark.gpu
@pytest.mark.parametrize("eps,size", [(0.0, 1.0), (1e-6, 0.0), (1e-5, 1e-3), (1e-6, 3e3)])
def test_eps_and_sizes(eps, size):
    """Rows of zeros (eps carries them), rows as small as eps, rows whose squares fp16 cannot hold."""
    c = make(17, 2, 2, 96, 96, torch.float16, 1, 100, seed=4, size=size)
    y, _ = vlf.vlf_norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["pos"], c["f"], c["sec"], eps=eps)
    check_forward(y, c["q"], c["wq"], c, False, eps)
    g = torch.ones_like(y) * 2.0 ** -10  # (gradients of rows near zero are large: fp16 has to hold them)
    dq, dk, dwq, dwk = vlf.vlf_norm_rope_bwd(g, g, c["q"], c["k"], c["wq"], c["wk"], c["pos"], c["f"], c["sec"], eps=eps)
    check_backward(dq, dwq, g, c["q"], c["wq"], c, False, eps)


@pytest.mark.gpu
def test_a_row_that_is_not_finite_stays_by_itself():
    c = make(9, 4, 2, 64, 64, torch.bfloat16, 1, 100, seed=5)
    args = (c["wq"], c["wk"], c["pos"], c["f"], c["sec"])
    want = vlf.vlf_norm_rope(c["q"], c["k"], *args)[0]
    q = c["q"].clone()
    q[3, 1, 7], q[5, 0, 2] = float("nan"), float("inf")
    got = vlf.vlf_norm_rope(q, c["k"], *args)[0]
    other = torch.ones(9, 4, dtype=torch.bool)
    other[3, 1] = other[5, 0] = False
    assert got[3, 1].isnan().all() and torch.equal(got[other.cuda()], want[other.cuda()])


@pytest.mark.gpu
def test_packed_slices_in_place_and_odd_strides():
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(70, 12, 64, generator=g).to(torch.bfloat16).cuda()
    c = make(70, 8, 2, 64, 64, torch.bfloat16, 1, 1000, seed=6)
    q, k, args = qkv[:, :8], qkv[:, 8:10], (c["wq"], c["wk"], c["pos"], c["f"], c["sec"])
    yq, yk = vlf.vlf_norm_rope(q.contiguous(), k.contiguous(), *args)
    check_forward(yq, q, c["wq"], c, False)
    assert all(torch.equal(a, b) for a, b in zip(vlf.vlf_norm_rope(q, k, *args), (yq, yk)))
    buf = torch.zeros_like(qkv)
    vlf.vlf_norm_rope(q, k, *args, q_out=buf[:, :8], k_out=buf[:, 8:10])
    assert torch.equal(buf[:, :8], yq) and torch.equal(buf[:, 8:10], yk) and not buf[:, 10:].any()
    want = vlf.vlf_norm_rope_bwd(yq, yk, q, k, *args)
    got = vlf.vlf_norm_rope_bwd(buf[:, :8], buf[:, 8:10], q, k, *args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dq, dk = yq.clone(), yk.clone()  # the gradients over those of the outputs
    vlf.vlf_norm_rope_bwd(dq, dk, q, k, *args, dq=dq, dk=dk)
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
    a = qkv.clone()
    vlf.vlf_norm_rope(a[:, :8], a[:, 8:10], *args, q_out=a[:, :8], k_out=a[:, 8:10])
    assert torch.equal(a[:, :8], yq) and torch.equal(a[:, 8:10], yk) and torch.equal(a[:, 10:], qkv[:, 10:])
    odd = torch.zeros(70, 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")  # the element path
    view = odd[:, :512].view(70, 8, 64)
    view.copy_(q)
    y = vlf.vlf_norm_rope(view, None, c["wq"], None, *args[2:])[0]
    check_forward(y, q, c["wq"], c, False)
    # slices of weights, positions and frequencies start anywhere
    shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:]  # noqa: E731
    got = vlf.vlf_norm_rope(q, k, shift(c["wq"]), shift(c["wk"]), shift(c["pos"]), shift(c["f"]), c["sec"])
    assert torch.equal(got[0], yq) and torch.equal(got[1], yk)


@pytest.mark.gpu
def test_autograd_against_formula_and_differences():
    c = make(21, 4, 2, 48, 32, torch.float32, 2, 300, seed=5)
    leaves = [c[x].requires_grad_() for x in ("q", "k", "wq", "wk")]
    gq, gk = torch.randn_like(c["q"]), torch.randn_like(c["k"])
    call = lambda *x: vlf.norm_rotary_embedding(*x, c["pos"], c["f"], c["sec"], interleaved=True)  # noqa: E731
    yq, yk = call(*leaves)
    ((yq * gq).sum() + (yk * gk).sum()).backward()
    check_backward(c["q"].grad, c["wq"].grad, gq, c["q"], c["wq"], c, True)
    check_backward(c["k"].grad, c["wk"].grad, gk, c["k"], c["wk"], c, True)
    # a difference of step h along a direction: the definition's second difference, h^2 / 2 |f''| with |f''|
    # of the size of |g| |dx|^2 / |x|^2 (about 1 here), and the forward's rounding over h
    with torch.no_grad():
        for i, t in enumerate(leaves):
            e, h = torch.randn_like(t), 2.0 ** -8
            up, down = ([x + s * h * e if j == i else x for j, x in enumerate(leaves)] for s in (1, -1))
            (uq, uk), (dq, dk) = call(*up), call(*down)
            num = (((uq.double() - dq.double()) * gq.double()).sum() + ((uk.double() - dk.double()) * gk.double()).sum()) / (2 * h)
            size = gq.abs().double().sum() + gk.abs().double().sum()
            assert abs(num - (t.grad.double() * e.double()).sum()) <= size * (2.0 ** -12 + 2.0 ** -18 / h)


@pytest.mark.gpu
def test_gradient_of_a_shared_weight_and_of_slices():
    """One weight for q and k gets the sum of both; a packed projection gets its slices' gradients."""
    c = make(30, 4, 2, 64, 64, torch.float32, 1, 300, seed=8)
    qkv = torch.cat([c["q"], c["k"], c["k"]], 1).requires_grad_()
    w = c["wq"].clone().requires_grad_()
    yq, yk = vlf.norm_rotary_embedding(qkv[:, :4], qkv[:, 4:6], w, w, c["pos"], c["f"], c["sec"])
    (yq.sum() + (yk * yk.detach()).sum()).backward()
    got = vlf.vlf_norm_rope_bwd(torch.ones_like(yq), yk.detach(), c["q"], c["k"], w, w, c["pos"], c["f"], c["sec"])
    assert torch.equal(qkv.grad[:, :4], got[0]) and torch.equal(qkv.grad[:, 4:6], got[1]) and not qkv.grad[:, 6:].any()
    assert torch.equal(w.grad, got[2] + got[3])


@pytest.mark.gpu
def test_captured_backward_replays_on_new_values():
    c = make(300, 8, 2, 128, 128, torch.bfloat16, 1, 1000, seed=9)
    dq, dk = torch.randn_like(c["q"]), torch.randn_like(c["k"])
    args = (c["wq"], c["wk"], c["pos"], c["f"], c["sec"])
    call = lambda: (*vlf.vlf_norm_rope(c["q"], c["k"], *args), *vlf.vlf_norm_rope_bwd(dq, dk, c["q"], c["k"], *args))  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for t in (c["q"], c["k"], dq, dk, c["wq"]):
        t.copy_(torch.randn_like(t))
    want = call()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def raw(backward=False, **kw):
    """The C entry point's status for arguments that are refused before anything is enqueued (no memory behind them)."""
    a = dict(q=16, qs=512, k=16, ks=128, wq=16, wk=16, wd=1, eps=1e-6, pos=16, axes=1, sec=None, f=16, total=4, hq=4, hk=1,
             d=128, rot=128, dtype=1, inter=0, qo=32, qos=512, ko=32, kos=128, dqo=16, dko=16, dwq=16, dwk=16, ws=16, wsn=1 << 30)
    a.update(kw)
    mid = [a[x] for x in ("q", "qs", "k", "ks", "wq", "wk", "wd", "eps", "pos", "axes", "sec", "f", "total", "hq", "hk", "d",
                          "rot", "dtype", "inter", "qo", "qos", "ko", "kos")]
    if backward:
        return vlf._lib.vlf_norm_rope_bwd(a["dqo"], 512, a["dko"], 128, *mid, a["dwq"], a["dwk"], a["ws"], a["wsn"], None)
    return vlf._lib.vlf_norm_rope(*mid, None)


REFUSED = [
    (dict(total=-1), -1), (dict(hq=0), -1), (dict(hk=-1), -1), (dict(d=0), -1), (dict(rot=130), -1), (dict(rot=3), -1),
    (dict(dtype=3), -1), (dict(wd=0), -1), (dict(wd=7), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(axes=0), -1), (dict(axes=5), -1), (dict(axes=2), -1), (dict(d=257, rot=2), -2),
    (dict(hq=65536), -2), (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(pos=None), -1), (dict(f=None), -1), (dict(qs=-1), -1), (dict(qos=511), -1), (dict(kos=127), -1), (dict(q=8), -3),
    (dict(wq=8), -3), (dict(qo=40), -3), (dict(qo=16, qos=1024), -1), (dict(ko=16, kos=256), -1)]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_refusals_before_any_launch(kw, status):
    assert raw(**kw) == status
    assert raw(True, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(dqo=None), -1), (dict(dko=None), -1), (dict(wq=None), -1), (dict(wk=None), -1),
                                       (dict(ws=None), -7), (dict(wsn=100), -7), (dict(dwq=8), -3), (dict(dqo=8), -3)])
def test_refusals_of_the_backward(kw, status):
    assert raw(True, **kw) == status


@pytest.mark.gpu
def test_refusals_with_tensors():
    c = make(4, 4, 2, 64, 64, torch.bfloat16, 1, 100, seed=1)
    q, k, wq, wk, pos, f = (c[x] for x in ("q", "k", "wq", "wk", "pos", "f"))
    for bad in [lambda: vlf.vlf_norm_rope(q, k, wq[:32], wk, pos, f), lambda: vlf.vlf_norm_rope(q, k, wq.half(), wk, pos, f),
                lambda: vlf.vlf_norm_rope(q, k, wq.float(), wk, pos, f), lambda: vlf.vlf_norm_rope(q, k.float(), wq, wk, pos, f),
                lambda: vlf.vlf_norm_rope(q, k[:3], wq, wk, pos, f), lambda: vlf.vlf_norm_rope(q, k, wq, wk, pos, None),
                lambda: vlf.vlf_norm_rope(q, k, wq, wk, pos.long(), f), lambda: vlf.vlf_norm_rope(q, k, wq, wk, pos[:, :3], f),
                lambda: vlf.vlf_norm_rope(q, None, wq, wk, pos, f), lambda: vlf.vlf_norm_rope(q, k, wq, wk, pos, f, eps=-1.0),
                lambda: vlf.vlf_norm_rope(q.transpose(1, 2), k, wq, wk, pos, f), lambda: vlf.vlf_norm_rope(q.cpu(), k, wq, wk, pos, f),
                lambda: vlf.vlf_norm_rope(q, k, wq.cpu(), wk, pos, f), lambda: vlf.vlf_norm_rope(q.double(), k, wq, wk, pos, f),
                lambda: vlf.vlf_norm_rope(q, k, wq, wk, pos, f, sections=(10, 22)),
                lambda: vlf.vlf_norm_rope_bwd(q, None, q, k, wq, wk, pos, f), lambda: vlf.vlf_norm_rope_bwd(q[:3], k, q, k, wq, wk, pos, f),
                lambda: vlf.vlf_norm_rope_bwd(q, k, q, k, None, wk, pos, f, dq_weight=wq),
                lambda: vlf.norm_rotary_embedding(q, k, wq, wk, pos, f.clone().requires_grad_())]:
        with pytest.raises((vlf.VlfError, TypeError, AttributeError)):
            bad()
