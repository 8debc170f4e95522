"""Rotary positions (vlf_rope, rotary_embedding) against the fp64 definition: types, pair layouts,
axes, partial rotation, odd widths, strided tokens, far and negative positions, in place, gradients.

Tolerance.  A sine or cosine is off by at most 2^-21: the turn's fraction is rounded to 2^-33 and to
fp32 (half an ulp of at most 2^-24 half turns, pi 2^-24 radians), and sincospi itself by 2 ulp
(2^-22).  Two products and their sum add 2^-23 (|a| + |b|) at most, the output half a step of its
type: |error| <= u |y| + (|a| + |b|) 2^-20, and 2^-25 more for fp16: below its least normal number,
2^-14, its step is 2^-24 whatever |y| is (2.12e-6 lies between 35 and 36 steps and rounds by up to
2.98e-8, where u |y| is 1e-9)."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import decoding as ref

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUBNORMAL = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def np64(t):
    return t.detach().cpu().double().numpy()


def make(tokens, hq, hk, d, rot, dtype, axes, far, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(tokens, hq, d, generator=g).to(dtype).to(device)
    k = torch.randn(tokens, hk, d, generator=g).to(dtype).to(device)
    pos = torch.randint(min(far, 0), abs(far), (axes, tokens), generator=g, dtype=torch.int32)
    half = rot // 2
    f = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    sec = [half // axes] * axes
    sec[-1] += half - sum(sec)
    return q, k, pos.to(device), f.to(device), sec


def check(y, x, pos, f, sec, rot, inter, inverse):
    want = ref.rope(np64(x), pos.cpu().numpy(), f.cpu().numpy(), sec, rot, inter, inverse)
    a = np64(x)
    mate = np.array(a)
    half = rot // 2
    if inter:
        mate[..., 0:rot:2], mate[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
    else:
        mate[..., :half], mate[..., half:rot] = a[..., half:rot], a[..., :half]
    tol = UNIT[y.dtype] * np.abs(want) + (np.abs(a) + np.abs(mate)) * 2.0 ** -20 + SUBNORMAL[y.dtype]
    got = np64(y)
    assert np.array_equal(got[..., rot:], a[..., rot:])  # passed through, bit for bit
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


CASES = [
    # tokens, hq, hk, d, rot, axes, interleaved, far
    (1, 1, 1, 2, 2, 1, False, 100),
    (1, 32, 8, 128, 128, 1, False, 1000000),
    (7, 3, 1, 64, 64, 3, False, 4000),
    (33, 8, 2, 96, 64, 1, True, 131072),
    (65, 4, 4, 80, 48, 2, True, 4000),        # 16-byte chunks end inside an axis
    (19, 5, 2, 40, 40, 4, False, 4000),       # half of 20 pairs: no whole 16-byte chunk
    (13, 2, 1, 33, 10, 1, True, 4000),        # odd width, scalar path
    (9, 2, 2, 24, 0, 1, False, 4000),         # nothing turns
    (257, 16, 16, 128, 128, 3, False, 32768),
    (3000, 8, 8, 64, 32, 1, False, 2 ** 31 - 1),
    (50, 2, 2, 256, 256, 2, True, -70000),    # negative positions
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,axes,inter,far", CASES)
def test_rotation_matches_the_definition(tokens, hq, hk, d, rot, axes, inter, far, dtype):
    q, k, pos, f, sec = make(tokens, hq, hk, d, rot, dtype, axes, far, seed=tokens + d)
    for inverse in (False, True):
        yq, yk = vlf.vlf_rope(q, k, pos, f, sections=sec, interleaved=inter, inverse=inverse)
        check(yq, q, pos, f, sec, rot, inter, inverse)
        check(yk, k, pos, f, sec, rot, inter, inverse)


@pytest.mark.gpu
def test_packed_slices_one_axis_and_no_keys():
    """q and k as slices of a projection's output, outputs as slices of another buffer; k None."""
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(70, 12, 64, generator=g).to(torch.bfloat16).cuda()
    q, k = qkv[:, :8], qkv[:, 8:10]
    pos = torch.arange(70, dtype=torch.int32, device="cuda") * 1001
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device="cuda")
    buf = torch.zeros_like(qkv)
    vlf.vlf_rope(q, k, pos, f, q_out=buf[:, :8], k_out=buf[:, 8:10])
    yq, yk = vlf.vlf_rope(q.contiguous(), k.contiguous(), pos, f)
    assert torch.equal(buf[:, :8], yq) and torch.equal(buf[:, 8:10], yk)
    assert not buf[:, 10:].any()
    check(yq, q, pos[None], f, [32], 64, False, False)
    only, none = vlf.vlf_rope(q, None, pos, f)
    assert none is None and torch.equal(only, yq)
    # a token stride that is no multiple of 16 bytes takes the element path: the same values
    odd = torch.zeros(70, 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    view = odd[:, :512].view(70, 8, 64)
    view.copy_(q)
    assert torch.equal(vlf.vlf_rope(view, None, pos, f)[0], yq)


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [64, 32])
def test_in_place_and_back(rot):
    q, k, pos, f, sec = make(90, 4, 2, 64, rot, torch.float32, 2, 5000, seed=1)
    yq, yk = vlf.vlf_rope(q, k, pos, f, sec)
    a, b = q.clone(), k.clone()
    vlf.vlf_rope(a, b, pos, f, sec, q_out=a, k_out=b)
    assert torch.equal(a, yq) and torch.equal(b, yk)
    # turned back: the inverse of the rotation, each turn off by at most 2^-20 of its pair
    vlf.vlf_rope(a, b, pos, f, sec, inverse=True, q_out=a, k_out=b)
    assert (a - q).abs().max() <= 2.0 ** -17 * q.abs().max()


@pytest.mark.gpu
def test_gradients_match_formula_and_differences():
    q, k, pos, f, sec = make(21, 4, 2, 48, 32, torch.float32, 2, 300, seed=5)
    q.requires_grad_(), k.requires_grad_()
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    yq, yk = vlf.rotary_embedding(q, k, pos, f, sec, interleaved=True)
    ((yq * gq).sum() + (yk * gk).sum()).backward()
    check(q.grad, gq, pos, f, sec, 32, True, True)
    check(k.grad, gk, pos, f, sec, 32, True, True)
    # the map is linear: the difference along a direction is the gradient's product with it, with
    # errors of 2^-19 (|a| + |b|) |g| per element
    dq = torch.randn_like(q)
    with torch.no_grad():
        lhs = ((vlf.rotary_embedding(q + dq, k, pos, f, sec, True)[0].double() - yq.double()) * gq.double()).sum()
        rhs = (q.grad.double() * dq.double()).sum()
        bound = 2.0 ** -18 * (gq.abs().double() * (q.abs().max() + dq.abs().max()).double() * 4).sum()
    assert abs(lhs - rhs) <= bound


@pytest.mark.gpu
def test_gradients_of_gradients():
    """The gradient is a rotation back, so a second derivative through it is the rotation again."""
    q, k, pos, f, sec = make(9, 2, 1, 32, 32, torch.float32, 1, 300, seed=4)
    q.requires_grad_()
    g = torch.randn_like(q).requires_grad_()
    y, _ = vlf.rotary_embedding(q, k, pos, f)
    (dq,) = torch.autograd.grad((y * g).sum(), q, create_graph=True)
    v = torch.randn_like(q)
    (dg,) = torch.autograd.grad((dq * v).sum(), g)
    check(dg, v, pos, f, sec, 32, False, False)


@pytest.mark.gpu
def test_gradient_through_strided_slices_and_half_types():
    qkv = torch.randn(40, 6, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    f = torch.full((32,), 0.3, device="cuda")
    yq, yk = vlf.rotary_embedding(qkv[:, :4], qkv[:, 4:5], pos, f)
    (yq.float().sum() + 2 * yk.float().sum()).backward()
    ones = torch.ones(40, 5, 64, device="cuda", dtype=torch.bfloat16)
    ones[:, 4] = 2
    check(qkv.grad[:, :5], ones, pos[None], f, [32], 64, False, True)
    assert not qkv.grad[:, 5].any()


@pytest.mark.gpu
def test_captured_into_a_graph_and_on_another_stream():
    q, k, pos, f, sec = make(31, 4, 2, 64, 64, torch.float16, 1, 5000, seed=9)
    want = vlf.vlf_rope(q, k, pos, f)
    oq, ok = torch.zeros_like(q), torch.zeros_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vlf.vlf_rope(q, k, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vlf.vlf_rope(q, k, pos, f, q_out=oq, k_out=ok)
    q.mul_(2), pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    want = vlf.vlf_rope(q, k, pos, f)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])


def _raw(**kw):
    """The C entry point with made-up pointers: every call here is refused on the host."""
    a = dict(q=16, qs=256, k=16, ks=128, pos=16, axes=1, sec=None, f=16, total=4, hq=4, hk=2, d=64, rot=64,
             dtype=1, inter=0, inv=0, qo=32, qos=256, ko=32, kos=128)
    a.update(kw)
    import ctypes
    sec = None if a["sec"] is None else (ctypes.c_int * len(a["sec"]))(*a["sec"])
    return vlf._lib.vlf_rope(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["axes"], sec, a["f"], a["total"],
                             a["hq"], a["hk"], a["d"], a["rot"], a["dtype"], a["inter"], a["inv"], a["qo"],
                             a["qos"], a["ko"], a["kos"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=63), vlf.VLF_ERR_INVALID), (dict(rot=66), vlf.VLF_ERR_INVALID),
    (dict(rot=-2), vlf.VLF_ERR_INVALID), (dict(dtype=9), vlf.VLF_ERR_INVALID),
    (dict(axes=0), vlf.VLF_ERR_INVALID), (dict(axes=5, sec=[8] * 5), vlf.VLF_ERR_INVALID),
    (dict(axes=2), vlf.VLF_ERR_INVALID),                       # several axes without sections
    (dict(axes=2, sec=[16, 15]), vlf.VLF_ERR_INVALID),         # 31 of 32 pairs
    (dict(axes=2, sec=[33, -1]), vlf.VLF_ERR_INVALID),
    (dict(axes=3, sec=[2 ** 31 - 1, 2 ** 31 - 1, 34]), vlf.VLF_ERR_INVALID),
    (dict(d=320, rot=64), vlf.VLF_ERR_UNSUPPORTED), (dict(hq=0), vlf.VLF_ERR_INVALID),
    (dict(total=-1), vlf.VLF_ERR_INVALID), (dict(q=None), vlf.VLF_ERR_INVALID),
    (dict(ko=None), vlf.VLF_ERR_INVALID), (dict(pos=None), vlf.VLF_ERR_INVALID),
    (dict(qos=255), vlf.VLF_ERR_INVALID), (dict(qs=-1), vlf.VLF_ERR_INVALID),
    (dict(q=32, qs=512), vlf.VLF_ERR_INVALID),                 # in place with another stride
    (dict(qo=40), vlf.VLF_ERR_ALIGN), (dict(pos=20), vlf.VLF_ERR_ALIGN),
    (dict(total=0), vlf.VLF_OK),
])
def test_host_refusals(kw, status):
    assert _raw(**kw) == status


def test_python_refusals_without_a_gpu():
    q = torch.zeros(4, 2, 8)
    with pytest.raises(vlf.VlfError, match="CUDA"):
        vlf.vlf_rope(q, None, torch.zeros(4, dtype=torch.int32), torch.zeros(4))


@pytest.mark.gpu
def test_python_refusals():
    q, k, pos, f, sec = make(6, 4, 2, 64, 64, torch.float16, 2, 50, seed=2)
    bad = [dict(sections=None), dict(sections=[16, 16, 0]), dict(sections=[16, 15]),
           dict(sections=sec, q=q.transpose(0, 1)), dict(sections=sec, k=k.float()),
           dict(sections=sec, positions=pos.long()), dict(sections=sec, positions=pos[:, :5].contiguous()),
           dict(sections=sec, inv_freq=f.double()), dict(sections=sec, q=q[..., ::2]),
           dict(sections=sec, q_out=q[:3]), dict(sections=sec, k=k[:, :, :32].contiguous())]
    for kw in bad:
        a = dict(q=q, k=k, positions=pos, inv_freq=f)
        a.update(kw)
        with pytest.raises(vlf.VlfError):
            vlf.vlf_rope(**a)
    with pytest.raises(vlf.VlfError):
        vlf.rotary_embedding(q, k, pos, f.clone().requires_grad_(), sec)


@pytest.mark.gpu
def test_far_turns_of_small_and_negative_frequencies():
    """The turn itself: (1, 0) in fp32 becomes (cos t, sin t) without a rounding of products.  Errors of the
    angle: |position| (|inv_freq| 2^-55 + 2^-64) turns, pi (2^-25 + 2^-32) radians for the fraction in
    32 bits and in fp32; two ulp (2^-23) for a sine or cosine: together less than 2^-22 and the first."""
    f = np.float32([1.0, 0.5, -0.5, 2.74e-4, 2.46e-6, 1e-7, 1e-10, -1e-10, -3e-7, -2.46e-6, -1e-3, -0.7, 3.0, 0.0,
                    -4.4e-5, -6.1e-6])
    pos = np.int64([2 ** 31 - 1, -2 ** 31, 1999999999, -1234567891, 2 ** 20, 1, 0])
    x = torch.zeros(len(pos), 1, 2 * len(f), device="cuda")
    x[..., :len(f)] = 1
    y, _ = vlf.vlf_rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(f, device="cuda"))
    want = ref.rope(np64(x), pos[None], f, [len(f)], 2 * len(f), False)
    turns = np.abs(pos[:, None].astype(np.float64)) * (np.abs(f.astype(np.float64)) * 2.0 ** -55 + 2.0 ** -64)
    tol = 2.0 ** -22 + 2 * np.pi * np.concatenate([turns, turns], 1)[:, None]
    err = np.abs(np64(y) - want)
    assert (err <= tol).all(), (err - tol).max()
