"""Attention over pages in e4m3 (vlf_attn_varlen_fwd_pages) against the fp64 definition on the values that the
bytes stand for: both kernel families, page sizes, head groups, ragged lengths with empty ones, windows, rows
that see nothing, what stands behind the last key, tables with holes in front of a window.

Tolerance.  A logit is a sum of products that are exact, added in fp32, and q is held to 2^-18 of its row's
largest element: it is off by at most d = 2^-16 of the largest sum_c |q_c k_c| scale of the row.  A weight is
rounded to 2^-11 (the sum of three e5m2 numbers) and off by 2^-20 from exp2, the sum by as much: with u for
the output, |error| <= u |out| + (2^-10 + 4 d) sum_j p_j |v_j|, and what falls below the least e5m2 number,
2^-24 of the largest weight for each key.  The lse is off by d and 2^-18 of itself."""
import random

import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SIMT = vlf.VLF_FLAG_FORCE_SIMT
BF, FP = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().cpu().double().numpy()


def problem(q_lens, kv_lens, page, hq, hkv, dk, dv, dtype, seed=0, size=1.0, extra=3, scales=True):
    """A pool whose unused bytes (other pages, slots behind a sequence's end) are NaN, in shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    pages = sum(-(-x // page) for x in kv_lens) + extra
    order = list(range(pages))
    r.shuffle(order)
    most = max([1] + [-(-x // page) for x in kv_lens])
    rows = []
    c = dict(q=(size * torch.randn(sum(q_lens), hq, dk, generator=g)).to(dtype).cuda())
    for name, d in (("k", dk), ("v", dv)):
        x = torch.randn(pages, hkv, page, d, generator=g).clamp(-4, 4)
        c[name + "_pages"] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.randint(-8, -3, (pages, hkv), generator=g) if scales else torch.full((pages, hkv), -6)
        c[name + "_scale"] = torch.exp2(e.float()).cuda()
    at = 0
    free = set(range(pages))
    for x in kv_lens:
        n = -(-x // page)
        rows.append(order[at:at + n] + [-1] * (most - n))
        at += n
        free -= set(rows[-1])
        if x % page:
            for name in ("k_pages", "v_pages"):
                c[name][rows[-1][n - 1], :, x % page:] = 127 if x % 2 else 255
    for p in free:
        c["k_pages"][p] = c["v_pages"][p] = 127
        c["k_scale"][p] = c["v_scale"][p] = float("nan")
    c["k_pages"], c["v_pages"] = c["k_pages"].cuda(), c["v_pages"].cuda()
    c["rows"], c["table"] = rows, ints(rows).view(len(rows), most)
    c["cu"] = [0] + [int(x) for x in np.cumsum(q_lens)]
    c["cu_q"], c["kv"], c["lens"] = ints(c["cu"]), ints(kv_lens), kv_lens
    c["max_q"] = max([0] + q_lens)
    return c


def call(c, **kw):
    return vlf.vlf_attn_varlen_fwd_pages(c["q"], c["k_pages"], c["v_pages"], c["k_scale"], c["v_scale"], c["table"], c["cu_q"],
                                         c["kv"], kw.pop("max_q", c["max_q"]), **kw)


def check(got, c, scale=None, causal=False, window=0):
    scale = scale or c["q"].shape[2] ** -0.5
    cache = [c[x].cpu().numpy() for x in ("k_pages", "v_pages", "k_scale", "v_scale")]
    O, L, size, reach = ref.pages_attention(np64(c["q"]), cache, c["rows"], c["cu"], c["lens"], scale, causal, window)
    out, lse = got
    off = (2.0 ** -16 * reach).T[..., None]
    few = 2.0 ** -24 * max(c["lens"] + [0]) * 4 * 2.0 ** 3
    tol = UNIT[out.dtype] * np.abs(O) + (2.0 ** -10 + 4 * off) * size + few + 1e-30
    assert (np.abs(np64(out) - O) <= tol).all(), np.nanmax(np.abs(np64(out) - O) / tol)
    live = L > -np.inf
    assert np.array_equal(np64(lse) > -np.inf, live)
    assert (np.abs(np64(lse) - L)[live] <= (2.0 ** -16 * reach + 2.0 ** -18 * (1 + np.abs(np.where(live, L, 0))))[live]).all()
    assert not np64(out)[~live.T].any()
    assert vlf.vlf_check_error() == 0


CASES = [
    # q_lens, kv_lens, page, hq, hkv, d, causal, window
    ([1], [1], 16, 1, 1, 128, True, 0),
    ([1, 1, 1], [17, 160, 1000], 16, 8, 8, 64, True, 0),
    ([1, 1, 1, 1], [129, 128, 127, 300], 64, 8, 2, 128, True, 0),
    ([1, 0, 1], [200, 50, 0], 32, 4, 1, 128, True, 0),      # no query, no key
    ([4, 1, 2], [33, 900, 2], 128, 6, 2, 64, True, 0),      # drafted tokens
    ([5, 3], [3, 700], 64, 4, 2, 128, True, 0),             # rows in front of the first key
    ([70, 33], [70, 400], 256, 4, 4, 128, True, 0),         # a whole prompt
    ([40, 1, 130], [513, 64, 700], 64, 8, 1, 64, True, 0),  # one kv head
    ([40, 7], [300, 511], 16, 8, 2, 128, True, 100),        # window
    ([1, 1], [1000, 40], 64, 16, 2, 64, True, 64),
    ([3, 9], [500, 20], 32, 4, 2, 128, False, 0),           # no causal rule
    ([9, 20], [300, 10], 128, 4, 2, 64, False, 30),         # a window's lower edge alone
    ([200], [2000], 128, 32, 8, 128, True, 0),
    ([1] * 20, [37 * i + 1 for i in range(20)], 32, 12, 4, 128, True, 0),
    ([2, 1], [40, 70], 16, 16, 1, 64, True, 0),
    ([1, 17], [130, 260], 64, 33, 1, 128, True, 0),         # more heads of a group than a tile's columns divide
    ([1], [5000], 64, 64, 1, 128, True, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("q_lens,kv_lens,page,hq,hkv,d,causal,window", CASES)
def test_matches_the_definition(q_lens, kv_lens, page, hq, hkv, d, causal, window, dtype, flags):
    c = problem(q_lens, kv_lens, page, hq, hkv, d, d, dtype, seed=len(q_lens) + page)
    got = call(c, causal=causal, window=window, flags=flags)
    check(got, c, causal=causal, window=window)
    again = call(c, causal=causal, window=window, flags=flags)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])  # the same bits
    # (a loose bound is any bound; it may cut the work otherwise)
    check(call(c, causal=causal, window=window, flags=flags, max_q=c["max_q"] + 5000), c, causal=causal, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv,dtype", [(32, 32, BF), (96, 96, FP), (192, 128, BF), (256, 256, FP), (33, 7, BF), (64, 64, torch.float32),
                                         (128, 128, torch.float32), (128, 64, BF), (1, 1, FP)])
def test_other_widths_and_fp32(dk, dv, dtype):
    c = problem([3, 1, 40], [100, 515, 60], 32, 4, 2, dk, dv, dtype, seed=dk)
    check(call(c, causal=True), c, causal=True)
    check(call(c, causal=True, window=33, scale=0.3), c, scale=0.3, causal=True, window=33)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
@pytest.mark.parametrize("seed", range(6))
def test_drawn_problems(seed, d, dtype):
    r = random.Random(seed)
    n = r.randint(1, 9)
    kv = [r.choice([0, r.randint(1, 40), r.randint(1, 3000)]) for _ in range(n)]
    q = [r.choice([0, 1, 1, r.randint(1, 90)]) for _ in range(n)]
    hkv = r.choice([1, 2, 3, 8])
    c = problem(q, kv, r.choice([16, 32, 64, 128, 256]), hkv * r.choice([1, 2, 3, 4, 8]), hkv, d, d, dtype, seed=seed)
    causal, window = r.random() < 0.7, r.choice([0, 0, 1, 50, 1000])
    check(call(c, causal=causal, window=window), c, causal=causal, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
def test_one_key_outweighs_a_long_tail(d, dtype):
    """A first key that takes half of the weight, and thousands with 2^-13 and less of its weight each: the tail's weights
    are far below the largest one, and its values all the same."""
    n = 6000
    c = problem([1, 2], [n, n], 64, 4, 1, d, d, dtype, scales=False)
    k, v = c["k_pages"].view(torch.float8_e4m3fn).float(), c["v_pages"].view(torch.float8_e4m3fn).float()
    k[:], v[:] = 0, 64  # (value 1 at the scale 2^-6)
    for row, kl in zip(c["rows"], c["lens"]):
        k[row[0], :, 0] = 64
        v[row[0], :, 0] = -32
    for name, x in (("k_pages", k), ("v_pages", v)):
        c[name] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    c["q"].fill_(1.0)
    for lift in (8.7, 11.0, 14.0):  # the first key's logit: e^8.7 is 6000
        check(call(c, scale=lift / d, causal=True), c, scale=lift / d, causal=True)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
def test_scales_of_pages_far_apart(d, dtype):
    """A page of huge values that gets no weight costs the others nothing, nor do pages of tiny values."""
    c = problem([1, 40], [700, 500], 64, 4, 2, d, d, dtype, seed=4, scales=False)
    for row in c["rows"]:
        c["v_scale"][row[2]] = 2.0 ** 40
        c["v_scale"][row[3]] = 2.0 ** -60
        c["k_pages"][row[2]] = 0
        c["k_scale"][row[4]] = 2.0 ** -20
    c["q"].abs_()
    first = c["k_pages"].view(torch.float8_e4m3fn).float()
    for row in c["rows"]:
        first[row[0]] = first[row[0]].abs() * 4 + 100  # (logits of 200 and more: the page of zeros gets e^-200)
    c["k_pages"] = first.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for row, n in zip(c["rows"], c["lens"]):
        if n % 64:
            c["k_pages"][row[-(-n // 64) - 1], :, n % 64:] = 127
    got = call(c)
    check(got, c)


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, SIMT])
def test_nan_reaches_the_rows_that_see_it(flags):
    c = problem([1, 3], [300, 200], 64, 4, 2, 128, 128, BF, seed=2)
    want = call(c, causal=True, flags=flags)
    k = c["k_pages"].clone()
    c["k_pages"][c["rows"][1][1], 0, 5, 3] = 127  # key 69 of the second sequence, heads 0 and 1
    out, lse = call(c, causal=True, flags=flags)
    assert out[1:, :2].isnan().all() and lse[:2, 1:].isnan().all()
    assert torch.equal(out[:1], want[0][:1]) and torch.equal(out[:, 2:], want[0][:, 2:]) and torch.equal(lse[2:], want[1][2:])
    c["k_pages"] = k
    c["v_pages"][c["rows"][1][1], 1, 5, 3] = 255
    out, lse = call(c, causal=True, flags=flags)
    assert out[1:, 2:, 3].isnan().all() and torch.equal(lse, want[1]) and torch.equal(out[:, :2], want[0][:, :2])
    q = c["q"].clone()
    c["q"][0, 3, 7] = float("nan")
    assert call(c, flags=flags)[0][0, 3].isnan().all() and not call(c, flags=flags)[0][0, :3].isnan().any()
    c["q"] = q
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, SIMT])
def test_pages_in_front_of_a_window_may_be_gone(flags):
    c = problem([1, 20], [1000, 900], 64, 4, 2, 64, 64, BF, seed=6)
    want = call(c, causal=True, window=100, flags=flags)
    check(want, c, causal=True, window=100)
    c["table"][0, :(1000 - 100) // 64] = -1
    c["table"][1, :(900 - 20 - 99) // 64] = 2 ** 31 - 1
    got = call(c, causal=True, window=100, flags=flags)
    assert vlf.vlf_check_error() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("change,status", [(dict(page=99), -8), (dict(page=-1), -8), (dict(length=2000), -6), (dict(length=-1), -6),
                                           (dict(cu=[0, 9, 4]), -6), (dict(cu=[0, 1, 5]), -6)])
def test_bad_tables_and_lengths_are_recorded(change, status, flags):
    c = problem([1, 3], [300, 200], 64, 4, 2, 128, 128, BF, seed=2)
    want = call(c, causal=True, flags=flags)
    if "page" in change:
        c["table"][1, 2] = change["page"]
    if "length" in change:
        c["kv"][1] = change["length"]
    if "cu" in change:
        c["cu_q"] = ints(change["cu"])
    out, _ = call(c, causal=True, flags=flags)
    assert vlf.vlf_check_error() == status
    if "cu" not in change:
        assert torch.equal(out[0], want[0][0])  # the other sequence is what it was
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", [([1] * 5, [700, 20, 1300, 90, 333], 8, 2), ([60, 9], [900, 400], 8, 2)])
def test_streams_graphs_and_given_buffers(q_lens, kv_lens, hq, hkv):
    c = problem(q_lens, kv_lens, 64, hq, hkv, 128, 128, BF, seed=12)
    want = [x.clone() for x in call(c, causal=True)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(c, causal=True, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    need = vlf.vlf_attn_varlen_fwd_pages_workspace_size(len(q_lens), sum(q_lens), c["max_q"], hq, hkv, 128, 128, BF)
    given = dict(out=torch.full_like(want[0], 7), lse=torch.full_like(want[1], 7),
                 workspace=torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda"))
    got = call(c, causal=True, **given)
    assert got[0] is given["out"] and all(torch.equal(a, b) for a, b in zip(got, want))
    assert given["workspace"][need:].eq(255).all()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        a = call(c, causal=True)
    with torch.cuda.graph(two):
        b = call(c, causal=True)
    c["q"].mul_(-1)
    c["kv"].sub_(3)  # (a graph takes what the lengths are when it runs)
    c["lens"] = [x - 3 for x in c["lens"]]
    want = [x.clone() for x in call(c, causal=True)]
    check(want, c, causal=True)
    for _ in range(3):
        one.replay()
        with torch.cuda.stream(side):
            two.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([*a, *b], [*want, *want]))


@pytest.mark.gpu
def test_no_queries_and_no_sequences():
    c = problem([0, 0], [30, 0], 16, 4, 2, 64, 64, BF)
    out, lse = call(c, causal=True)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    c = problem([2], [0], 16, 4, 2, 64, 64, BF)
    out, lse = call(c)
    assert not out.any() and lse.eq(-float("inf")).all()
    assert vlf.vlf_check_error() == 0


def raw(**kw):
    a = dict(q=16, kp=16, vp=16, ks=16, vs=16, t=16, cu=16, lens=16, n=2, tq=5, mq=4, most=8, pages=9, page=16, hq=4, hkv=2, dk=64,
             dv=64, dtype=1, scale=0.0, causal=1, window=0, out=16, lse=16, ws=None, wsn=0)
    a.update(kw)
    return vlf._lib.vlf_attn_varlen_fwd_pages(*a.values(), None, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(tq=-1), -1), (dict(mq=-1), -1), (dict(most=-1), -1), (dict(pages=-1), -1), (dict(hq=3), -1), (dict(hkv=0), -1),
    (dict(dk=0), -1), (dict(dtype=5), -1), (dict(q=None), -1), (dict(kp=None), -1), (dict(vs=None), -1), (dict(t=None), -1),
    (dict(cu=None), -1), (dict(lens=None), -1), (dict(out=None), -1), (dict(n=0), -1), (dict(page=48), -2), (dict(dv=257), -2),
    (dict(most=2 ** 27), -2), (dict(tq=2 ** 31 - 2), -2), (dict(n=70000), -2), (dict(q=8), -3), (dict(t=8), -3), (dict(out=8), -3),
    (dict(lse=4), -3), (dict(n=0, tq=0), 0), (dict(tq=0), 0)])
def test_refusals_before_any_launch(kw, status):
    assert raw(**kw) == status


@pytest.mark.gpu
def test_refusals_with_tensors():
    c = problem([1, 3], [30, 20], 16, 4, 2, 64, 64, BF)
    a = [c[x] for x in ("q", "k_pages", "v_pages", "k_scale", "v_scale", "table", "cu_q", "kv")]
    swap = lambda i, t: vlf.vlf_attn_varlen_fwd_pages(*a[:i], t, *a[i + 1:], 3)  # noqa: E731
    for i, t in [(0, a[0].double()), (0, a[0][..., :32].contiguous()), (0, a[0].transpose(0, 1)), (0, a[0].cpu()), (1, a[1].half()),
                 (1, a[1][:2]), (2, a[2][:, :1].contiguous()), (3, a[3].half()), (4, a[4][:2]), (5, a[5].long()), (5, a[5][:1]),
                 (6, a[6][:2]), (7, a[7][:1]), (7, a[7].cpu())]:
        with pytest.raises(vlf.VlfError):
            swap(i, t)
    with pytest.raises(vlf.VlfError):
        vlf.vlf_attn_varlen_fwd_pages(*a, 3, out=a[0][:1])
    need = vlf.vlf_attn_varlen_fwd_pages_workspace_size(2, 4, 3, 4, 2, 64, 64, BF)
    if need:
        with pytest.raises(vlf.VlfError):
            vlf.vlf_attn_varlen_fwd_pages(*a, 3, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("q_len,d,dtype,window", [(1, 128, BF, 0), (2, 64, FP, 7000), (20, 128, FP, 0)])
def test_long_caches_in_pages_of_every_size(page, q_len, d, dtype, window):
    """More pages than are looked up at a time, and ends inside pages and tiles."""
    c = problem([q_len, q_len], [20011, 9001], page, 4, 2, d, d, dtype, seed=page)
    check(call(c, causal=True, window=window), c, causal=True, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, SIMT])
def test_many_sequences_with_and_without_rows(flags):
    """More sequences than a block has threads; most have no rows, or no keys."""
    n = 1500
    q = [1 if s % 7 == 0 else 0 for s in range(n)]
    kv = [0 if s % 11 == 0 else s % 90 for s in range(n)]
    kv[700], q[700] = 3000, 1
    c = problem(q, kv, 16, 4, 2, 64, 64, BF, seed=3)
    check(call(c, causal=True, flags=flags), c, causal=True)
    q[350] = 40
    c = problem(q, kv, 16, 4, 2, 64, 64, BF, seed=3)
    check(call(c, causal=True, flags=flags), c, causal=True)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,rows", [(3, 1, 30), (5, 1, 60), (7, 1, 9), (130, 1, 2), (300, 1, 3), (20, 1, 7)])
def test_groups_that_do_not_divide_a_tile(hq, hkv, rows):
    c = problem([rows, 1], [rows + 100, 333], 32, hq, hkv, 64, 64, FP, seed=hq)
    check(call(c, causal=True), c, causal=True)


@pytest.mark.gpu
def test_queries_of_every_size():
    """Rows of zeros, of fp16's largest numbers, of bf16's smallest and largest: the powers of two that they are held over."""
    for dtype, sizes in ((FP, (0.0, 6e-8, 1.0, 6e4)), (BF, (0.0, 1e-38, 1e-20, 1e4))):
        for rows in (1, 40):
            c = problem([rows] * 4, [200, 90, 64, 300], 64, 4, 2, 128, 128, dtype, seed=5)
            scale = 2.0 ** -10
            for s, size in enumerate(sizes):
                x = c["q"][c["cu"][s]:c["cu"][s + 1]]
                x.copy_((x.float().clamp(-1, 1) * size).to(dtype))
            c["k_scale"].clamp_(max=2.0 ** -7)
            check(call(c, scale=scale), c, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [999, 40]), ([1, 1], [3, 5000]), ([300, 1, 400], [700, 31, 400])])
@pytest.mark.parametrize("hq,hkv,dk,dv", [(4, 4, 40, 40), (2, 1, 100, 100), (3, 1, 96, 96), (10, 2, 250, 129), (9, 3, 64, 6), (5, 1, 17, 256)])
def test_heads_and_rows_of_the_fma_kernel(q_lens, kv_lens, hq, hkv, dk, dv):
    """Groups that its blocks of four heads do not divide; a row's keys in one block, and shared out to eight."""
    c = problem(q_lens, kv_lens, 32, hq, hkv, dk, dv, BF, seed=dk)
    check(call(c, causal=True), c, causal=True)
    check(call(c, causal=True, window=37), c, causal=True, window=37)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,flags", [([1, 3], 0), ([60, 30], 0), ([1, 3], SIMT)])
def test_pages_past_32_bits(q_lens, flags):
    """The same pages at the end of a pool of more than 4 GB: the same bits."""
    c = problem(q_lens, [700, 130], 64, 8, 2, 128, 128, BF, seed=9)
    want = call(c, causal=True, flags=flags)
    n = c["k_pages"].shape[0]
    first = (1 << 32) // c["k_pages"][0].numel() + 3
    far = dict(c, table=torch.where(c["table"] >= 0, c["table"] + first, c["table"]))
    for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
        far[x] = torch.empty(first + n, *c[x].shape[1:], dtype=c[x].dtype, device="cuda")
        far[x][first:] = c[x]
    got = call(far, causal=True, flags=flags)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert vlf.vlf_check_error() == 0
