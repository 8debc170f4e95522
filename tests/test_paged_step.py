"""Serving from pages as a program runs it: norm and rotary positions of a step's projection, the tables of the
next step, the copies they ask for, the new keys and values into their pages, attention over them, and the pool
compacted between steps; each stage against its definition on what the stage before produced.  Beams fork and
end, requests come and go, prompts and single tokens mix."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def np64(t):
    return t.detach().cpu().double().numpy()


def attention_holds(got, q, cache, rows, cu, lens, window=0):
    """out and lse within the bounds that test_pages_attention.py derives."""
    O, L, size, reach = ref.pages_attention(np64(q), cache, rows, cu, lens, q.shape[2] ** -0.5, True, window)
    tol = UNIT[q.dtype] * np.abs(O) + (2.0 ** -10 + 4 * (2.0 ** -16 * reach).T[..., None]) * size + 2.0 ** -24 * max(lens) * 32
    assert (np.abs(np64(got[0]) - O) <= tol).all()
    assert (np.abs(np64(got[1]) - L) <= 2.0 ** -16 * reach + 2.0 ** -18 * (1 + np.abs(L))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,hq,hkv,page,rot", [(torch.bfloat16, 128, 8, 2, 16, 128), (torch.float16, 64, 4, 4, 32, 32),
                                                    (torch.bfloat16, 96, 6, 2, 64, 96)])
def test_a_serving_loop(dtype, d, hq, hkv, page, rot):
    g = torch.Generator().manual_seed(d)
    most, pages, layers = 320 // page, 4000 // page, 2
    f = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().cuda()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    caches = [[torch.full((pages, hkv, page, d), 127, dtype=torch.uint8, device="cuda") for _ in range(2)] +
              [torch.full((pages, hkv), float("nan"), device="cuda") for _ in range(2)] for _ in range(layers)]
    table, lens, refs = torch.full((1, most), -1, dtype=I32, device="cuda"), ints([0]), ints([0] * pages)
    # (each step's rows: parents among the step's before, tokens that they get)
    steps = [([-1, -1, -1], [40, 3, 100]), ([0, 0, 1, 2], [1, 1, 1, 1]), ([1, 0, 3, 3, -1], [1, 1, 1, 1, 64]),
             ([0, 0, 0, 4], [1, 2, 5, 1]), ([2, 3, 1], [30, 1, 1])]
    for n, (parents, new) in enumerate(steps):
        rows0, lens0, refs0 = table.tolist(), lens.tolist(), refs.tolist()
        table, lens, refs, src, dst, left = vlf.vlf_pages_fork(table, lens, refs, ints(parents), ints(new), page)
        want = ref.fork([r[:-(-x // page)] for r, x in zip(rows0, lens0)], lens0, refs0, parents, new, page)
        assert [table.tolist(), lens.tolist(), refs.tolist(), src.tolist(), dst.tolist(), left.tolist()] == \
               [[r + [-1] * (most - len(r)) for r in want[0]], *want[1:5], [want[5]]]
        cu = [0] + [int(x) for x in np.cumsum(new)]
        now = lens.tolist()
        pos = ints([now[s] - new[s] + i for s in range(len(new)) for i in range(new[s])])
        for cache in caches:
            qkv = torch.randn(cu[-1], hq + 2 * hkv, d, generator=g).to(dtype).cuda()
            q, k = vlf.vlf_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], wq, wk, pos, f)
            for y, x, w in ((q, qkv[:, :hq], wq), (k, qkv[:, hq:hq + hkv], wk)):
                a = np64(x)
                should = ref.norm_rope(a, np64(w), 1e-6, pos.cpu().numpy()[None], f.cpu().numpy(), [rot // 2], rot, False)
                assert (np.abs(np64(y) - should) <= UNIT[dtype] * np.abs(should) + 2.0 ** -17 * np.abs(a).max() * 2).all()
            before = [x.cpu().numpy() for x in cache]
            vlf.vlf_pages_copy(*cache, src, dst)
            for x in before:
                for a, b in zip(src.tolist(), dst.tolist()):
                    if a >= 0:
                        x[b] = x[a]
            v = qkv[:, hq + hkv:]
            vlf.vlf_pages_write(k, v, *cache, table, ints(cu), lens)
            before = ref.pages_write(np64(k), np64(v), before, table.tolist(), cu, now)
            assert all(np.array_equal(x.cpu().numpy(), y, equal_nan=True) for x, y in zip(cache, before))
            got = vlf.vlf_attn_varlen_fwd_pages(q, *cache, table, ints(cu), lens, max(new), causal=True)
            attention_holds(got, q, before, table.tolist(), cu, now)
        if n % 2:  # between steps the pool is compacted, for every layer alike
            kept = [[x[r[:-(-y // page)]].clone() for r, y in zip(table.tolist(), now)] for c in caches for x in c]
            table, refs, to, src, dst, used = vlf.vlf_pages_compact(table, refs)
            for cache in caches:
                vlf.vlf_pages_copy(*cache, src, dst)
            after = [[x[r[:-(-y // page)]] for r, y in zip(table.tolist(), now)] for c in caches for x in c]
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for x, y in zip(kept, after) for a, b in zip(x, y))
            held = [p for r, y in zip(table.tolist(), now) for p in r[:-(-y // page)]]
            assert int(used) == len(set(held)) and max(held) < int(used) and refs.tolist() == [held.count(p) for p in range(pages)]
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_a_captured_decode_step():
    """A whole step in one graph, replayed token after token: lengths and tables move on the device."""
    g = torch.Generator().manual_seed(1)
    d, hq, hkv, page, most, pages, n = 128, 8, 2, 16, 16, 64, 3
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    cache = [torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.ones(pages, hkv, device="cuda") for _ in range(2)]
    table, lens, refs = torch.full((n, most), -1, dtype=I32, device="cuda"), ints([0] * n), ints([0] * pages)
    go_on, one, cu = ints(list(range(n))), ints([1] * n), ints(list(range(n + 1)))
    qkv = torch.zeros(n, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")

    def step():
        t, l, r, src, dst, left = vlf.vlf_pages_fork(table, lens, refs, go_on, one, page)
        vlf.vlf_pages_copy(*cache, src, dst)
        table.copy_(t), lens.copy_(l), refs.copy_(r)
        q, k = vlf.vlf_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], w, w, l - 1, f)
        vlf.vlf_pages_write(k, qkv[:, hq + hkv:], *cache, t, cu, l)
        return (*vlf.vlf_attn_varlen_fwd_pages(q, *cache, t, cu, l, 1, causal=True), q)

    saved = [x.clone() for x in (table, lens, refs, *cache)]
    step()  # (warm-up: memory and kernels; what it changed is put back)
    for x, y in zip((table, lens, refs, *cache), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, q = step()
    for i in range(40):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        if i % 13 == 0 or i == 39:
            assert lens.tolist() == [i + 1] * n
            attention_holds((out, lse), q, [x.cpu().numpy() for x in cache], table.tolist(), list(range(n + 1)), lens.tolist())
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_norm_in_front_of_attention_in_training():
    """Gradients through norm, rotary positions and attention together, against differences of the loss in fp32."""
    g = torch.Generator().manual_seed(2)
    t, hq, hkv, d = 37, 4, 2, 64
    qkv = torch.randn(t, hq + 2 * hkv, d, generator=g).cuda().requires_grad_()
    wq, wk = (torch.ones(d, device="cuda", requires_grad=True) for _ in range(2))
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    pos, cu = torch.arange(t, dtype=I32, device="cuda"), ints([0, 20, t])
    go = torch.randn(t, hq, d, generator=g).cuda()

    def loss(qkv, wq, wk):
        q, k = vlf.norm_rotary_embedding(qkv[:, :hq], qkv[:, hq:hq + hkv], wq, wk, pos, f)
        return (vlf.varlen_attention(q, k, qkv[:, hq + hkv:], cu, cu, 20, 20, causal=True).double() * go.double()).sum()

    loss(qkv, wq, wk).backward()
    with torch.no_grad():
        for x in (qkv, wq, wk):
            e, h = torch.randn(x.shape, generator=g).cuda(), 2.0 ** -7
            args = [(y + h * e, y - h * e) if y is x else (y, y) for y in (qkv, wq, wk)]
            num = (loss(*[a for a, _ in args]) - loss(*[b for _, b in args])) / (2 * h)
            # second differences of a loss of |go| summed over 37 x 4 x 64 entries, with terms of size one: h^2 of
            # it; fp32 forwards are off by 2^-18 of it, over h
            size = go.abs().double().sum()
            assert abs(num - (x.grad.double() * e.double()).sum()) <= size * (h * h + 2.0 ** -18 / h)
