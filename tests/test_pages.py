"""Pages of a cache: tokens rounded into them (vlf_pages_write), pages copied (vlf_pages_copy), tables forked
and compacted (vlf_pages_fork, vlf_pages_compact), against plain definitions.  Everything here is exact: a
rounding to e4m3 is one definite byte, scales are powers of two, tables are whole numbers."""
import random

import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref

I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def some_cache(pages, h, page, dk, dv, seed, scale=2.0 ** -7):
    """Bytes of every value, NaN among them, and scales."""
    g = torch.Generator().manual_seed(seed)
    c = [torch.randint(0, 256, (pages, h, page, d), generator=g, dtype=torch.uint8).cuda() for d in (dk, dv)]
    return c + [torch.full((pages, h), scale, device="cuda") for _ in range(2)]


def some_table(lens, page, pages, seed, most=None):
    r = random.Random(seed)
    order = list(range(pages))
    r.shuffle(order)
    most = most or max(1, max(-(-x // page) for x in lens))
    rows = []
    for x in lens:
        n = -(-x // page)
        rows.append(order[:n] + [-1] * (most - n))
        order = order[n:]
    return rows


def same(got, want):
    for a, b in zip(got, want):
        assert np.array_equal(a.view(torch.uint8).cpu().numpy() if a.dtype != torch.float32 else a.cpu().numpy(), b)


def check_write(k, v, cache, rows, new, lens):
    want = ref.pages_write(k.cpu().double().numpy(), v.cpu().double().numpy(), [x.cpu().numpy() for x in cache], rows,
                           cu_of(new), lens)
    vlf.vlf_pages_write(k, v, *cache, ints(rows), ints(cu_of(new)), ints(lens))
    assert vlf.vlf_check_error() == 0
    same(cache, want)


CASES = [
    # new tokens, lengths with them, page, h_kv, d_qk, d_v
    ([1], [1], 16, 1, 64, 64),
    ([1, 1, 1], [17, 16, 500], 16, 2, 128, 128),
    ([5, 0, 40, 33], [5, 20, 71, 64], 32, 3, 64, 128),
    ([64, 65, 200], [64, 65, 256], 64, 2, 96, 64),
    ([300, 1, 0], [300, 129, 0], 128, 2, 192, 128),
    ([257, 12], [1000, 12], 256, 1, 256, 256),
    ([20, 3], [33, 3], 16, 2, 33, 7),          # odd widths, the element path
    ([2] * 40, [2 + 3 * i for i in range(40)], 16, 2, 40, 40),
    ([0, 0], [5, 0], 16, 1, 64, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("new,lens,page,h,dk,dv", CASES)
def test_write_matches_the_definition(new, lens, page, h, dk, dv, dtype):
    g = torch.Generator().manual_seed(sum(new) + dk)
    # (sizes over many powers of two, so that scales of pages differ and many bytes are subnormal)
    r = lambda d: (torch.randn(sum(new), h, d, generator=g) * torch.exp2(torch.randint(-6, 7, (sum(new), h, 1), generator=g))).to(dtype).cuda()  # noqa: E731
    pages = sum(-(-x // page) for x in lens) + 3
    check_write(r(dk), r(dv), some_cache(pages, h, page, dk, dv, 7), some_table(lens, page, pages, 3), new, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_page_filled_token_by_token(dtype):
    """The scale grows with the values and the bytes there follow; a page that is begun anew starts from its own values."""
    g = torch.Generator().manual_seed(0)
    cache = some_cache(5, 2, 16, 64, 64, 1, scale=2.0 ** 20)
    rows = [[3, 1, 4]]
    for i in range(40):
        size = 2.0 ** (i % 13 - 6 if i < 20 else -3)
        k, v = ((size * torch.randn(1, 2, 64, generator=g)).to(dtype).cuda() for _ in range(2))
        check_write(k, v, cache, rows, [1], [i + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
def test_values_at_the_borders(few):
    """448 and its neighbours, ties, zeros, the least scale, values that are not finite."""
    t = torch.zeros(16 if few else 200, 1, 64)
    t[0, 0, :6] = torch.tensor([448.0, -448.0, 449.0, 1.0625, 1.1875, 2.0 ** -10])
    t[1, 0, :5] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.0, -0.0])
    t[2, 0, 0] = 3e38
    t[3, 0, 0] = 1e-44
    t[4, 0, :2] = torch.tensor([2.0 ** -60, 448 * 2.0 ** -64])
    t[5, 0, :] = float("nan")
    if few:  # a sequence for each token
        new, lens, rows = [1] * 16, [1] * 16, [[i] for i in range(16)]
    else:
        new, lens, rows = [200], [200], [list(range(13))]
    check_write(t.cuda(), (-t).cuda(), some_cache(16, 1, 16, 64, 64, 2), rows, new, lens)


@pytest.mark.gpu
def test_write_takes_slices_and_leaves_the_rest():
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(70, 12, 64, generator=g).to(torch.bfloat16).cuda()
    new, lens, page = [1, 40, 29], [30, 40, 64], 32
    rows = some_table(lens, page, 20, 5, most=6)
    a, b = some_cache(20, 2, page, 64, 64, 4), some_cache(20, 2, page, 64, 64, 4)
    untouched = [p for p in range(20) if p not in {rows[0][0], *rows[1][:2], *rows[2][1:2]}]
    check_write(qkv[:, 8:10], qkv[:, 10:], a, rows, new, lens)
    for i, x in enumerate(a):
        assert torch.equal(x[untouched], b[i][untouched])
    # e4m3 tensors, arguments that are slices, another stream
    e = [x.view(torch.float8_e4m3fn) for x in b[:2]] + b[2:]
    shift = lambda x: torch.cat([ints([0]), ints(x).flatten()])[1:]  # noqa: E731
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    vlf.vlf_pages_write(qkv[:, 8:10], qkv[:, 10:], *e, shift(rows).view(3, 6), shift(cu_of(new)), shift(lens), stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    odd = torch.zeros(70, 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, :128].view(70, 2, 64)  # the element path
    odd.copy_(qkv[:, 8:10])
    c = some_cache(20, 2, page, 64, 64, 4)
    vlf.vlf_pages_write(odd, odd, *c, ints(rows), ints(cu_of(new)), ints(lens))
    assert torch.equal(c[0], a[0]) and torch.equal(c[2], a[2])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,new,lens,status", [
    ([[0, 1], [9, 2]], [1, 1], [17, 1], -8), ([[0, -1], [3, 2]], [1, 1], [17, 1], -8),
    ([[0, 1], [3, 2]], [1, 1], [33, 1], -6), ([[0, 1], [3, 2]], [2, 1], [1, 1], -6), ([[0, 1], [3, 2]], [1, 1], [-5, 1], -6)])
def test_bad_tables_are_recorded_and_passed_over(rows, new, lens, status):
    cache = some_cache(9, 1, 16, 64, 64, 1)
    before = [x.clone() for x in cache]
    k = torch.ones(sum(new), 1, 64, device="cuda")
    vlf.vlf_pages_write(k, k, *cache, ints(rows), ints(cu_of(new)), ints(lens))
    assert vlf.vlf_check_error() == status
    assert vlf.vlf_check_error() == 0
    good = 2 if rows[1][0] == 9 else 3
    for x, y in zip(cache, before):
        rest = [p for p in range(9) if p not in (1, good)]
        assert torch.equal(x[rest], y[rest])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of over 2^32 bytes a tensor, its first and last pages written, copied and read."""
    h, page, d = 8, 128, 256
    pages = (1 << 32) // (h * page * d) + 5
    k, v = (torch.zeros(pages, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(pages, h, device="cuda") for _ in range(2))
    x = torch.randn(130, h, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    vlf.vlf_pages_write(x, x, k, v, ks, vs, ints([[pages - 1, 0]]), ints([0, 130]), ints([130]))
    vlf.vlf_pages_copy(k, v, ks, vs, ints([pages - 1, -1]), ints([pages - 3, -1]))
    small = [torch.zeros(2, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.ones(2, h, device="cuda") for _ in range(2)]
    vlf.vlf_pages_write(x, x, *small, ints([[1, 0]]), ints([0, 130]), ints([130]))
    for a, b in zip((k, v, ks, vs), small):
        assert torch.equal(a[pages - 1], b[1]) and torch.equal(a[0], b[0]) and torch.equal(a[pages - 3], b[1])
    assert not k[1:pages - 3].any() and not k[pages - 2].any()
    q = x[:3].repeat(1, 2, 1)
    want = vlf.vlf_attn_varlen_fwd_pages(q, *small, ints([[1, 0]]), ints([0, 3]), ints([130]), 3)
    got = vlf.vlf_attn_varlen_fwd_pages(q, k, v, ks, vs, ints([[pages - 3, 0]]), ints([0, 3]), ints([130]), 3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert vlf.vlf_check_error() == 0


# ------------------------------------------------------------------------------ copies
@pytest.mark.gpu
@pytest.mark.parametrize("n,h,page,dk,dv", [(1, 1, 16, 1, 3), (7, 2, 16, 64, 64), (300, 3, 32, 33, 64), (40, 8, 128, 128, 128)])
def test_copies(n, h, page, dk, dv):
    pages = 3 * n + 2
    r = random.Random(n)
    order = list(range(pages))
    r.shuffle(order)
    src, dst = order[:n], order[n:2 * n]
    for i in range(0, n, 3):
        if n > 1:
            src[i] = -1
    src += src[:1]  # a page that goes to two places
    dst += order[2 * n:2 * n + 1]
    cache = some_cache(pages, h, page, dk, dv, n)
    cache[2:] = [torch.rand(pages, h, device="cuda") for _ in range(2)]
    want = [x.clone() for x in cache]
    for a, b in zip(src, dst):
        for x in want:
            if a >= 0:
                x[b] = x[a]
    vlf.vlf_pages_copy(*cache, ints(src), ints(dst))
    assert vlf.vlf_check_error() == 0 and all(torch.equal(a, b) for a, b in zip(cache, want))


@pytest.mark.gpu
def test_copies_of_pages_outside_the_pool_are_recorded():
    cache = some_cache(6, 1, 16, 64, 64, 1)
    before = [x.clone() for x in cache]
    for src, dst in ([6], [1]), ([1], [6]), ([1], [-1]), ([2 ** 31 - 1], [0]):
        vlf.vlf_pages_copy(*cache, ints(src), ints(dst))
        assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_PAGES
        assert all(torch.equal(a, b) for a, b in zip(cache, before))
    vlf.vlf_pages_copy(*cache, ints([]), ints([]))


# ------------------------------------------------------------------------------ tables
def tables_of(r, n, page, most, share, spare):
    """Old rows of ragged lengths (zero among them), some sharing a prompt's whole pages, pages that others hold, free ones."""
    lens = [r.choice([0, 1, page, page * most, r.randint(0, page * most)]) for _ in range(n)]
    held = [-(-x // page) for x in lens]
    pages = sum(held) + spare
    order = list(range(pages))
    r.shuffle(order)
    rows, refs = [], [0] * pages
    for i, x in enumerate(held):
        common = min(lens[i] // page, lens[i - 1] // page, r.randint(0, most)) if i and r.random() < share else 0
        rows.append((rows[i - 1][:common] if common else []) + [order.pop() for _ in range(x - common)])
        for p in rows[-1]:
            refs[p] += 1
    for p in range(pages):
        if r.random() < 0.1:
            refs[p] += 1  # (held by someone else as well)
    pad = [row + [r.choice([-1, 7, 2 ** 31 - 1])] * (most - len(row)) for row in rows]  # (what is behind a row's end is not looked at)
    return pad, lens, refs


def check_fork(rows, lens, refs, parents, grow, page):
    most = len(rows[0]) if rows else 4
    want = ref.fork(rows, lens, refs, parents, grow, page)
    table = ints(rows).view(len(rows), most)
    got = vlf.vlf_pages_fork(table, ints(lens), ints(refs), ints(parents), ints(grow), page)
    assert vlf.vlf_check_error() == 0
    assert got[0].tolist() == [row + [-1] * (most - len(row)) for row in want[0]]
    for a, b in zip(got[1:], want[1:]):
        assert a.tolist() == (b if isinstance(b, list) else [b])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_fork_matches_the_definition(seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 64, 128, 256])
    n, most = r.choice([1, 5, 30]), r.choice([1, 3, 20, 300])
    rows, lens, refs = tables_of(r, n, page, most, 0.5, r.choice([0, 5, 4000]))
    m = r.choice([1, 8, 40, 300])
    parents = [r.randint(-1, n - 1) for _ in range(m)]
    grow = [min(r.choice([0, 1, page, 3 * page]), page * most - (lens[p] if p >= 0 else 0)) for p in parents]
    check_fork(rows, lens, refs, parents, grow, page)


@pytest.mark.gpu
def test_steps_of_forks_keep_the_counts():
    """Forked, ended, begun and grown over many steps: counts are what the tables hold, no page is lost, none shared that
    is written to."""
    r = random.Random(5)
    page, most, pages = 16, 12, 200
    table, lens, refs = torch.full((4, most), -1, dtype=I32, device="cuda"), ints([0] * 4), ints([0] * pages)
    for _ in range(30):
        n, m = lens.numel(), r.randint(1, 12)
        parents = [r.randint(-1, n - 1) for _ in range(m)]
        now = lens.tolist()
        grow = [min(r.randint(0, 20), page * most - (now[p] if p >= 0 else 0)) for p in parents]
        old = [row[:-(-x // page)] for row, x in zip(table.tolist(), now)]
        want = ref.fork(old, now, refs.tolist(), parents, grow, page)
        got = vlf.vlf_pages_fork(table, lens, refs, ints(parents), ints(grow), page)
        assert [x.tolist() for x in got[1:]] == [want[1], want[2], want[3], want[4], [want[5]]]
        if want[5] < 0:
            table, lens, refs = torch.full((1, most), -1, dtype=I32, device="cuda"), ints([0]), ints([0] * pages)
            continue
        table, lens, refs = got[:3]
        held = [p for row, x in zip(table.tolist(), lens.tolist()) for p in row[:-(-x // page)]]
        assert refs.tolist() == [held.count(p) for p in range(pages)]
        for row, x, g in zip(table.tolist(), lens.tolist(), grow):
            assert all(refs[p] == 1 for p in row[(x - g) // page:-(-x // page)])
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_fork_without_room_changes_nothing():
    rows, lens, refs = [[2, 0], [1, -1]], [20, 3], [1, 1, 1, 0]
    got = vlf.vlf_pages_fork(ints(rows), ints(lens), ints(refs), ints([0, 0, 1]), ints([0, 0, 13]), 16)
    assert got[5].tolist() == [0]
    got = check_fork(rows, lens, refs, [0, 0, 1, 1], [0, 0, 0, 0], 16)  # two copies, one page
    assert got[5].tolist() == [-1] and got[2].tolist() == refs


@pytest.mark.gpu
@pytest.mark.parametrize("change,status", [
    (dict(parents=[2, 0]), -8), (dict(rows=[[4, 0], [1, 9]]), -8), (dict(rows=[[-1, 0], [1, 9]]), -8), (dict(lens=[33, 3]), -6),
    (dict(lens=[-1, 3]), -6), (dict(grow=[13, 0]), -6), (dict(grow=[-1, 0]), -6), (dict(refs=[0, 1, 1, 0]), -8),
    (dict(refs=[1, 1, 1, -1]), -8), (dict(grow=[2 ** 31 - 1, 0]), -6)])
def test_fork_refuses_tables_that_disagree(change, status):
    a = dict(rows=[[2, 0], [1, 9]], lens=[20, 3], refs=[1, 1, 1, 0], parents=[0, 1], grow=[12, 0])
    check_fork(a["rows"], a["lens"], a["refs"], a["parents"], a["grow"], 16)
    a.update(change)
    got = vlf.vlf_pages_fork(ints(a["rows"]), ints(a["lens"]), ints(a["refs"]), ints(a["parents"]), ints(a["grow"]), 16)
    assert vlf.vlf_check_error() == status
    assert [x.tolist() for x in got] == [[[-1, -1]] * 2, [0, 0], a["refs"], [-1, -1], [-1, -1], [-2 ** 31]]


@pytest.mark.gpu
@pytest.mark.parametrize("pages,rows,most,every", [(300001, 9, 7000, 3), (300001, 700, 40, 50), (5000, 300, 17, 1), (4097, 1, 4097, 1)])
def test_fork_takes_free_pages_from_all_over_the_pool(pages, rows, most, every):
    """Rows whose new pages lie in many of the pool's chunks, more chunks and rows than are looked at at a time, and a pool
    that is used up to its last page."""
    r = random.Random(pages + rows)
    refs = [0 if p % every == 0 else r.randint(1, 3) for p in range(pages)]
    left = refs.count(0)
    grow = []
    for _ in range(rows):
        n = min(r.randint(0, most), left)
        grow.append(16 * n - (r.randint(0, 15) if n else 0))
        left -= n
    if left and left <= most - -(-grow[-1] // 16):
        grow[-1] += 16 * left
    none = torch.empty(0, most, dtype=I32, device="cuda")
    got = vlf.vlf_pages_fork(none, ints([]), ints(refs), ints([-1] * rows), ints(grow), 16)
    want = ref.fork([], [], refs, [-1] * rows, grow, 16)
    full = [x + [-1] * (most - len(x)) for x in want[0]]
    assert [x.tolist() for x in got] == [full, want[1], want[2], want[3], want[4], [want[5]]]
    assert want[5] >= 0 and vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_fork_of_nothing():
    none = torch.empty(0, 4, dtype=I32, device="cuda")
    got = vlf.vlf_pages_fork(none, ints([]), ints([0, 1]), ints([-1]), ints([5]), 16)
    assert [x.tolist() for x in got] == [[[0, -1, -1, -1]], [5], [1, 1], [-1], [-1], [0]]
    got = vlf.vlf_pages_fork(ints([[1, -1]]), ints([3]), ints([0, 1]), ints([]), ints([]), 16)  # all end
    assert got[0].shape == (0, 2) and got[2].tolist() == [0, 0] and got[5].tolist() == [2]
    got = vlf.vlf_pages_fork(none, ints([]), ints([]), ints([]), ints([]), 16)
    assert got[2].numel() == 0 and got[5].tolist() == [0]
    got = vlf.vlf_pages_fork(none, ints([]), ints([]), ints([-1]), ints([1]), 16)
    assert got[0].tolist() == [[-1] * 4] and got[5].tolist() == [-1]
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(10))
def test_compact_matches_the_definition(seed):
    r = random.Random(seed)
    pages = r.choice([1, 2, 3, 100, 1024, 1025, 5000, 40000])
    used = r.choice([0.0, 0.02, 0.5, 0.9, 1.0])
    refs = [r.randint(1, 4) if r.random() < used else 0 for _ in range(pages)]
    table = [[r.choice([-1, pages, 2 ** 31 - 1, r.randrange(pages)]) for _ in range(37)] for _ in range(r.choice([1, 9, 300]))]
    want = ref.compact(table, refs)
    got = vlf.vlf_pages_compact(ints(table), ints(refs))
    pad = [-1] * (pages // 2 - len(want[3]))
    for a, b in zip(got, (want[0], want[1], want[2], want[3] + pad, want[4] + pad, [want[5]])):
        assert a.tolist() == b


@pytest.mark.gpu
def test_compacted_pages_hold_what_they_held():
    r = random.Random(3)
    lens, page = [40, 300, 17], 16
    rows = some_table(lens, page, 90, 8)
    cache = some_cache(90, 2, page, 64, 64, 5)
    cache[2:] = [torch.rand(90, 2, device="cuda") for _ in range(2)]
    refs = [sum(p in row for row in rows) for p in range(90)]
    before = [[x[row[:-(-n // page)]].clone() for row, n in zip(rows, lens)] for x in cache]
    table, counts, to, src, dst, used = vlf.vlf_pages_compact(ints(rows), ints(refs))
    vlf.vlf_pages_copy(*cache, src, dst)
    n = int(used)
    assert n == sum(refs) and max(table.flatten().tolist()) < n and counts[:n].min() == 1 and not counts[n:].any()
    for x, b in zip(cache, before):
        for row, y, ln in zip(table.tolist(), b, lens):
            assert torch.equal(x[row[:-(-ln // page)]], y)


@pytest.mark.gpu
def test_tables_captured_on_streams_and_given_outputs():
    r = random.Random(9)
    rows, lens, refs = tables_of(r, 6, 32, 20, 0.5, 300)
    args = (ints(rows), ints(lens), ints(refs), ints([0, 0, 3, -1, 5]), ints([4, 0, 0, 40, 0]), 32)
    lens[0] = min(lens[0], 600)
    args[1].copy_(ints(lens))
    want = [x.clone() for x in vlf.vlf_pages_fork(*args)]
    moved = [x.clone() for x in vlf.vlf_pages_compact(args[0], args[2])]
    vlf.vlf_check_error()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, also = vlf.vlf_pages_fork(*args, stream=side), vlf.vlf_pages_compact(args[0], args[2], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*got, *also], [*want, *moved]))
    names = ("table_out", "seqlens_out", "refs_out", "src", "dst", "left")
    outs = {n: torch.full_like(x, 77) for n, x in zip(names, want)}
    back = vlf.vlf_pages_fork(*args, **outs)
    assert all(a is outs[n] and torch.equal(a, b) for n, a, b in zip(names, back, want))
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        a = vlf.vlf_pages_fork(*args)
    with torch.cuda.graph(two):
        b = vlf.vlf_pages_fork(*args)
    for _ in range(3):  # (two graphs at once: each has a workspace of its own)
        one.replay()
        with torch.cuda.stream(side):
            two.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, want))
    vlf.vlf_check_error()


# ------------------------------------------------------------------------------ refusals
def raw_write(**kw):
    a = dict(k=16, ks=128, v=16, vs=128, kp=16, vp=16, ksc=16, vsc=16, t=16, cu=16, lens=16, n=2, total=5, most=4, pages=9,
             page=16, h=2, dk=64, dv=64, dtype=1)
    a.update(kw)
    return vlf._lib.vlf_pages_write(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(total=-1), -1), (dict(most=-1), -1), (dict(pages=-1), -1), (dict(h=0), -1), (dict(dk=0), -1),
    (dict(dtype=9), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(kp=None), -1), (dict(vsc=None), -1), (dict(t=None), -1),
    (dict(cu=None), -1), (dict(lens=None), -1), (dict(n=0), -1), (dict(ks=-1), -1), (dict(page=0), -2), (dict(page=24), -2),
    (dict(page=512), -2), (dict(dk=257), -2), (dict(h=32768), -2), (dict(n=65536), -2), (dict(most=2 ** 27), -2),
    (dict(total=2 ** 31 - 1), -2), (dict(k=8), -3), (dict(vp=8), -3), (dict(t=4), -3), (dict(lens=4), -3)])
def test_write_refusals_before_any_launch(kw, status):
    if kw == dict(page=0):
        status = -2
    assert raw_write(**kw) == status


def raw_fork(**kw):
    a = dict(t=1 << 20, lens=2 << 20, refs=3 << 20, par=4 << 20, grow=5 << 20, n=2, m=3, most=4, pages=9, page=16, to=6 << 20,
             lo=7 << 20, ro=8 << 20, src=9 << 20, dst=10 << 20, left=11 << 20, ws=12 << 20, wsn=1 << 18)
    a.update(kw)
    return vlf._lib.vlf_pages_fork(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(m=-1), -1), (dict(pages=-1), -1), (dict(most=-1), -1), (dict(page=17), -2), (dict(m=65536), -2),
    (dict(n=65536), -2), (dict(most=2 ** 28), -2), (dict(t=None), -1), (dict(lens=None), -1), (dict(refs=None), -1),
    (dict(par=None), -1), (dict(to=None), -1), (dict(left=None), -1), (dict(ro=None), -1), (dict(left=4), -3), (dict(par=8), -3),
    (dict(ws=None), -7), (dict(wsn=64), -7), (dict(to=1 << 20), -1), (dict(ro=3 << 20), -1), (dict(lo=(6 << 20) + 16), -1),
    (dict(src=(12 << 20) + 256), -1), (dict(dst=9 << 20), -1), (dict(left=2 << 20), -1)])
def test_fork_refusals_before_any_launch(kw, status):
    assert raw_fork(**kw) == status


def raw_compact(**kw):
    a = dict(t=1 << 20, refs=2 << 20, n=2, most=4, pages=9, to=3 << 20, ro=4 << 20, map=5 << 20, src=6 << 20, dst=7 << 20,
             used=8 << 20, ws=9 << 20, wsn=1 << 18)
    a.update(kw)
    return vlf._lib.vlf_pages_compact(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(most=-1), -1), (dict(pages=0), -1), (dict(n=65536), -2), (dict(t=None), -1), (dict(refs=None), -1),
    (dict(to=None), -1), (dict(map=None), -1), (dict(src=None), -1), (dict(used=None), -1), (dict(used=4), -3),
    (dict(ws=None), -7), (dict(wsn=16), -7), (dict(to=1 << 20), -1), (dict(ro=2 << 20), -1), (dict(map=4 << 20), -1)])
def test_compact_refusals_before_any_launch(kw, status):
    assert raw_compact(**kw) == status


def raw_copy(**kw):
    a = dict(kp=16, vp=16, ksc=16, vsc=16, src=16, dst=16, n=2, pages=9, page=16, h=2, dk=64, dv=64)
    a.update(kw)
    return vlf._lib.vlf_pages_copy(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(src=None), -1), (dict(dst=None), -1), (dict(kp=None), -1), (dict(page=8), -2), (dict(dv=300), -2),
    (dict(src=4), -3), (dict(vp=4), -3), (dict(n=0), 0)])
def test_copy_refusals_before_any_launch(kw, status):
    assert raw_copy(**kw) == status


@pytest.mark.gpu
def test_refusals_with_tensors():
    c = some_cache(6, 2, 16, 64, 64, 1)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, cu, lens = ints([[0, 1], [2, 3]]), ints([0, 1, 3]), ints([5, 6])
    vlf.vlf_pages_write(k, k, *c, t, cu, lens)
    for bad in [lambda: vlf.vlf_pages_write(k[:, :1], k, *c, t, cu, lens), lambda: vlf.vlf_pages_write(k, k.float(), *c, t, cu, lens),
                lambda: vlf.vlf_pages_write(k, k[:2], *c, t, cu, lens), lambda: vlf.vlf_pages_write(k, k, *c, t[0], cu, lens),
                lambda: vlf.vlf_pages_write(k, k, *c, t, cu[:2], lens), lambda: vlf.vlf_pages_write(k, k, *c, t, cu, lens[:1]),
                lambda: vlf.vlf_pages_write(k, k, *c, t.long(), cu, lens), lambda: vlf.vlf_pages_write(k, k, *c, t, cu.cpu(), lens),
                lambda: vlf.vlf_pages_write(k, k, c[0].float(), *c[1:], t, cu, lens),
                lambda: vlf.vlf_pages_write(k, k, c[0][:5], *c[1:], t, cu, lens),
                lambda: vlf.vlf_pages_write(k, k, *c[:2], c[2][:, :1], c[3], t, cu, lens),
                lambda: vlf.vlf_pages_write(k, k, *c, t.t(), cu, lens),
                lambda: vlf.vlf_pages_copy(*c, ints([0]), ints([1, 2])), lambda: vlf.vlf_pages_copy(*c, ints([0]).long(), ints([1])),
                lambda: vlf.vlf_pages_fork(t, lens, ints([1] * 6), ints([0]), ints([0, 1]), 16),
                lambda: vlf.vlf_pages_fork(t, lens, ints([1] * 6), ints([0]), ints([0]), 15),
                lambda: vlf.vlf_pages_fork(t, lens, ints([1] * 6), ints([0]), ints([0]), 16, left=ints([1, 2])),
                lambda: vlf.vlf_pages_fork(t, lens, ints([1] * 6), ints([0, 1]), ints([0, 0]), 16, table_out=t),
                lambda: vlf.vlf_pages_compact(t[0], ints([1] * 6)), lambda: vlf.vlf_pages_compact(t, ints([]))]:
        with pytest.raises(vlf.VlfError):
            bad()
    assert vlf.vlf_check_error() == 0
