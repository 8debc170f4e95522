"""Cache eviction (vlf_cache_evict) against its definition: what is kept, its order, the gathered rows
and the output sequence lengths are all exact."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import decoding as ref

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def run(lens, h, dk, dv, dtype, budget, sink, recent, weights=None, seed=0, extra=0, max_kv=None):
    g = torch.Generator().manual_seed(seed)
    tk = sum(lens)
    k = torch.randn(tk, h, dk, generator=g).to(dtype).cuda()
    v = torch.randn(tk, h, dv, generator=g).to(dtype).cuda()
    if weights is None:
        weights = torch.randn(h, tk, generator=g).exp()
        weights[torch.rand(h, tk, generator=g) < 0.3] = 0.0  # ties
    w = weights.cuda()
    cu = cu_of(lens)
    kept, cu_out = ref.evict(weights.numpy(), cu.tolist(), budget, sink, recent)
    n = cu_out[-1] + extra
    # rows behind the last kept one stay as they were
    outs = dict(k_out=torch.full((n, h, dk), 7.0, dtype=dtype, device="cuda"),
                v_out=torch.full((n, h, dv), 7.0, dtype=dtype, device="cuda"),
                weights_out=torch.full((h, n), 7.0, device="cuda"),
                index_out=torch.full((h, n), 7, dtype=torch.int32, device="cuda"))
    ko, vo, wo, io, co = vlf.vlf_cache_evict(k, v, w, cu.cuda(), budget, sink, recent, max_seqlen_kv=max_kv,
                                             total_out=n, **outs)
    assert vlf.vlf_check_error() == 0
    assert co.tolist() == cu_out
    for hh in range(h):
        want = [j for s in kept[hh] for j in s]
        assert io[hh].tolist() == want + [7] * extra, (hh, len(want))
        at = torch.tensor([int(cu[s]) + j for s, js in enumerate(kept[hh]) for j in js], dtype=torch.long, device="cuda")
        m = len(want)
        assert torch.equal(ko[:m, hh], k[at, hh]) and torch.equal(vo[:m, hh], v[at, hh])
        a, b = wo[hh, :m], w[hh, at]
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    assert (ko[cu_out[-1]:] == 7).all() and (vo[cu_out[-1]:] == 7).all() and (wo[:, cu_out[-1]:] == 7).all()


CASES = [
    # lens, h, dk, dv, dtype, budget, sink, recent
    ([1], 1, 64, 64, BF, 1, 0, 0),
    ([5], 1, 64, 64, BF, 0, 0, 0),                       # nothing stays
    ([0, 3, 0], 2, 64, 64, HF, 2, 0, 1),                 # empty sequences
    ([17, 64, 100, 255], 4, 64, 64, HF, 64, 4, 16),
    ([1000, 31, 2047, 1], 3, 96, 96, BF, 100, 4, 32),
    ([1024, 1025, 1023], 2, 128, 128, BF, 1024, 1, 1),   # around a block's width
    ([5000, 300], 8, 128, 128, BF, 700, 4, 128),
    ([4097], 2, 192, 128, HF, 1000, 0, 0),               # latent head widths
    ([700, 900], 2, 40, 24, FP, 128, 3, 5),
    ([333], 3, 33, 7, HF, 50, 0, 10),                    # rows that are no whole 16-byte pieces
    ([333], 2, 5, 3, FP, 50, 10, 0),
    ([600], 2, 64, 64, BF, 40, 20, 20),                  # the protected keys fill the budget
    ([20000, 9000], 1, 64, 64, BF, 3001, 4, 64),
    ([40000], 2, 64, 64, HF, 12345, 16, 512),
    ([140001, 70000], 1, 64, 64, HF, 20001, 16, 512),
    ([420001], 1, 8, 16, HF, 5000, 4, 64),               # more keys than shared memory holds
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,h,dk,dv,dtype,budget,sink,recent", CASES)
def test_kept_keys_and_rows(lens, h, dk, dv, dtype, budget, sink, recent):
    run(lens, h, dk, dv, dtype, budget, sink, recent, seed=sum(lens))
    run(lens, h, dk, dv, dtype, budget, sink, recent, seed=sum(lens) + 1, extra=3, max_kv=max(lens) + 1000)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "inf", "lowest", "denormal", "close", "ascending"])
@pytest.mark.parametrize("n", [900, 30000])
def test_unusual_weights(kind, n):
    lens = [n, n // 3]
    tk = sum(lens)
    g = torch.Generator().manual_seed(1)
    w = torch.rand(2, tk, generator=g)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":
        w = torch.where(w < 0.5, torch.tensor(-0.0), torch.tensor(0.0))  # -0 equals +0
    elif kind == "nan":
        w[w < 0.8] = float("nan")  # NaN below every number, -inf among them
        w[:, 100:200] = -float("inf")
    elif kind == "inf":
        w[w < 0.7] = float("inf")
    elif kind == "lowest":
        w[w < 0.9] = torch.finfo(torch.float32).min
    elif kind == "denormal":
        w = w * 1e-40
    elif kind == "close":  # neighbours in the last bits
        w = (torch.randint(0, 50, (2, tk), generator=g, dtype=torch.int32) + 0x3f800000).view(torch.float32)
    else:
        w = torch.arange(2 * tk).view(2, tk).float()
    run(lens, 2, 64, 64, BF, n // 4, 4, 16, weights=w)


@pytest.mark.gpu
def test_many_sequences():
    lens = [(37 * i) % 90 for i in range(1500)]
    run(lens, 2, 64, 64, BF, 30, 2, 5)


@pytest.mark.gpu
def test_repeatable_and_captured():
    lens, h = [3000, 2500], 4
    k = torch.randn(5500, h, 64, device="cuda").to(BF)
    v = torch.randn(5500, h, 64, device="cuda").to(BF)
    w = torch.rand(h, 5500, device="cuda")
    cu = cu_of(lens).cuda()
    call = lambda **kw: vlf.vlf_cache_evict(k, v, w, cu, 512, 4, 64, max_seqlen_kv=3000, total_out=1024, **kw)  # noqa: E731
    first = call()
    for a, b in zip(first, call()):
        assert torch.equal(a, b)
    outs = [torch.zeros_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(k_out=outs[0], v_out=outs[1], weights_out=outs[2], index_out=outs[3], cu_out=outs[4])
    w.copy_(torch.rand(h, 5500, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, call()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    for a, b in zip(got, call()):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_default_rows_and_errors_on_the_device():
    k = torch.randn(300, 2, 64, device="cuda").to(BF)
    w = torch.rand(2, 300, device="cuda")
    cu = cu_of([100, 200]).cuda()
    ko, _, _, _, co = vlf.vlf_cache_evict(k, k, w, cu, 150)
    assert ko.shape[0] == 300 and co.tolist() == [0, 100, 250] and vlf.vlf_check_error() == 0
    # too few rows; a sequence longer than max_seqlen_kv; lengths that decrease; a total that differs
    before = torch.full((200, 2, 64), 3.0, device="cuda", dtype=BF)
    vlf.vlf_cache_evict(k, k, w, cu, 150, max_seqlen_kv=200, total_out=200, k_out=before)
    assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_SEQLENS
    assert (before[100:] == 3).all()
    for bad, mk in (([0, 100, 300], 150), ([0, 200, 100], 300), ([0, 100, 250], 300), ([5, 100, 300], 300),
                    ([0, 400, 300], 300), ([0, -7, 300], 300)):
        vlf.vlf_cache_evict(k, k, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), 150, max_seqlen_kv=mk)
        assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_SEQLENS, bad
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_a_budget_without_end_keeps_everything():
    k = torch.randn(50, 2, 64, device="cuda").to(BF)
    w = torch.rand(2, 50, device="cuda")
    cu = cu_of([20, 30]).cuda()
    ko, vo, wo, io, co = vlf.vlf_cache_evict(k, k, w, cu, 2 ** 40, sink=4)
    assert torch.equal(ko, k) and torch.equal(wo, w) and co.tolist() == [0, 20, 50]
    assert io[1].tolist() == list(range(20)) + list(range(30))
    with pytest.raises(vlf.VlfError):
        vlf.vlf_cache_evict(k, k, w, cu, 2 ** 40, sink=2 ** 33)
    with pytest.raises(vlf.VlfError):
        vlf.vlf_cache_evict(k, k, w, cu, 10, max_seqlen_kv=2 ** 32 + 30)


def _raw(**kw):
    a = dict(k=16, v=16, w=16, cu=16, n=1, tk=8, mk=8, h=2, dk=64, dv=64, dtype=1, budget=4, sink=1, recent=1,
             to=4, ko=16, vo=16, wo=16, io=16, co=16)
    a.update(kw)
    return vlf._lib.vlf_cache_evict(*[a[x] for x in ("k", "v", "w", "cu", "n", "tk", "mk", "h", "dk", "dv", "dtype",
                                                      "budget", "sink", "recent", "to", "ko", "vo", "wo", "io", "co")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(budget=-1, sink=0, recent=0), vlf.VLF_ERR_INVALID), (dict(sink=2, recent=3), vlf.VLF_ERR_INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), vlf.VLF_ERR_INVALID), (dict(sink=-1), vlf.VLF_ERR_INVALID),
    (dict(dtype=3), vlf.VLF_ERR_INVALID), (dict(w=None), vlf.VLF_ERR_INVALID), (dict(io=None), vlf.VLF_ERR_INVALID),
    (dict(co=None), vlf.VLF_ERR_INVALID), (dict(h=0), vlf.VLF_ERR_INVALID), (dict(n=0), vlf.VLF_ERR_INVALID),
    (dict(dk=257), vlf.VLF_ERR_UNSUPPORTED), (dict(n=70000), vlf.VLF_ERR_UNSUPPORTED),
    (dict(io=20), vlf.VLF_ERR_ALIGN), (dict(n=0, tk=0), vlf.VLF_OK),
])
def test_host_refusals(kw, status):
    assert _raw(**kw) == status


@pytest.mark.gpu
def test_python_refusals():
    k = torch.zeros(10, 2, 64, device="cuda", dtype=BF)
    w = torch.zeros(2, 10, device="cuda")
    cu = cu_of([10]).cuda()
    for kw in (dict(weights=w.t().contiguous()), dict(weights=w.double()), dict(v=k.float()), dict(k=k[:, :1].contiguous()),
               dict(budget=3, sink=4), dict(cu_seqlens_kv=cu.long()), dict(total_out=5, k_out=k), dict(k=k.transpose(0, 1))):
        a = dict(k=k, v=k, weights=w, cu_seqlens_kv=cu, budget=5)
        a.update(kw)
        with pytest.raises(vlf.VlfError):
            vlf.vlf_cache_evict(**a)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[20000, 9000], [100, 300, 7], [140001]])
def test_loose_bounds_on_the_lengths(lens):
    """A longest length that is an upper bound alone, up to the largest int."""
    for most in (sum(lens), 10 ** 6, 2 ** 31 - 8, 2 ** 31 - 1):
        run(lens, 2, 64, 64, BF, 64, 4, 16, seed=3, max_kv=most)


def test_sizes_next_to_the_largest_int_are_refused():
    assert _raw(tk=2 ** 31 - 1) == vlf.VLF_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(ko=1 << 20), dict(vo=(1 << 20) + 2032), dict(vo=1 << 20), dict(wo=2 << 20), dict(io=3 << 20),
                                dict(co=(4 << 20) + 16), dict(ko=5 << 20), dict(wo=(5 << 20) + 1008)])
def test_outputs_that_overlap_are_refused(kw):
    """In place, on another input, on another output: k is 8 rows x 2 heads x 64 x 2 bytes at 1 MB."""
    a = dict(k=1 << 20, v=2 << 20, w=3 << 20, cu=4 << 20, n=4, ko=16, vo=5 << 20, wo=6 << 20, io=7 << 20, co=8 << 20)
    assert _raw(**dict(a, **kw)) == vlf.VLF_ERR_INVALID


@pytest.mark.gpu
def test_a_cache_is_not_cut_in_place():
    k, w, cu = torch.randn(300, 2, 64, device="cuda").to(BF), torch.rand(2, 300, device="cuda"), cu_of([100, 200]).cuda()
    for kw in (dict(k_out=k), dict(v_out=k[:200]), dict(k_out=k[100:]), dict(cu_out=cu), dict(weights_out=w)):
        rows = kw["k_out"].shape[0] if "k_out" in kw else 300 if "weights_out" in kw else 200
        with pytest.raises(vlf.VlfError):
            vlf.vlf_cache_evict(k, k.clone(), w, cu, 100, max_seqlen_kv=200, total_out=rows, **kw)
