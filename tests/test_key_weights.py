"""The attention weight each key received (vlf_attn_key_weights) against its fp64 definition.

Tolerance.  A logit is off by Delta = scale D 2^-23 sum |q k| at most, the exponent's argument by 2^-22
of |logit| and |lse|, the exponential by 2^-21; a key's sum of n positive terms, kept in sums of at
most 1024 terms that are then added, by 2^-24 (1024 + n / 1024) of it:
    |error| <= w (exp(max Delta + 2^-21 (1 + max |logit| + max |lse|)) - 1 + 2^-13)
The bound on long sums is the worst case; 2^-16 is asserted up to 64 terms."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import decoding as ref

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def np64(t):
    return t.detach().cpu().double().numpy()


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def make(q_lens, kv_lens, hq, hkv, d, dtype, causal, window, seed, scale=None, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (sigma * torch.randn(sum(q_lens), hq, d, generator=g)).to(dtype).cuda()
    k = (sigma * torch.randn(sum(kv_lens), hkv, d, generator=g)).to(dtype).cuda()
    cq, ck = cu_of(q_lens), cu_of(kv_lens)
    none = np.zeros((0, hkv, d))
    _, L = ref.prefix_forward(np64(q), none, none, np64(k), np64(k), cq.tolist(), ck.tolist(), scale or d ** -0.5,
                              causal, window)
    lse = torch.tensor(L, dtype=torch.float32).cuda()
    return dict(q=q, k=k, lse=lse, cu_seqlens_q=cq.cuda(), cu_seqlens_kv=ck.cuda(), max_seqlen_q=max(q_lens),
                max_seqlen_kv=max(kv_lens), causal=causal, window=window, scale=scale)


def verify(x, w, prev=None):
    q, k, lse = np64(x["q"]), np64(x["k"]), np64(x["lse"])
    d, sc = q.shape[2], x["scale"] or q.shape[2] ** -0.5
    args = (q, k, lse, x["cu_seqlens_q"].tolist(), x["cu_seqlens_kv"].tolist(), sc, x["causal"], x["window"])
    want = ref.key_weights(*args)
    reach = sc * np.sqrt((q ** 2).sum(-1).max() * (k ** 2).sum(-1).max()) if q.size and k.size else 0.0
    live = lse[np.isfinite(lse)]
    arg = reach * d * 2.0 ** -23 + 2.0 ** -21 * (1 + reach + (np.abs(live).max() if live.size else 0.0))
    terms = x["max_seqlen_q"] * q.shape[1] // k.shape[1]
    tol = want * (np.expm1(arg) + (2.0 ** -16 if terms <= 64 else 2.0 ** -13)) + 1e-37
    if prev is not None:
        want = want + np64(prev)
        tol = tol + 2.0 ** -23 * np.abs(want)
    got = np64(w)
    assert got.shape == want.shape
    err = np.abs(got - want)
    assert (err <= tol).all(), (err.max(), (err / np.maximum(want, 1e-30)).max())


CASES = [
    # q_lens, kv_lens, hq, hkv, d, dtype, causal, window
    ([1], [1], 1, 1, 64, BF, True, 0),
    ([1, 1, 1, 1], [17, 64, 100, 255], 8, 2, 128, BF, True, 0),
    ([1, 1], [1000, 129], 32, 4, 128, HF, True, 0),
    ([1] * 7, [128, 127, 129, 1, 500, 256, 64], 6, 2, 96, BF, True, 0),         # groups of 3
    ([32, 17], [700, 300], 8, 2, 128, HF, True, 0),                             # 128 columns
    ([33, 5], [700, 300], 8, 2, 64, BF, True, 0),                               # just above
    ([300, 129], [300, 129], 4, 4, 128, BF, True, 0),
    ([300, 129], [300, 129], 4, 4, 128, BF, False, 0),
    ([200, 64], [450, 640], 6, 2, 64, HF, True, 100),                           # window, groups of 3
    ([200, 64], [450, 640], 4, 2, 128, BF, False, 50),
    ([90, 4], [30, 2], 4, 2, 64, BF, True, 0),                                  # rows that see no key
    ([0, 5, 0], [50, 60, 0], 4, 2, 64, HF, True, 0),                            # keys without rows
    ([3], [900], 16, 1, 192, BF, True, 0),                                      # latent head width
    ([70], [333], 130, 1, 64, BF, True, 0),                                     # 130 heads on one
    ([9, 40], [90, 100], 4, 2, 256, BF, True, 0),
    ([9, 40], [90, 100], 4, 2, 40, HF, True, 0),
    ([9, 40], [90, 100], 4, 2, 33, BF, True, 7),
    ([9, 40], [90, 100], 6, 2, 64, FP, True, 0),
    ([1, 1], [90, 100], 6, 2, 128, FP, True, 0),
    ([1500], [1500], 8, 1, 64, HF, True, 0),                                    # few CTAs, long rows: split
    ([2000], [40], 4, 1, 128, BF, False, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,dtype,causal,window", CASES)
def test_matches_the_definition(q_lens, kv_lens, hq, hkv, d, dtype, causal, window):
    x = make(q_lens, kv_lens, hq, hkv, d, dtype, causal, window, seed=sum(kv_lens))
    prev = torch.rand(hkv, sum(kv_lens), device="cuda")
    for flags in (0, vlf.VLF_FLAG_FORCE_SIMT):
        w = vlf.vlf_attn_key_weights(**x, flags=flags)
        verify(x, w)
        verify(x, vlf.vlf_attn_key_weights(**x, flags=flags, prev=prev), prev)
        acc = prev.clone()
        assert vlf.vlf_attn_key_weights(**x, flags=flags, prev=acc, weights=acc) is acc  # in place
        verify(x, acc, prev)
        assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_random_shapes():
    rng = np.random.default_rng(5)
    for n in range(40):
        seqs, top = int(rng.integers(1, 8)), int(rng.choice([1, 4, 40, 300]))
        q_lens = [int(rng.integers(0 if seqs > 1 else 1, top + 1)) for _ in range(seqs)]
        q_lens[0] = max(1, q_lens[0])
        kv_lens = [int(rng.integers(0, 500)) for _ in range(seqs)]
        kv_lens[-1] = max(1, kv_lens[-1])
        hkv, grp = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 4, 5, 8]))
        x = make(q_lens, kv_lens, hkv * grp, hkv, int(rng.choice([64, 96, 128, 192])), [BF, HF][n % 2],
                 bool(rng.integers(0, 2)), int(rng.choice([0, 0, 1, 50, 400])), seed=n)
        verify(x, vlf.vlf_attn_key_weights(**x))
        assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_rows_of_a_full_softmax_add_up():
    """Without a mask every row's weights sum to 1, so a group's keys receive rows x heads."""
    x = make([50], [700], 8, 2, 128, BF, False, 0, seed=3)
    w = vlf.vlf_attn_key_weights(**x)
    assert (w.double().sum(1) - 50 * 4).abs().max() <= 200 * 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [150, 90, 10]])
def test_other_sequences_never_reach_a_key(q_lens):
    x = make(q_lens, [200, 180, 150], 8, 2, 128, BF, True, 0, seed=4)
    clean = vlf.vlf_attn_key_weights(**x)
    a, b = q_lens[0], q_lens[0] + q_lens[1]
    x["q"][a:b] = float("nan")
    w = vlf.vlf_attn_key_weights(**x)
    assert torch.equal(w[:, :200], clean[:, :200]) and torch.equal(w[:, 380:], clean[:, 380:])
    x["q"][a:b] = 0
    x["k"][200:380] = float("inf")
    w = vlf.vlf_attn_key_weights(**x)
    assert torch.equal(w[:, :200], clean[:, :200]) and torch.equal(w[:, 380:], clean[:, 380:])


@pytest.mark.gpu
def test_masked_rows_and_lowest_lse():
    """lse = -inf takes a row out; nothing else changes."""
    x = make([40, 1], [300, 100], 8, 2, 128, HF, True, 0, seed=6)
    x["lse"][:, 3] = -float("inf")
    x["lse"][2] = -float("inf")
    verify(x, vlf.vlf_attn_key_weights(**x))


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, vlf.VLF_FLAG_FORCE_SIMT])
@pytest.mark.parametrize("q_lens,causal", [([1, 1], True), ([2, 9], True), ([20, 32], True), ([32, 32], False),
                                           ([200, 40], False), ([200, 40], True)])
def test_rows_without_an_lse_may_hold_anything(q_lens, causal, flags):
    """(a row without an lse gives exactly nothing, so the sums are the same to the bit)"""
    x = make(q_lens, [300, 150], 8, 2, 128, BF, causal, 0, seed=8)
    rows = [0, sum(q_lens) // 2, sum(q_lens) - 1]
    x["lse"][:, rows] = -float("inf")
    x["q"][rows] = 0
    want = vlf.vlf_attn_key_weights(**x, flags=flags)
    assert want.isfinite().all()
    for bad in (float("nan"), float("inf")):
        x["q"][rows] = bad
        assert torch.equal(vlf.vlf_attn_key_weights(**x, flags=flags), want)


@pytest.mark.gpu
def test_no_rows_at_all():
    q = torch.empty(0, 4, 64, device="cuda", dtype=BF)
    k = torch.randn(30, 2, 64, device="cuda").to(BF)
    prev = torch.rand(2, 30, device="cuda")
    a = dict(q=q, k=k, lse=torch.empty(4, 0, device="cuda"), cu_seqlens_q=cu_of([0, 0]).cuda(),
             cu_seqlens_kv=cu_of([10, 20]).cuda(), max_seqlen_q=0, max_seqlen_kv=20)
    assert not vlf.vlf_attn_key_weights(**a).any()
    assert torch.equal(vlf.vlf_attn_key_weights(**a, prev=prev), prev)
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [500, 900]), ([700], [700])])
def test_captured_on_streams_and_repeatable(q_lens, kv_lens):
    x = make(q_lens, kv_lens, 8, 2, 128, BF, True, 0, seed=7)
    first = vlf.vlf_attn_key_weights(**x)
    for _ in range(3):
        assert torch.equal(vlf.vlf_attn_key_weights(**x), first)
    need = vlf.vlf_attn_key_weights_workspace_size(len(q_lens), sum(kv_lens), max(q_lens), max(kv_lens), 8, 2, 128, BF)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    acc = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vlf.vlf_attn_key_weights(**x, prev=acc, weights=acc, workspace=ws)
    acc.zero_(), ws.fill_(255)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(acc, first + first)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [vlf.vlf_attn_key_weights(**x, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, first) for g in got)
    if need:
        with pytest.raises(vlf.VlfError):
            vlf.vlf_attn_key_weights(**x, workspace=ws[:need - 1].clone())


@pytest.mark.gpu
def test_bad_sequence_lengths_are_reported():
    x = make([4, 4], [50, 60], 4, 2, 64, BF, True, 0, seed=1)
    for name, bad in (("cu_seqlens_q", [0, 4, 9]), ("cu_seqlens_q", [0, 9, 8]), ("cu_seqlens_kv", [0, 50, 100]),
                      ("cu_seqlens_kv", [0, 90, 110]), ("cu_seqlens_kv", [1, 50, 110]), ("cu_seqlens_q", [0, -3, 8])):
        y = dict(x, **{name: torch.tensor(bad, dtype=torch.int32, device="cuda")})
        for flags in (0, vlf.VLF_FLAG_FORCE_SIMT):
            vlf.vlf_attn_key_weights(**y, flags=flags)
            assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_SEQLENS, (name, bad, flags)


def _raw(**kw):
    a = dict(q=16, k=16, lse=16, cq=16, ck=16, n=2, tq=2, tk=8, mq=1, mk=8, hq=4, hkv=2, d=64, dtype=1, scale=0.0,
             causal=1, window=0, prev=None, w=16, ws=None, wb=0)
    a.update(kw)
    return vlf._lib.vlf_attn_key_weights(*[a[x] for x in (
        "q", "k", "lse", "cq", "ck", "n", "tq", "tk", "mq", "mk", "hq", "hkv", "d", "dtype", "scale", "causal", "window",
        "prev", "w", "ws", "wb")], None, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), vlf.VLF_ERR_INVALID), (dict(w=None), vlf.VLF_ERR_INVALID), (dict(k=None), vlf.VLF_ERR_INVALID),
    (dict(hq=5), vlf.VLF_ERR_INVALID), (dict(dtype=-1), vlf.VLF_ERR_INVALID), (dict(d=0), vlf.VLF_ERR_INVALID),
    (dict(d=257), vlf.VLF_ERR_UNSUPPORTED), (dict(prev=20), vlf.VLF_ERR_ALIGN), (dict(w=20), vlf.VLF_ERR_ALIGN),
    (dict(mk=0), vlf.VLF_OK), (dict(n=0, tq=0, tk=0), vlf.VLF_OK),
])
def test_host_refusals(kw, status):
    assert _raw(**kw) == status


@pytest.mark.gpu
def test_python_refusals():
    x = make([4], [50], 4, 2, 64, BF, True, 0, seed=1)
    for kw in (dict(lse=x["lse"].double()), dict(lse=x["lse"][:, :3].contiguous()), dict(k=x["k"].float()),
               dict(weights=torch.empty(2, 49, device="cuda")), dict(prev=torch.empty(2, 50)),
               dict(cu_seqlens_q=cu_of([2, 2]).cuda()), dict(q=x["q"].transpose(0, 1))):
        with pytest.raises(vlf.VlfError):
            vlf.vlf_attn_key_weights(**dict(x, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, vlf.VLF_FLAG_FORCE_SIMT])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [17, 136, 255]), ([90, 150], [190, 201]), ([700], [700])])
def test_loose_bounds_on_the_lengths(q_lens, kv_lens, flags):
    """Longest lengths that are upper bounds alone, up to the largest int."""
    x = make(q_lens, kv_lens, 8, 2, 128, BF, True, 0, seed=1)
    for mq, mk in ((max(q_lens), 16384), (1000, 100000), (2 ** 31 - 1, 2 ** 31 - 1)):
        verify(x, vlf.vlf_attn_key_weights(**dict(x, max_seqlen_q=mq, max_seqlen_kv=mk), flags=flags))
        assert vlf.vlf_check_error() == 0


@pytest.mark.parametrize("kw", [dict(tq=2 ** 31 - 1), dict(tk=2 ** 31 - 1)])
def test_sizes_next_to_the_largest_int_are_refused(kw):
    assert _raw(**kw) == vlf.VLF_ERR_UNSUPPORTED
