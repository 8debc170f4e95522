"""Attention behind a shared prefix (vlf_attn_varlen_fwd_prefix) against the fp64 softmax over the
concatenated keys, and against vlf_attn_varlen_fwd on them.

Tolerances.  A logit is a dot product of D exact products in fp32: off by Delta = scale D 2^-23
sum |q k| at most.  A weight is then off by a factor of 2 max Delta, of 2^-20 (exponential, maxima and
sums in fp32) and, where the weights are rounded to the 16-bit type before the product with V and the
output is divided by their rounded sum, of 2 u; the output is rounded once (u).
    out: u |out| + (2 u + 2 max Delta + 2^-20) sum_j P_j |v_j|
    lse: max Delta + 2^-20 (1 + |lse|)"""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import decoding as ref

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, HF: 2.0 ** -11, FP: 2.0 ** -24}


def np64(t):
    return t.detach().cpu().double().numpy()


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def make(prefix, q_lens, kv_lens, hq, hkv, dqk, dv, dtype, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (sigma * torch.randn(*s, generator=g)).to(dtype).cuda()  # noqa: E731
    return dict(q=r(sum(q_lens), hq, dqk), k_prefix=r(prefix, hkv, dqk), v_prefix=r(prefix, hkv, dv),
                k=r(sum(kv_lens), hkv, dqk), v=r(sum(kv_lens), hkv, dv), cu_seqlens_q=cu_of(q_lens).cuda(),
                cu_seqlens_kv=cu_of(kv_lens).cuda(), max_seqlen_q=max(q_lens), max_seqlen_kv=max(kv_lens))


def verify(x, out, lse, causal, window, scale=None):
    a = {n: np64(t) if isinstance(t, torch.Tensor) and t.is_floating_point() else t for n, t in x.items()}
    cq, ck = x["cu_seqlens_q"].tolist(), x["cu_seqlens_kv"].tolist()
    sc = scale or x["q"].shape[2] ** -0.5
    args = (a["q"], a["k_prefix"], a["v_prefix"], a["k"], a["v"], cq, ck, sc, causal, window)
    O, L = ref.prefix_forward(*args)
    Oabs, _ = ref.prefix_forward(a["q"], a["k_prefix"], np.abs(a["v_prefix"]), a["k"], np.abs(a["v"]), *args[5:])
    # max Delta over a row's keys is at most scale D 2^-23 |q| max |k|
    kn = max([np.sqrt((a[n] ** 2).sum(-1)).max() for n in ("k", "k_prefix") if a[n].size] or [0.0])
    delta = sc * x["q"].shape[2] * 2.0 ** -23 * np.sqrt((a["q"] ** 2).sum(-1)) * kn  # [Tq, Hq]
    u = UNIT[out.dtype]
    uw = u if out.dtype != FP else 0.0
    tol = u * np.abs(O) + (2 * uw + 2 * delta[..., None] + 2.0 ** -20) * Oabs
    err = np.abs(np64(out) - O)
    assert (err <= tol).all(), (err.max(), (err - tol).max())
    gl = np64(lse)
    dead = np.isneginf(L)
    assert (np.isneginf(gl) == dead).all()
    lerr = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, L))
    assert (lerr <= delta.T + 2.0 ** -20 * (1 + np.abs(np.where(dead, 0, L)))).all(), lerr.max()


CASES = [
    # prefix, q_lens, kv_lens, hq, hkv, (dqk, dv), dtype, causal, window
    (1000, [1, 1, 1], [17, 136, 255], 8, 8, (64, 64), HF, True, 0),
    (700, [1] * 9, [64, 65, 1, 127, 128, 300, 63, 5, 200], 8, 2, (128, 128), BF, True, 0),
    (130, [1, 1], [1, 1], 4, 1, (96, 96), BF, True, 0),
    (63, [5, 64, 1, 100], [5, 200, 9, 100], 6, 2, (128, 128), BF, True, 0),      # groups of 3
    (257, [33, 130, 300], [300, 130, 333], 8, 2, (128, 128), HF, True, 0),       # several row blocks
    (640, [40, 1, 200], [100, 700, 250], 4, 4, (64, 64), BF, True, 0),
    (640, [40, 1, 200], [100, 700, 250], 4, 4, (64, 64), BF, False, 0),          # no causal rule
    (500, [3, 90], [50, 100], 8, 4, (64, 64), HF, True, 77),                     # window: own keys and a bit of the prefix
    (500, [3, 90], [50, 100], 8, 4, (128, 128), BF, True, 7),                    # window inside the own keys
    (500, [70, 5], [50, 100], 8, 4, (128, 128), BF, False, 300),                 # window alone
    (200, [50, 20], [10, 0], 4, 2, (64, 64), BF, True, 0),                       # rows inside the prefix; no own keys
    (40, [90, 3], [10, 2], 4, 2, (128, 128), HF, True, 0),                       # more rows than keys: some see none
    (0, [7, 1], [30, 100], 4, 2, (128, 128), BF, True, 0),                       # no prefix
    (0, [7, 2], [0, 3], 4, 2, (64, 64), BF, False, 0),                           # a sequence without keys
    (128, [0, 4, 0, 1], [5, 60, 0, 64], 4, 2, (64, 64), HF, True, 0),            # empty sequences
    (300, [1] * 5, [40, 80, 120, 160, 200], 16, 1, (64, 64), BF, True, 0),       # one kv head
    (300, [2, 1], [40, 80], 130, 1, (64, 64), BF, True, 0),                      # 130 heads on one
    (5000, [1, 2], [30, 500], 4, 2, (128, 128), BF, True, 0),                    # long prefix, split
    (70, [1, 3], [90, 200], 4, 2, (256, 256), BF, True, 0),
    (70, [1, 3], [90, 200], 4, 2, (192, 128), BF, True, 0),
    (70, [9, 3], [90, 200], 4, 2, (80, 48), HF, True, 0),
    (70, [9, 3], [90, 200], 4, 2, (33, 17), BF, True, 50),
    (70, [9, 3], [90, 200], 6, 2, (64, 64), FP, True, 0),
    (129, [1, 1], [33, 64], 4, 2, (128, 128), FP, True, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,q_lens,kv_lens,hq,hkv,d,dtype,causal,window", CASES)
def test_matches_the_softmax_over_concatenated_keys(prefix, q_lens, kv_lens, hq, hkv, d, dtype, causal, window):
    x = make(prefix, q_lens, kv_lens, hq, hkv, *d, dtype, seed=prefix + hq)
    for flags in (0, vlf.VLF_FLAG_FORCE_SIMT):
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=causal, window=window, flags=flags)
        assert vlf.vlf_check_error() == 0
        verify(x, out, lse, causal, window)


@pytest.mark.gpu
def test_random_shapes():
    rng = np.random.default_rng(11)
    for n in range(40):
        seqs = int(rng.integers(1, 12))
        top = int(rng.choice([1, 3, 40, 150]))
        q_lens = [int(rng.integers(0 if seqs > 1 else 1, top + 1)) for _ in range(seqs)]
        q_lens[0] = max(1, q_lens[0])
        kv_lens = [int(rng.integers(0, 300)) for _ in range(seqs)]
        hkv, grp = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 4, 5, 8]))
        d = int(rng.choice([64, 96, 128]))
        x = make(int(rng.integers(0, 900)), q_lens, kv_lens, hkv * grp, hkv, d, d, [BF, HF][n % 2], seed=n)
        causal, window = bool(rng.integers(0, 2)), int(rng.choice([0, 0, 1, 50, 400]))
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=causal, window=window)
        assert vlf.vlf_check_error() == 0
        verify(x, out, lse, causal, window)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [70, 33, 100]), ([80, 150], [90, 201])])
def test_other_sequences_never_reach_a_row(q_lens, kv_lens):
    """NaN and infinities in one sequence's keys and values stay in that sequence; so do the rows of q."""
    x = make(200, q_lens, kv_lens, 8, 2, 128, 128, BF, seed=4)
    clean, clean_lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True)
    last = len(q_lens) - 1
    a, b = kv_lens[0], kv_lens[0] + kv_lens[1]
    x["k"][a:b], x["v"][a:b] = float("nan"), float("inf")
    out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True)
    assert vlf.vlf_check_error() == 0
    q0, q1 = q_lens[0], q_lens[0] + q_lens[1]
    assert torch.equal(out[:q0], clean[:q0]) and torch.equal(lse[:, :q0], clean_lse[:, :q0])
    if last > 1:
        assert torch.equal(out[q1:], clean[q1:]) and torch.equal(lse[:, q1:], clean_lse[:, q1:])
    assert out[q0:q1].isnan().any()
    x["k"][a:b], x["v"][a:b] = 1.0, 1.0
    x["q"][:q0] = float("nan")
    out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True)
    assert out[q0:].isfinite().all() and lse[:, q0:].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,q_lens,kv_lens", [(200, [1, 1], [70, 33]), (5000, [1, 3], [40, 90]), (300, [80, 150], [90, 201])])
def test_a_nan_key_reaches_its_rows(prefix, q_lens, kv_lens):
    """However the keys are cut: a visible NaN makes the row and its log-sum-exp NaN, a masked one does not."""
    x = make(prefix, q_lens, kv_lens, 8, 2, 64, 64, BF, seed=3)
    for name, rows in (("k_prefix", slice(None)), ("k", slice(q_lens[0], None))):
        y = dict(x, **{name: x[name].clone()})
        y[name][17 if name == "k_prefix" else kv_lens[0] + 1] = float("nan")
        for flags in (0, vlf.VLF_FLAG_FORCE_SIMT):
            out, lse = vlf.vlf_attn_varlen_fwd_prefix(**y, causal=True, flags=flags)
            assert out[rows].isnan().all() and lse[:, rows].isnan().all()
            if name == "k":
                assert out[:q_lens[0]].isfinite().all() and lse[:, :q_lens[0]].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("sigma", [0.02, 6.0])
def test_flat_and_sharp_weights(sigma):
    x = make(900, [1, 40], [100, 90], 8, 2, 128, 128, HF, seed=8, sigma=sigma)
    out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, scale=0.1)
    verify(x, out, lse, True, 0, scale=0.1)


@pytest.mark.gpu
def test_agrees_with_the_forward_on_concatenated_keys():
    lens = [64, 300, 5]
    x = make(512, [1, 1, 1], lens, 8, 2, 128, 128, BF, seed=2)
    out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True)
    ks, vs, a = [], [], 0
    for n in lens:
        ks += [x["k_prefix"], x["k"][a:a + n]]
        vs += [x["v_prefix"], x["v"][a:a + n]]
        a += n
    full = [512 + n for n in lens]
    want, wlse = vlf.vlf_attn_varlen_fwd(x["q"], torch.cat(ks), torch.cat(vs), x["cu_seqlens_q"], cu_of(full).cuda(), 1,
                                         max(full), causal=True)
    # both are within the tolerance above of the same value: |v| < 5, weights sum to 1
    assert (out.float() - want.float()).abs().max() <= 2 * 4 * 2.0 ** -8 * want.float().abs().max() + 2 * 3 * 2.0 ** -8
    assert (lse - wlse).abs().max() <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("q_len", [1, 100])
def test_captured_on_streams_and_repeatable(q_len):
    x = make(4000, [q_len] * 3, [300, 200, 150], 8, 2, 128, 128, BF, seed=5)
    call = lambda **kw: vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, **kw)  # noqa: E731
    out, lse = call()
    for _ in range(3):
        o, l = call()
        assert torch.equal(o, out) and torch.equal(l, lse)
    need = vlf.vlf_attn_varlen_fwd_prefix_workspace_size(3, 3 * q_len, q_len, 300, 4000, 8, 2, 128, 128, BF)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=o, lse=l, workspace=ws)
    x["q"].copy_(torch.randn_like(x["q"]))
    ws.fill_(255)  # (NaN: nothing is read before it is written)
    graph.replay()
    torch.cuda.synchronize()
    want, wl = call()
    assert torch.equal(o, want) and torch.equal(l, wl)
    side, side2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [call(stream=s) for s in (side, side2)]  # two calls at once, each with its own workspace
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, wl)
    if need:
        with pytest.raises(vlf.VlfError):
            call(workspace=ws[:need - 1].clone())


@pytest.mark.gpu
def test_bad_sequence_lengths_are_reported():
    x = make(100, [4, 4], [50, 60], 4, 2, 64, 64, BF, seed=1)
    for name, bad in (("cu_seqlens_q", [0, 4, 9]), ("cu_seqlens_q", [0, 9, 8]), ("cu_seqlens_kv", [0, 50, 100]),
                      ("cu_seqlens_kv", [0, 90, 110]), ("cu_seqlens_kv", [1, 50, 110]), ("cu_seqlens_q", [0, -3, 8])):
        y = dict(x, **{name: torch.tensor(bad, dtype=torch.int32, device="cuda")})
        for flags in (0, vlf.VLF_FLAG_FORCE_SIMT):
            vlf.vlf_attn_varlen_fwd_prefix(**y, causal=True, flags=flags)
            assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_SEQLENS, (name, bad, flags)
    vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True)
    assert vlf.vlf_check_error() == 0


def _raw(**kw):
    a = dict(q=16, kp=16, vp=16, pl=100, k=16, v=16, cq=16, ck=16, n=2, tq=2, tk=8, mq=1, mk=8, hq=4, hkv=2, dqk=64,
             dv=64, dtype=1, scale=0.0, causal=1, window=0, out=16, lse=16, ws=None, wb=0)
    a.update(kw)
    return vlf._lib.vlf_attn_varlen_fwd_prefix(*[a[x] for x in (
        "q", "kp", "vp", "pl", "k", "v", "cq", "ck", "n", "tq", "tk", "mq", "mk", "hq", "hkv", "dqk", "dv", "dtype",
        "scale", "causal", "window", "out", "lse", "ws", "wb")], None, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(kp=None), vlf.VLF_ERR_INVALID), (dict(pl=-1), vlf.VLF_ERR_INVALID), (dict(out=None), vlf.VLF_ERR_INVALID),
    (dict(hq=3), vlf.VLF_ERR_INVALID), (dict(dtype=5), vlf.VLF_ERR_INVALID), (dict(k=None), vlf.VLF_ERR_INVALID),
    (dict(dqk=300), vlf.VLF_ERR_UNSUPPORTED), (dict(pl=2 ** 31 - 5), vlf.VLF_ERR_UNSUPPORTED),
    (dict(vp=8), vlf.VLF_ERR_ALIGN), (dict(lse=8), vlf.VLF_ERR_ALIGN), (dict(ws=24), vlf.VLF_ERR_ALIGN),
    (dict(mq=0), vlf.VLF_OK), (dict(n=0, tq=0, tk=0), vlf.VLF_OK),
])
def test_host_refusals(kw, status):
    assert _raw(**kw) == status


@pytest.mark.gpu
def test_python_refusals():
    x = make(30, [4], [50], 4, 2, 64, 64, BF, seed=1)
    for kw in (dict(k_prefix=x["k_prefix"].float()), dict(v_prefix=x["v_prefix"][:5].contiguous()),
               dict(k_prefix=x["k_prefix"][:, :1].contiguous()), dict(cu_seqlens_kv=cu_of([20, 30]).cuda()),
               dict(q=x["q"].transpose(0, 1)), dict(out=torch.empty(4, 4, 64, device="cuda")),
               dict(lse=torch.empty(4, 3, device="cuda")), dict(k_prefix=x["k_prefix"].cpu())):
        with pytest.raises(vlf.VlfError):
            vlf.vlf_attn_varlen_fwd_prefix(**dict(x, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype,flags", [(64, FP, 0), (128, FP, 0), (40, HF, 0), (128, BF, vlf.VLF_FLAG_FORCE_SIMT),
                                           (128, BF, 0), (64, HF, 0)])
def test_nan_logits_alone_in_their_tiles_reach_their_rows(d, dtype, flags):
    """A row of q that is NaN, a prefix of one NaN key, a window whose first key is NaN: the row and its
    log-sum-exp are NaN; rows that do not see it are what they were."""
    q_lens, kv_lens = [1, 3], [70, 33]
    for prefix in (1, 200):
        x = make(prefix, q_lens, kv_lens, 4, 2, d, d, dtype, seed=prefix)
        x["q"][2] = float("nan")
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, flags=flags)
        assert out[2].isnan().all() and lse[:, 2].isnan().all()
        assert out[[0, 1, 3]].isfinite().all() and lse[:, [0, 1, 3]].isfinite().all()
    x = make(1, q_lens, kv_lens, 4, 2, d, d, dtype, seed=1)
    x["k_prefix"][0] = float("nan")
    out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, flags=flags)
    assert out.isnan().all() and lse.isnan().all()
    # (the window's first key at many places of its tile, the last ones among them)
    for window in range(2, 70):
        x = make(26, [1], [70], 4, 2, d, d, dtype, seed=window)
        x["k"][70 - window] = float("nan")
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, window=window, flags=flags)
        assert out.isnan().all() and lse.isnan().all(), window
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, window=window - 1, flags=flags)
        assert out.isfinite().all() and lse.isfinite().all(), window


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,flags", [(BF, 0), (HF, 0), (BF, vlf.VLF_FLAG_FORCE_SIMT)])
@pytest.mark.parametrize("prefix,q_lens,kv_lens", [(200, [1, 1], [70, 33]), (5000, [1, 3], [40, 90]), (300, [80, 150], [190, 201]),
                                                   (0, [1, 2, 1], [70, 33, 500])])
def test_an_infinite_value_that_is_seen_gives_infinity(prefix, q_lens, kv_lens, dtype, flags):
    """Rows that all see the key: its column is infinite with the value's sign, the others what they were."""
    x = make(prefix, q_lens, kv_lens, 8, 2, 64, 64, dtype, seed=3)
    clean, clean_lse = vlf.vlf_attn_varlen_fwd_prefix(**x, causal=True, flags=flags)
    assert clean.isfinite().all()
    for name, key, rows in (("v_prefix", 17, slice(None)), ("v", sum(kv_lens[:-1]) + 3, slice(sum(q_lens[:-1]), None))):
        if name == "v_prefix" and not prefix:
            continue
        y = dict(x, **{name: x[name].clone()})
        y[name][key, 0, 5], y[name][key, 1, 63] = float("inf"), -float("inf")
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**y, causal=True, flags=flags)
        assert vlf.vlf_check_error() == 0
        want = clean.clone()
        want[rows, :4, 5], want[rows, 4:, 63] = float("inf"), -float("inf")
        assert torch.equal(out, want) and torch.equal(lse, clean_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, vlf.VLF_FLAG_FORCE_SIMT])
@pytest.mark.parametrize("prefix,q_lens,kv_lens", [(1000, [1, 1, 1], [17, 136, 255]), (300, [80, 150, 3], [190, 201, 30]), (0, [40], [77])])
def test_loose_bounds_on_the_lengths(prefix, q_lens, kv_lens, flags):
    """Longest lengths that are upper bounds alone, up to the largest that are taken."""
    x = make(prefix, q_lens, kv_lens, 8, 2, 64, 64, BF, seed=prefix)
    for mq, mk in ((max(q_lens), 4096), (max(q_lens), 16384), (1000, 100000), (2 ** 31 - 1, 2 ** 31 - 1)):
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(**dict(x, max_seqlen_q=mq, max_seqlen_kv=mk), causal=True, flags=flags)
        assert vlf.vlf_check_error() == 0
        verify(x, out, lse, True, 0)


@pytest.mark.parametrize("kw", [dict(tq=2 ** 31 - 1, mq=2 ** 31 - 1), dict(tk=2 ** 31 - 1, mk=2 ** 31 - 1),
                                dict(pl=2 ** 31 - 2 ** 16 - 8)])
def test_sizes_next_to_the_largest_int_are_refused(kw):
    assert _raw(**kw) == vlf.VLF_ERR_UNSUPPORTED
