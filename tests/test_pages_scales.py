"""Attention over pages whose scales lie far apart, with pages smaller than a key tile: a row's result depends on
the keys that it sees alone, in every kernel (max_seqlen_q only chooses one).

Tolerance, for each row of its own.  Bytes are exact and a key's scale multiplies its finished sum, so a logit is off
by what its own products are off by: q to 2^-18 of the row's largest element and fp32 sums, d_j = 2^-16 scale max|q|
sum_c |k_jc|; with D the largest d_j that the row sees, weights are off by 2^-11, 2^-20 and 2 D relatively:
    |error| <= u |out| + (2^-10 + 4 D) sum_j p_j |v_j| + n e max_j p_j s_j + half the least step of the output,
n keys seen, s_j the value scale of key j's page.  Weights times scales have a largest between 2^7 and 2^15 and are held in
fp16, steps of 2^-24 and more (many rows), or in e5m2, steps of 2^-16 and more (few rows): off by half of that, over
the largest 2^-32 and 2^-24, and a byte is 448 at most, so e = 2^-23 and 2^-15.  The lse is off by D and 2^-18 of
itself."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 2.0 ** -133, FP: 2.0 ** -24, F32: 2.0 ** -149}
SIMT = vlf.VLF_FLAG_FORCE_SIMT


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().cpu().double().numpy()


def problem(q_lens, kv_lens, page, hq, hkv, d, dtype, k_exp, v_exp, seed=0):
    """Page i of a sequence has the scales 2^k_exp[i % n] and 2^v_exp[i % n], times 1 or 2 by head."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-x // page) for x in kv_lens]
    pages, most = sum(counts) + 1, max(counts)
    order = torch.randperm(pages, generator=g).tolist()
    c = dict(q=torch.randn(sum(q_lens), hq, d, generator=g).to(dtype).cuda(), rows=[], lens=kv_lens, page=page)
    for name in ("k", "v"):
        x = torch.randn(pages, hkv, page, d, generator=g).clamp(-4, 4)
        c[name + "_pages"] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        c[name + "_scale"] = torch.full((pages, hkv), float("nan"), device="cuda")
    at = 0
    for n in counts:
        c["rows"].append(order[at:at + n] + [-1] * (most - n))
        for i, p in enumerate(order[at:at + n]):
            for name, e in (("k", k_exp), ("v", v_exp)):
                c[name + "_scale"][p] = torch.exp2(torch.tensor([float(e[i % len(e)] + h % 2) for h in range(hkv)]))
        at += n
    c["table"], c["kv"] = ints(c["rows"]), ints(kv_lens)
    c["cu"] = [0] + [int(x) for x in np.cumsum(q_lens)]
    c["cu_q"], c["max_q"] = ints(c["cu"]), max(q_lens)
    return c


def call(c, max_q=None, **kw):
    return vlf.vlf_attn_varlen_fwd_pages(c["q"], c["k_pages"], c["v_pages"], c["k_scale"], c["v_scale"], c["table"], c["cu_q"],
                                         c["kv"], max_q or c["max_q"], **kw)


def definition(c, causal, window=0):
    """Per row: out, lse, sum_j p_j |v_j|, n max_j p_j s_j, D."""
    q = np64(c["q"])
    hq, d = q.shape[1:]
    kp, vp, ks, vs = (c[x].cpu().numpy() for x in ("k_pages", "v_pages", "k_scale", "v_scale"))
    hkv, page = kp.shape[1:3]
    scale = d ** -0.5
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, top, far = (np.zeros(q.shape[:2]) for _ in range(3))
    for s, n in enumerate(c["lens"]):
        k, v = ref.keys_of(kp, ks, c["rows"][s], n), ref.keys_of(vp, vs, c["rows"][s], n)
        sv = np.array([vs[c["rows"][s][j // page]] for j in range(n)], np.float64)
        a, b = c["cu"][s], c["cu"][s + 1]
        for i in range(a, b):
            at = i - a + n - (b - a)
            lo, hi = max(0, at - window + 1) if window else 0, at + 1 if causal else n
            for h in range(hq):
                g = h // (hq // hkv)
                x = scale * (k[lo:hi, g] @ q[i, h])
                p = np.exp(x - x.max())
                lse[i, h] = x.max() + np.log(p.sum())
                p /= p.sum()
                out[i, h], size[i, h] = p @ v[lo:hi, g], p @ np.abs(v[lo:hi, g])
                top[i, h] = (hi - lo) * (p * sv[lo:hi, g]).max()
                far[i, h] = 2.0 ** -16 * scale * np.abs(q[i, h]).max() * np.abs(k[lo:hi, g]).sum(axis=1).max()
    return out, lse, size, top, far


MANY, FEW = 2.0 ** -23, 2.0 ** -15


def check(got, c, want, e=MANY):
    (out, lse), (O, L, size, top, far) = got, want
    tol = UNIT[out.dtype] * np.abs(O) + (2.0 ** -10 + 4 * far[..., None]) * size + e * top[..., None] + LEAST[out.dtype] / 2
    off = np.abs(np64(out) - O) / tol
    assert (off <= 1).all(), (off.max(), np.argwhere(~(off <= 1))[:5])
    assert (np.abs(np64(lse).T - L) <= far + 2.0 ** -18 * (1 + np.abs(L))).all()
    assert vlf.vlf_check_error() == 0


# exponents of the pages in turn: keys, values (the first rows of a prompt see the first page alone)
SPREADS = [([-60, -6, -20], [-60, -3, -30, 0]), ([-6], [-40, 20]), ([-30, -6], [-6]), ([-24, -6, -8], [-10, -2, 3])]


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("k_exp,v_exp", SPREADS)
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, BF)])
def test_a_prompt_row_sees_only_its_own_pages(page, k_exp, v_exp, d, dtype):
    c = problem([150, 70], [150, 200], page, 4, 2, d, dtype, k_exp, v_exp, seed=page)
    want = definition(c, True)
    check(call(c, causal=True), c, want)
    check(call(c, causal=True, flags=SIMT), c, want)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("d", [128, 64])
def test_fp16_rows_and_windows(page, d):
    c = problem([150, 40], [150, 170], page, 4, 2, d, FP, [-26, -6, -8], [-20, 4, -8], seed=d)
    check(call(c, causal=True), c, definition(c, True))
    check(call(c, causal=True, window=17), c, definition(c, True, 17))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("rows", [1, 8])
def test_a_loose_bound_chooses_another_kernel_not_another_result(page, rows, d):
    """The same rows by the kernel for few and by the one for many, with every spread."""
    for k_exp, v_exp in SPREADS:
        c = problem([rows, rows], [300, 90], page, 4, 2, d, BF, k_exp, v_exp, seed=rows)
        want = definition(c, True)
        check(call(c, causal=True), c, want, FEW)
        check(call(c, causal=True, max_q=5000), c, want)
        check(call(c, causal=True, window=20, max_q=5000), c, definition(c, True, 20))
