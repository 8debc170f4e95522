"""What attention over pages does with what should not be there, in each of its three kernels (few rows, many rows,
FMA): pages outside the pool, keys, values and queries that are not finite.

A page outside the pool is recorded and its keys are passed over: a row's weights are those of its other keys, and a row
that has no other is 0 with an lse of minus infinity.  Bounds as in test_pages_attention.py, which derives them."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import paging as ref
from tests.test_pages_attention import BF, FP, SIMT, call, np64, problem

UNIT = {BF: 2.0 ** -8, FP: 2.0 ** -11, torch.float32: 2.0 ** -24}
INF, NAN = float("inf"), float("nan")
# (rows of the two sequences, flags): with groups of two heads the kernels for few and for many rows, and FMA
KERNELS = [([1, 3], 0), ([40, 70], 0), ([1, 3], SIMT), ([40, 70], SIMT)]


def holds(got, c, causal=True, window=0):
    cache = [c[x].cpu().numpy() for x in ("k_pages", "v_pages", "k_scale", "v_scale")]
    rows = c["table"].tolist()
    O, L, size, reach = ref.pages_attention(np64(c["q"]), cache, rows, c["cu"], c["lens"], c["q"].shape[2] ** -0.5, causal, window)
    out, lse = (np64(x) for x in got)
    tol = UNIT[got[0].dtype] * np.abs(O) + (2.0 ** -10 + 4 * (2.0 ** -16 * reach).T[..., None]) * size
    tol = tol + 2.0 ** -24 * max(c["lens"]) * 32 + 1e-30
    assert (np.abs(out - O) <= tol).all(), np.argwhere(~(np.abs(out - O) <= tol))[:4]
    live = L > -np.inf
    assert np.array_equal(lse > -np.inf, live) and not np.isnan(lse).any()
    L0, lse0 = np.where(live, L, 0), np.where(live, lse, 0)
    assert (np.abs(lse0 - L0) <= 2.0 ** -16 * reach + 2.0 ** -18 * (1 + np.abs(L0))).all()
    assert not out[~live.T].any()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("q_lens,flags", KERNELS)
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
def test_a_page_outside_the_pool_is_passed_over(page, q_lens, flags, d, dtype):
    c = problem(q_lens, [300, 700], page, 4, 2, d, d, dtype, seed=page)
    want = call(c, causal=True, flags=flags)
    n = c["k_pages"].shape[0]
    for bad in (-1, n, 2 ** 31 - 1, -2 ** 31):
        c["table"][1, 1] = bad
        got = call(c, causal=True, flags=flags)
        assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_PAGES
        assert torch.equal(got[0][:q_lens[0]], want[0][:q_lens[0]])  # the other sequence is what it was
        assert torch.equal(got[1][:, :q_lens[0]], want[1][:, :q_lens[0]])
        holds(got, c)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("q_lens,flags", KERNELS)
def test_rows_that_have_no_other_page(page, q_lens, flags):
    """A sequence without a page of the pool, one with the last page alone, and a whole tile of bad pages between others."""
    c = problem(q_lens, [300, 700], page, 4, 2, 128, 128, BF, seed=page)
    good = c["table"].clone()
    c["table"][0] = -1
    holds(call(c, causal=True, flags=flags), c)
    holds(call(c, causal=True, window=90, flags=flags), c, window=90)
    c["table"][1, :(700 - 1) // page] = 2 ** 30
    holds(call(c, causal=True, flags=flags), c)
    c["table"].copy_(good)
    c["table"][1, 256 // page:512 // page] = -1
    holds(call(c, causal=True, flags=flags), c)
    holds(call(c, flags=flags), c, causal=False)
    assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_PAGES
    c["table"].copy_(good)
    holds(call(c, causal=True, flags=flags), c)
    assert vlf.vlf_check_error() == 0
