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


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("q_lens,flags", KERNELS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_query_that_is_not_finite_makes_its_row_nan(page, q_lens, flags, dtype):
    """Whatever the signs of its products are; a row that sees no key is 0 all the same, and no other row changes."""
    c = problem(q_lens, [20, 700], page, 4, 2, 128, 128, dtype, seed=page)
    for name in ("k_pages",):  # (keys of one sign: an infinite query's logits are all infinite, and of one sign)
        c[name] = torch.where(c[name] & 127 == 127, c[name], c[name] & 127)
    want = call(c, causal=True, flags=flags)
    sees = [i >= q_lens[0] - 20 for i in range(q_lens[0])] + [True] * q_lens[1]
    for x in (INF, -INF, NAN):
        for i, h, col in ((0, 0, 0), (q_lens[0] - 1, 1, 77), (q_lens[0], 3, 127), (sum(q_lens) - 1, 2, 5)):
            d = dict(c, q=c["q"].clone())
            d["q"][i, h, col] = x
            out, lse = call(d, causal=True, flags=flags)
            if sees[i]:
                assert out[i, h].isnan().all() and lse[h, i].isnan()
            else:
                assert not out[i, h].any() and lse[h, i] == -INF
            out, lse = out.clone(), lse.clone()
            out[i, h], lse[h, i] = want[0][i, h], want[1][h, i]
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("q_lens,flags", KERNELS)
def test_a_nan_in_the_cache_reaches_the_rows_that_see_it(page, q_lens, flags):
    """A key's: rows in front of it keep their bits, the others are NaN.  A value's: its column, and the lse is what it was.
    Rows of other kv heads and of the other sequence never change."""
    c = problem(q_lens, [300, 200], page, 4, 2, 128, 128, BF, seed=2)
    a, b = q_lens
    want = call(c, causal=True, flags=flags)
    pool = c["k_pages"].clone(), c["v_pages"].clone()
    j = 200 - b + b // 2  # seen from row b // 2 on
    c["k_pages"][c["rows"][1][j // page], 0, j % page, 3] = 127
    out, lse = call(c, causal=True, flags=flags)
    at = a + b // 2
    assert out[at:, :2].isnan().all() and lse[:2, at:].isnan().all()
    assert torch.equal(out[:at], want[0][:at]) and torch.equal(lse[:, :at], want[1][:, :at])
    assert torch.equal(out[:, 2:], want[0][:, 2:]) and torch.equal(lse[2:], want[1][2:])
    c["k_pages"].copy_(pool[0])
    c["v_pages"][c["rows"][1][j // page], 1, j % page, 3] = 255
    out, lse = call(c, causal=True, flags=flags)
    assert out[at:, 2:, 3].isnan().all() and torch.equal(lse, want[1])
    rest = torch.tensor([x for x in range(128) if x != 3], device="cuda")
    assert torch.equal(out[:, :, rest], want[0][:, :, rest]) and torch.equal(out[:a], want[0][:a])
    assert torch.equal(out[:, :2], want[0][:, :2]) and vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("change,status", [(dict(length=2000), -6), (dict(length=-1), -6), (dict(cu=[0, 90, 40]), -6), (dict(cu=[0, 40, 500]), -6)])
def test_bad_lengths_with_many_rows_are_recorded(change, status, page):
    c = problem([40, 70], [300, 200], page, 4, 2, 128, 128, BF, seed=2)
    want = call(c, causal=True)
    if "length" in change:
        c["kv"][1] = change["length"]
    else:
        c["cu_q"] = torch.tensor(change["cu"], dtype=torch.int32, device="cuda")
    out, _ = call(c, causal=True)
    assert vlf.vlf_check_error() == status
    if change != dict(cu=[0, 90, 40]):
        assert torch.equal(out[:40], want[0][:40])
    assert vlf.vlf_check_error() == 0
