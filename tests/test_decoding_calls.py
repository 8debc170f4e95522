"""How the decoding entry points are called: streams, batches without sequences, alignment, sizes and
bounds far from the usual ones, and what the package does without the native side of its calls."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf

BF = torch.bfloat16


def cu_of(lens, device="cuda"):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=device)


def some_calls(max_kv=50):
    """A call of each entry point, as a function of further arguments; the inputs are ready when it returns."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    qkv, pos = r(9, 12, 64), torch.arange(9, dtype=torch.int32, device="cuda")
    f = torch.rand(32, generator=g).cuda()
    q, k, kp, vp, kc, vc = r(5, 8, 64), r(90, 2, 64), r(3000, 2, 64), r(3000, 2, 64), r(90, 2, 64), r(90, 2, 64)
    cu_q, cu_kv, w = cu_of([1, 4]), cu_of([40, 50]), torch.rand(2, 90, generator=g).cuda()
    lse = torch.full((8, 5), 3.0, device="cuda")
    long_q, long_k, long_lse = r(700, 8, 64), r(700, 1, 64), torch.full((8, 700), 6.0, device="cuda")
    one = cu_of([700])
    torch.cuda.synchronize()
    return dict(
        rope=lambda **kw: vlf.vlf_rope(qkv[:, :8], qkv[:, 8:10], pos, f, **kw),
        prefix=lambda cu=cu_kv, mk=max_kv, **kw: vlf.vlf_attn_varlen_fwd_prefix(q, kp, vp, kc, vc, cu_q, cu, 4, mk, causal=True, **kw),
        weights=lambda cu=cu_kv, mk=max_kv, **kw: vlf.vlf_attn_key_weights(q, k, lse, cu_q, cu, 4, mk, causal=True, prev=w, **kw),
        # (in parts: a workspace)
        prompt=lambda **kw: vlf.vlf_attn_key_weights(long_q, long_k, long_lse, one, one, 700, 700, causal=True, **kw),
        evict=lambda cu=cu_kv, mk=max_kv, **kw: vlf.vlf_cache_evict(kc, vc, w, cu, 20, 2, 3, max_seqlen_kv=mk, total_out=40, **kw))


def as_list(x):
    return [x] if torch.is_tensor(x) else list(x)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rope", "prefix", "weights", "prompt", "evict"])
def test_outputs_on_another_stream_are_allocated_in_its_order(name):
    """Blocks that are free on the current stream, but still to be written by what is queued there, are
    not what a call on another stream writes to."""
    call = some_calls()[name]
    want = as_list(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        sizes = [t.numel() * t.element_size() for t in want] + [1 << 20, 1 << 18]
        held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda._sleep(40_000_000)
        for t in held:
            t.fill_(1)
        del held, t
        got = as_list(call(stream=side))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["prefix", "weights", "evict"])
def test_lengths_left_to_the_call_are_read_in_its_stream(name):
    call = some_calls()[name]
    want = as_list(call())
    cu, late = cu_of([40, 50]), cu_of([0, 0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        late.copy_(cu)
    got = as_list(call(cu=late, mk=None, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_eviction_of_an_empty_batch():
    """No sequences: cu_seqlens [0] out, whichever way the call goes and whoever holds the output."""
    k, w, cu = torch.empty(0, 2, 64, device="cuda", dtype=BF), torch.empty(2, 0, device="cuda"), cu_of([])
    for kw in (dict(total_out=0, max_seqlen_kv=0), dict(), dict(stream=torch.cuda.current_stream()),
               dict(stream=torch.cuda.Stream()), dict(cu_out=torch.full((1,), 9, dtype=torch.int32, device="cuda"))):
        # (what a fresh output of this size would hold)
        junk = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        del junk
        ko, vo, wo, io, co = vlf.vlf_cache_evict(k, k, w, cu, 4, **kw)
        torch.cuda.synchronize()
        assert co.tolist() == [0] and ko.shape == (0, 2, 64) and wo.shape == io.shape == (2, 0)
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,why", [(60, "lengths"), (1500, "lengths"), (60, "rows"), (1500, "rows")])
def test_no_rows_are_copied_behind_a_refused_sequence(n, why):
    """In one launch (60 keys) and in two: of four sequences the second is refused; its rows and the next
    one's stay as they were, the others are copied."""
    h, budget = 2, 20
    lens = [n, n + 40 if why == "lengths" else n, n, n]
    k = torch.randn(sum(lens), h, 64, device="cuda").to(BF)
    w, cu = torch.rand(h, sum(lens), device="cuda"), cu_of(lens)
    rows = 4 * budget if why == "lengths" else budget + 5  # (the second one and those behind it do not fit)
    out = torch.full((rows, h, 64), 7.0, device="cuda", dtype=BF)
    got = torch.full((h, rows), 7.0, device="cuda")
    ko, _, wo, io, co = vlf.vlf_cache_evict(k, k, w, cu, budget, max_seqlen_kv=n, total_out=rows, k_out=out, weights_out=got)
    assert vlf.vlf_check_error() == vlf.VLF_ERR_BAD_SEQLENS
    if why == "lengths":
        assert co.tolist() == [0, budget, -1, 3 * budget, 4 * budget]
        copied = [0, 3]
        assert (ko[budget:3 * budget] == 7).all() and (wo[:, budget:3 * budget] == 7).all()
    else:
        assert co.tolist() == [0, budget, -1, -1, -1]
        copied = [0]
        assert (ko[budget:] == 7).all() and (wo[:, budget:] == 7).all()
    for s in copied:
        for g in range(h):
            at = int(cu[s]) + io[g, s * budget:(s + 1) * budget].long()
            assert torch.equal(ko[s * budget:(s + 1) * budget, g], k[at, g])
            assert torch.equal(wo[g, s * budget:(s + 1) * budget], w[g, at])


@pytest.mark.gpu
def test_positions_and_frequencies_may_be_slices():
    """A chunk of a prompt's positions, a run of the frequencies: from any element on, on any route."""
    g = torch.Generator().manual_seed(2)
    pos = torch.randint(0, 10 ** 6, (40,), generator=g, dtype=torch.int32).cuda()
    freq = torch.rand(70, generator=g).cuda()
    q, k = (torch.randn(9, h, 64, generator=g).to(BF).cuda() for h in (4, 2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for a in range(5):
        for b in range(5):
            p, f = pos[a:a + 9], freq[b:b + 32]
            want = vlf.vlf_rope(q, k, p.clone(), f.clone())
            got = [vlf.vlf_rope(q, k, p, f), vlf.rotary_embedding(q, k, p, f), vlf.vlf_rope(q, k, p, f, stream=side)]
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for pair in got for x, y in zip(want, pair))
    two = pos[1:19].view(2, 9)
    want = vlf.vlf_rope(q, k, two.clone(), freq[:32], [20, 12])
    assert all(torch.equal(x, y) for x, y in zip(want, vlf.vlf_rope(q, k, two, freq[:32], [20, 12])))


def test_the_package_works_without_its_native_calls(tmp_path):
    """libvlf.so is enough: the import warns, and every call goes through the Python functions."""
    import os
    import subprocess
    import sys
    src = os.path.dirname(vlf.LIB_PATH)
    dst = tmp_path / os.path.basename(src)
    dst.mkdir()
    for name in ("__init__.py", "functional.py", "flops.py", "libvlf.so"):
        os.symlink(os.path.join(src, name), dst / name)
    code = """
import warnings
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    import variable_length_flash_gb300 as vlf
assert any("native calls" in str(x.message) for x in w), w
assert vlf.__file__.startswith(%r), vlf.__file__
assert vlf._calls.rope(1, 2) is None
import torch
try:
    vlf.vlf_rope(torch.zeros(4, 2, 8), None, torch.zeros(4, dtype=torch.int32), torch.zeros(4))
except vlf.VlfError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_native_calls_of_another_torch_are_not_bound(monkeypatch):
    import types
    bound = []
    for other in (types.SimpleNamespace(TORCH="1.2.3+other", bind=lambda *a: bound.append(a)),
                  types.SimpleNamespace(bind=lambda *a: bound.append(a))):
        monkeypatch.setattr(vlf, "_calls", other)
        with pytest.warns(UserWarning, match="native calls"):
            got = vlf._load_calls(vlf._lib)
        assert not bound and got.evict(1, 2, 3) is None


def test_native_calls_of_another_torch_are_built_anew(monkeypatch, tmp_path):
    from variable_length_flash_gb300 import _build
    stamp, lib = tmp_path / "calls.for", tmp_path / "_calls.so"
    monkeypatch.setattr(_build, "CALLS_FOR", str(stamp))
    monkeypatch.setattr(_build, "CALLS", str(lib))
    assert _build._calls_stale()
    lib.write_text("")
    assert _build._calls_stale()
    stamp.write_text(_build._calls_for())
    assert not _build._calls_stale()
    stamp.write_text("1.2.3 .so")
    assert _build._calls_stale()


@pytest.mark.gpu
def test_results_do_not_depend_on_the_native_calls(monkeypatch):
    calls = some_calls()
    want = {n: as_list(c()) for n, c in calls.items()}
    monkeypatch.setattr(vlf, "_calls", vlf._NoCalls())
    for n, c in calls.items():
        assert all(torch.equal(a, b) for a, b in zip(want[n], as_list(c()))), n


class _Huge:
    """What the Python functions ask of a CUDA tensor, without its memory."""
    is_cuda, requires_grad = True, False

    def __init__(self, *shape, dtype=BF):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:], dtype=np.int64)) for i in range(len(self.shape)))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape, dtype=np.int64))

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 16


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5])
def test_sizes_that_no_c_int_holds_are_refused(monkeypatch, n):
    """2^32 + 5 tokens are not 5."""
    monkeypatch.setattr(vlf, "_elsewhere", lambda t: False)
    i32, f32, cu = torch.int32, torch.float32, _Huge(3, dtype=torch.int32)
    t, few, w = _Huge(n, 2, 8), _Huge(4, 2, 8), _Huge(2, n, dtype=f32)
    calls = [lambda: vlf.vlf_rope(t, None, _Huge(n, dtype=i32), _Huge(4, dtype=f32)),
             lambda: vlf.vlf_rope(t, t, _Huge(n, dtype=i32), _Huge(4, dtype=f32)),
             lambda: vlf.vlf_rope(_Huge(4, n, 8), None, _Huge(4, dtype=i32), _Huge(4, dtype=f32)),
             lambda: vlf.vlf_attn_varlen_fwd_prefix(t, few, few, few, few, cu, cu, 1, 4),
             lambda: vlf.vlf_attn_varlen_fwd_prefix(few, t, t, few, few, cu, cu, 1, 4),
             lambda: vlf.vlf_attn_varlen_fwd_prefix(few, few, few, t, t, cu, cu, 1, 4),
             lambda: vlf.vlf_attn_key_weights(t, few, w, cu, cu, 1, 4),
             lambda: vlf.vlf_attn_key_weights(few, t, _Huge(2, 4, dtype=f32), cu, cu, 1, 4),
             lambda: vlf.vlf_cache_evict(t, t, w, cu, 4, max_seqlen_kv=4, total_out=4)]
    for call in calls:
        with pytest.raises(vlf.VlfError, match="out of range"):
            call()


def test_an_output_without_its_input_is_refused(monkeypatch):
    monkeypatch.setattr(vlf, "_elsewhere", lambda t: False)
    q, out = _Huge(4, 2, 8), _Huge(4, 2, 8)
    with pytest.raises(vlf.VlfError, match="k_out without k"):
        vlf.vlf_rope(q, None, _Huge(4, dtype=torch.int32), _Huge(4, dtype=torch.float32), q_out=out, k_out=_Huge(4, 1, 8))
