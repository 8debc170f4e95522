"""The decoding operators together, as a serving loop runs them: rotary positions of the step's q and k,
attention over a shared prefix and each sequence's own cache, the weights the cached keys receive, and
the cache cut to its budget; and rotary positions in front of attention in training.  Each stage is
checked against its fp64 definition on the inputs that the stage before it produced."""
import numpy as np
import pytest
import torch

import variable_length_flash_gb300 as vlf
from oracle import decoding as ref

BF = torch.bfloat16
U = 2.0 ** -8


def np64(t):
    return t.detach().cpu().double().numpy()


def append(old, new, cu_old, cu_new):
    """Packed rows: each sequence's old ones, then its new ones."""
    parts = []
    for s in range(len(cu_old) - 1):
        parts += [old[cu_old[s]:cu_old[s + 1]], new[cu_new[s]:cu_new[s + 1]]]
    return torch.cat(parts)


@pytest.mark.gpu
@pytest.mark.parametrize("axes,d,hq,hkv", [(1, 128, 8, 2), (3, 64, 4, 4)])
def test_a_serving_loop(axes, d, hq, hkv):
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    n, P, budget, sink, recent = 3, 300, 40, 2, 8
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    sec = [d // 2] if axes == 1 else [d // 2 - 2 * (d // 6), d // 6, d // 6]
    kp, vp = r(P, hkv, d), r(P, hkv, d)
    lens = [0] * n                  # own keys in the cache
    seen = [P] * n                  # tokens so far: positions go on although keys are evicted
    k_cache, v_cache = r(0, hkv, d), r(0, hkv, d)
    weights = torch.zeros(hkv, 0, device="cuda")
    for new in ([30, 7, 1], [1, 1, 1], [25, 1, 60], [1, 1, 1]):
        total = sum(new)
        qkv = r(total, hq + 2 * hkv, d)
        pos = torch.tensor([seen[s] + i for s in range(n) for i in range(new[s])], dtype=torch.int32)
        pos = torch.stack([pos * (a + 1) for a in range(axes)]).cuda()
        q, k = vlf.vlf_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, f, sec)
        for y, x in ((q, qkv[:, :hq]), (k, qkv[:, hq:hq + hkv])):
            want = ref.rope(np64(x), pos.cpu().numpy(), f.cpu().numpy(), sec, d, False)
            top = np.abs(np64(x)).max()
            assert (np.abs(np64(y) - want) <= U * np.abs(want) + 2 * top * 2.0 ** -20).all()
        cu_q = [0] + list(np.cumsum(new))
        cu_c = [0] + list(np.cumsum(lens))
        k_cache = append(k_cache, k, cu_c, cu_q)
        v_cache = append(v_cache, qkv[:, hq + hkv:].contiguous(), cu_c, cu_q)
        weights = append(weights.t(), torch.zeros(total, hkv, device="cuda"), cu_c, cu_q).t().contiguous()
        lens = [a + b for a, b in zip(lens, new)]
        seen = [a + b for a, b in zip(seen, new)]
        cu_kv = [0] + list(np.cumsum(lens))
        t_q, t_kv = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_kv))
        out, lse = vlf.vlf_attn_varlen_fwd_prefix(q, kp, vp, k_cache, v_cache, t_q, t_kv, max(new), max(lens), causal=True)
        args = (np64(q), np64(kp), np64(vp), np64(k_cache), np64(v_cache), cu_q, cu_kv, d ** -0.5, True, 0)
        O, L = ref.prefix_forward(*args)
        Oabs, _ = ref.prefix_forward(args[0], args[1], np.abs(args[2]), args[3], np.abs(args[4]), *args[5:])
        # u for the output, 2 u for the rounded weights; logits of these sizes are off by less than 2^-12
        assert (np.abs(np64(out) - O) <= U * np.abs(O) + (2 * U + 2.0 ** -11) * Oabs).all()
        assert np.abs(np64(lse) - L).max() <= 2.0 ** -12
        prev = weights
        weights = vlf.vlf_attn_key_weights(q, k_cache, lse, t_q, t_kv, max(new), max(lens), causal=True, prev=prev)
        # (the definition counts the end-aligned rows over the own keys: the rows' own positions)
        W = ref.key_weights(np64(q), np64(k_cache), np64(lse), cu_q, cu_kv, d ** -0.5, True, 0, prev=np64(prev))
        assert (np.abs(np64(weights) - W) <= 2.0 ** -11 * W + 1e-30).all()
        kept, cu_out = ref.evict(weights.cpu().numpy(), cu_kv, budget, sink, recent)
        ko, vo, wo, index, co = vlf.vlf_cache_evict(k_cache, v_cache, weights, t_kv, budget, sink, recent,
                                                    max_seqlen_kv=max(lens), total_out=cu_out[-1])
        assert co.tolist() == cu_out
        for h in range(hkv):
            rows = torch.tensor([cu_kv[s] + j for s in range(n) for j in kept[h][s]], device="cuda")
            assert index[h].tolist() == [j for s in range(n) for j in kept[h][s]]
            assert torch.equal(ko[:, h], k_cache[rows, h]) and torch.equal(vo[:, h], v_cache[rows, h])
            assert torch.equal(wo[h], weights[h, rows])
        k_cache, v_cache, weights, lens = ko, vo, wo, [b - a for a, b in zip(cu_out[:-1], cu_out[1:])]
        assert vlf.vlf_check_error() == 0


def test_native_calls_leave_what_is_not_theirs():
    """The native side of the calls returns None for anything but plain CUDA tensors and plain numbers,
    and counts arguments; the Python functions then say what was wrong."""
    x, n = torch.zeros(4, 2, 8), torch.zeros(3, dtype=torch.int32)
    calls = vlf._calls
    assert calls.rope(x, x, n, torch.zeros(4), None, False, False) is None
    assert calls.rope(None, 3, "x", [], {}, 1, 2) is None and calls.rope(x) is None and calls.rope() is None
    assert calls.prefix(x, x, x, x, x, n, n, 1, 1, None, True, 0, 0) is None
    assert calls.weights(x, x, x, n, n, 1, 1, None, True, 0, None, 0) is None
    assert calls.evict(x, x, x, n, 2 ** 70, 0, 0, 4, 4) is None
    for f, args in ((vlf.vlf_rope, (x, x, n, torch.zeros(4))),
                    (vlf.vlf_attn_varlen_fwd_prefix, (x, x, x, x, x, n, n, 1, 1)),
                    (vlf.vlf_attn_key_weights, (x, x, x, n, n, 1, 1)), (vlf.vlf_cache_evict, (x, x, x, n, 4))):
        with pytest.raises(vlf.VlfError, match="CUDA"):
            f(*args)


@pytest.mark.gpu
def test_captured_steps_replay_like_eager_ones():
    """A whole step in a graph, two such graphs of different batches replayed in turn on two streams, with
    eager calls between: every replay gives the eager step's results to the bit."""
    hq, hkv, d, P = 8, 2, 64, 700

    def batch(lens, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
        n, f = len(lens), (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
        cu_q = torch.arange(n + 1, dtype=torch.int32).cuda()
        cu_kv = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
        qkv, pos = r(n, hq + 2 * hkv, d), torch.randint(0, 10 ** 6, (n,), generator=g, dtype=torch.int32).cuda()
        kp, vp, k, v, w = r(P, hkv, d), r(P, hkv, d), r(sum(lens), hkv, d), r(sum(lens), hkv, d), \
            torch.rand(hkv, sum(lens), generator=g).cuda()
        top, rows = max(lens), sum(min(x, 100) for x in lens)

        def step():
            q, _ = vlf.vlf_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, f)
            out, lse = vlf.vlf_attn_varlen_fwd_prefix(q, kp, vp, k, v, cu_q, cu_kv, 1, top, causal=True)
            got = vlf.vlf_attn_key_weights(q, k, lse, cu_q, cu_kv, 1, top, causal=True, prev=w)
            return (out, lse, got) + tuple(vlf.vlf_cache_evict(k, v, got, cu_kv, 100, 4, 16, top, rows))
        return step

    steps = [batch([300, 90, 1200], 1), batch([9000], 2)]
    want = [s() for s in steps]
    graphs, held = [], []
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(s())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, outs in zip(graphs, streams, held):
            with torch.cuda.stream(stream):
                for t in outs:
                    t.zero_()
                graph.replay()
        again = [s() for s in steps]
        torch.cuda.synchronize()
        for a, b, c in zip(want, again, held):
            assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_calls_go_to_the_device_of_their_tensors(monkeypatch):
    """Where another device is the current one, the tensors' own becomes it for the call."""
    t, h, d = 6, 2, 64
    r = lambda *s: torch.randn(*s, device="cuda").to(BF)  # noqa: E731
    q, k, v, st = r(t, h, d), r(t, h, d), r(t, h, d), torch.cuda.current_stream()
    cu = torch.tensor([0, 2, t], dtype=torch.int32, device="cuda")
    w, f = torch.rand(h, t, device="cuda"), torch.rand(d // 2, device="cuda")
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    entered, real = [], torch.cuda.device

    class Entered(real):
        def __enter__(self):
            entered.append(self.idx)
            monkeypatch.setattr(torch.cuda, "current_device", lambda: self.idx)
            return super().__enter__()

    monkeypatch.setattr(torch.cuda, "device", Entered)
    for call in (lambda: vlf.vlf_rope(q, k, pos, f, stream=st),
                 lambda: vlf.vlf_attn_varlen_fwd_prefix(q, k, v, k, v, cu, cu, 4, 4, stream=st),
                 lambda: vlf.vlf_attn_key_weights(q, k, w, cu, cu, 4, 4, stream=st),
                 lambda: vlf.vlf_cache_evict(k, v, w, cu, 2, max_seqlen_kv=4, total_out=4, stream=st)):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: q.get_device() + 1)
        call()
    monkeypatch.undo()
    assert entered == 4 * [q.get_device()]
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_native_and_python_calls_agree():
    """The same call through the native side and through Python (which a stream of the caller's takes)."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    here = torch.cuda.current_stream()
    qkv, pos, f = r(9, 12, 64), t(*range(9)), torch.rand(32, generator=g).cuda()
    q, k, kp, vp, kc, vc = r(5, 8, 64), r(90, 2, 64), r(700, 2, 64), r(700, 2, 64), r(90, 2, 64), r(90, 2, 64)
    cu_q, cu_kv, w = t(0, 1, 5), t(0, 40, 90), torch.rand(2, 90, generator=g).cuda()
    lse = torch.full((8, 5), 3.0, device="cuda")
    calls = [(vlf.vlf_rope, (qkv[:, :8], qkv[:, 8:10], pos, f), dict(sections=[32], interleaved=True)),
             (vlf.vlf_attn_varlen_fwd_prefix, (q, kp, vp, kc, vc, cu_q, cu_kv, 4, 50), dict(causal=True, window=600, scale=0.2)),
             (vlf.vlf_attn_key_weights, (q, k, lse, cu_q, cu_kv, 4, 50), dict(causal=True, prev=w)),
             (vlf.vlf_cache_evict, (kc, vc, w, cu_kv, 20), dict(sink=2, recent=3, max_seqlen_kv=50, total_out=40))]
    for fn, args, kw in calls:
        native, python = fn(*args, **kw), fn(*args, **kw, stream=here)
        native, python = ([x] if torch.is_tensor(x) else list(x) for x in (native, python))
        assert len(native) == len(python)
        for a, b in zip(native, python):
            assert a.shape == b.shape and a.dtype == b.dtype and a.is_contiguous() and torch.equal(a, b)
    # refused by the library: the same error either way
    for kw in (dict(), dict(stream=here)):
        with pytest.raises(vlf.VlfError):
            vlf.vlf_cache_evict(kc, vc, w, cu_kv, 4, sink=3, recent=3, max_seqlen_kv=50, total_out=8, **kw)
        with pytest.raises(vlf.VlfError):
            vlf.vlf_rope(qkv[:, 1:8], qkv[:, 8:10], pos, torch.zeros(40, device="cuda"), **kw)
    assert vlf.vlf_check_error() == 0


@pytest.mark.gpu
def test_prefix_keys_receive_the_rest():
    """Own and prefix keys' weights from the same lse: each (row, head)'s sum to 1."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    q, kp, vp, k, v = r(5, 8, 64), r(700, 2, 64), r(700, 2, 64), r(90, 2, 64), r(90, 2, 64)
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu_q, cu_kv = t(0, 1, 5), t(0, 40, 90)
    _, lse = vlf.vlf_attn_varlen_fwd_prefix(q, kp, vp, k, v, cu_q, cu_kv, 4, 50, causal=True)
    own = vlf.vlf_attn_key_weights(q, k, lse, cu_q, cu_kv, 4, 50, causal=True)
    pre = vlf.vlf_attn_key_weights(q, kp, lse, t(0, 5), t(0, 700), 5, 700)
    # 20 (row, head) pairs per kv head; sums of 790 weights, each off by less than 2^-13 of itself
    assert (own.double().sum(1) + pre.double().sum(1) - 20).abs().max() <= 20 * 2.0 ** -12


@pytest.mark.gpu
def test_rotary_positions_in_front_of_attention_train():
    """Gradients through rotary_embedding and varlen_attention against fp64 autograd on the same inputs
    (fp32 tensors: every stage is off by a few 2^-20 of what it sums)."""
    g = torch.Generator().manual_seed(9)
    lens = [20, 45]
    total, hq, hkv, d = sum(lens), 4, 2, 32
    cu = torch.tensor([0, 20, 65], dtype=torch.int32, device="cuda")
    qkv = torch.randn(total, hq + 2 * hkv, d, generator=g).cuda().requires_grad_()
    do = torch.randn(total, hq, d, generator=g).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    q, k = vlf.rotary_embedding(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, f)
    out = vlf.varlen_attention(q, k, qkv[:, hq + hkv:], cu, cu, 45, 45, causal=True)
    (out * do).sum().backward()

    x = qkv.detach().double().cpu().requires_grad_()
    ang = pos.cpu().double()[:, None] * f.cpu().double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    turn = lambda y: torch.cat([y[..., :d // 2] * c - y[..., d // 2:] * s, y[..., d // 2:] * c + y[..., :d // 2] * s], -1)  # noqa: E731
    rq, rk, rv = turn(x[:, :hq]), turn(x[:, hq:hq + hkv]), x[:, hq + hkv:]
    outs = []
    for a, b in ((0, 20), (20, 65)):
        kk, vv = rk[a:b].repeat_interleave(2, 1), rv[a:b].repeat_interleave(2, 1)
        z = torch.einsum("ihd,jhd->hij", rq[a:b], kk) * d ** -0.5
        z = z.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -float("inf"))
        outs.append(torch.einsum("hij,jhd->ihd", z.softmax(-1), vv))
    want = torch.cat(outs)
    (want * do.double().cpu()).sum().backward()
    assert (out.detach().cpu().double() - want.detach()).abs().max() <= 1e-5
    assert (qkv.grad.cpu().double() - x.grad).abs().max() <= 1e-4 * x.grad.abs().max()
