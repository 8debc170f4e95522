"""fp64 definitions of the operators of decoding on a bounded cache (numpy, CPU): rotary positions,
attention behind a shared prefix, the weight each key received, cache eviction.  Plain loops over
sequences and heads; nothing here is shared with the GPU path."""
from __future__ import annotations

import numpy as np

from oracle import attention as orc


def rope(x, positions, inv_freq, sections, rot, interleaved, inverse=False):
    """x [T, H, D] float64; positions int [axes, T]; inv_freq [rot / 2] (taken as exact)."""
    y = np.array(x, np.float64)
    axis = np.repeat(np.arange(len(sections)), sections)
    half = rot // 2
    for c in range(half):
        # positions and fp32 frequencies: their product is exact in 64 bits up to 2^29 x 24 bits;
        # whole turns are taken off in extended precision where the platform has it
        t = np.asarray(positions[axis[c]], np.longdouble) * np.longdouble(np.float32(inv_freq[c]))
        t = np.asarray(np.fmod(t, 2 * np.longdouble("3.14159265358979323846264338327950288")), np.float64)
        if inverse:
            t = -t
        a, b = (2 * c, 2 * c + 1) if interleaved else (c, c + half)
        co, si = np.cos(t)[:, None], np.sin(t)[:, None]
        y[..., a] = x[..., a] * co - x[..., b] * si
        y[..., b] = x[..., b] * co + x[..., a] * si
    return y


def prefix_forward(q, kp, vp, k, v, cu_q, cu_kv, scale, causal, window):
    """out [Tq, Hq, Dv] and lse [Hq, Tq] of attention over [prefix ; own keys] of each sequence."""
    hq, hkv = q.shape[1], kp.shape[1]
    out = np.zeros((q.shape[0], hq, vp.shape[2]))
    lse = np.full((hq, q.shape[0]), -np.inf)
    for s in range(len(cu_q) - 1):
        a, b = cu_q[s], cu_q[s + 1]
        ks = np.concatenate([kp, k[cu_kv[s]:cu_kv[s + 1]]])
        vs = np.concatenate([vp, v[cu_kv[s]:cu_kv[s + 1]]])
        if a == b or len(ks) == 0:
            continue
        ok = orc.visible(b - a, len(ks), causal, window)
        for h in range(hq):
            g = h // (hq // hkv)
            x = np.where(ok, scale * (q[a:b, h] @ ks[:, g].T), -np.inf)
            top = x.max(axis=1)
            live = top > -np.inf
            e = np.exp(x - np.where(live, top, 0.0)[:, None])
            z = e.sum(axis=1)
            out[a:b, h] = np.where(live[:, None], e @ vs[:, g] / np.where(live, z, 1.0)[:, None], 0.0)
            with np.errstate(divide="ignore"):
                lse[h, a:b] = np.where(live, top + np.log(z), -np.inf)
    return out, lse


def key_weights(q, k, lse, cu_q, cu_kv, scale, causal, window, prev=None):
    """[Hkv, Tkv]: prev + column sums of exp(logit - lse) over the rows that see a key."""
    hq, hkv = q.shape[1], k.shape[1]
    w = np.zeros((hkv, k.shape[0])) if prev is None else np.array(prev, np.float64)
    for s in range(len(cu_q) - 1):
        a, b, c, d = cu_q[s], cu_q[s + 1], cu_kv[s], cu_kv[s + 1]
        if a == b or c == d:
            continue
        ok = orc.visible(b - a, d - c, causal, window)
        for h in range(hq):
            g = h // (hq // hkv)
            live = lse[h, a:b] > -np.inf
            x = scale * (q[a:b, h] @ k[c:d, g].T) - np.where(live, lse[h, a:b], 0.0)[:, None]
            w[g, c:d] += np.where(ok & live[:, None], np.exp(np.where(ok, x, -np.inf)), 0.0).sum(axis=0)
    return w


def evict(weights, cu_kv, budget, sink, recent):
    """(index [H][sequence] lists of kept sequence-local keys, cu_out)."""
    h = weights.shape[0]
    kept, cu = [[] for _ in range(h)], [0]
    for a, b in zip(cu_kv[:-1], cu_kv[1:]):
        n = b - a
        cu.append(cu[-1] + min(n, budget))
        for g in range(h):
            if n <= budget:
                kept[g].append(list(range(n)))
                continue
            w = np.array(weights[g, a:b], np.float64)
            w[np.isnan(w)] = -np.inf
            nan = np.isnan(np.asarray(weights[g, a:b], np.float64))
            mid = list(range(sink, n - recent))
            # largest first, a NaN behind every number, ties by index
            mid.sort(key=lambda j: (bool(nan[j]), -w[j], j))
            take = list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n))
            kept[g].append(sorted(take))
    return kept, cu
