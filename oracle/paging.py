"""64-bit definitions of the operators of serving from a cache of pages in 8 bits (numpy, CPU): the norm of
each head with its rotary positions and its gradients, e4m3 and the scales of pages, attention over
pages, page tables.  Plain loops; nothing here is shared with the GPU path."""
from __future__ import annotations

import numpy as np

from oracle import attention as orc
from oracle import decoding as dec


def norm_rope(x, w, eps, positions, inv_freq, sections, rot, interleaved):
    """R(t) (w o x / sqrt(mean(x^2) + eps)); x [T, H, D], w [D]."""
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * w
    return dec.rope(y, positions, inv_freq, sections, rot, interleaved)


def norm_rope_bwd(dy, x, w, eps, positions, inv_freq, sections, rot, interleaved):
    """(dx, dw) of sum(norm_rope(x) o dy)."""
    g = dec.rope(dy, positions, inv_freq, sections, rot, interleaved, inverse=True)
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    u = x * r
    gw = g * w
    return r * (gw - u * (gw * u).mean(axis=-1, keepdims=True)), (g * u).sum(axis=(0, 1))


def e4m3_values():
    """The value of each byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = np.nan if b & 127 == 127 else -x if b & 128 else x
    return out


VALUES = e4m3_values()
_SORTED = VALUES[:127]  # 0 .. 448, ascending, the byte is the index


def to_e4m3(x):
    """Bytes of x rounded to nearest, ties to the even byte; NaN (0x7f, with the sign) where not finite."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.searchsorted(_SORTED, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _SORTED[lo], _SORTED[hi] - a
    take = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    take = np.where(np.isfinite(x), take, 127)
    return (take | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax):
    e = -64
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def pages_write(k, v, cache, table, cu, lens):
    """cache: (k_pages, v_pages uint8 [N, H, P, D], k_scale, v_scale [N, H]); returns it written."""
    kp, vp, ks, vs = (np.array(x) for x in cache)
    page = kp.shape[2]
    for s in range(len(lens)):
        first = lens[s] - (cu[s + 1] - cu[s])
        for p in range(first // page, -(-lens[s] // page)) if cu[s + 1] > cu[s] else ():
            a, b = max(first, p * page), min(lens[s], (p + 1) * page)
            n = table[s][p]
            for x, pages, scales in ((k, kp, ks), (v, vp, vs)):
                for h in range(kp.shape[1]):
                    y = np.asarray(x[cu[s] + a - first:cu[s] + b - first, h], np.float64)
                    fine = np.abs(y[np.isfinite(y)])
                    scale = scale_for(fine.max() if fine.size else 0.0)
                    if a > p * page:
                        was = float(scales[n, h])
                        scale = max(scale, was)
                        if scale != was:
                            pages[n, h] = to_e4m3(VALUES[pages[n, h]] * (was / scale))
                    scales[n, h] = scale
                    pages[n, h, a - p * page:b - p * page] = to_e4m3(y / scale)
    return kp, vp, ks, vs


def keys_of(pages, scale, row, length):
    """[length, H, D]: what a sequence's bytes stand for (0 for a page outside the pool)."""
    page = pages.shape[2]
    out = np.zeros((length, pages.shape[1], pages.shape[3]))
    for j in range(length):
        n = row[j // page]
        if 0 <= n < pages.shape[0]:
            out[j] = VALUES[pages[n, :, j % page]] * np.asarray(scale[n], np.float64)[:, None]
    return out


def pages_attention(q, cache, table, cu_q, lens, scale, causal, window):
    """out [Tq, Hq, Dv], lse [Hq, Tq], and for the tolerances sum_j p_j |v_j| and scale sum_c |q_c k_c| at most."""
    kp, vp, ks, vs = cache
    hq, hkv = q.shape[1], kp.shape[1]
    out = np.zeros((q.shape[0], hq, vp.shape[3]))
    size = np.zeros_like(out)
    lse = np.full((hq, q.shape[0]), -np.inf)
    reach = np.zeros((hq, q.shape[0]))
    for s in range(len(lens)):
        a, b = cu_q[s], cu_q[s + 1]
        if a == b or lens[s] == 0:
            continue
        k, v = keys_of(kp, ks, table[s], lens[s]), keys_of(vp, vs, table[s], lens[s])
        ok = orc.visible(b - a, lens[s], causal, window)
        page = np.asarray(table[s])[np.arange(lens[s]) // kp.shape[2]]
        ok = ok & ((page >= 0) & (page < kp.shape[0]))  # (keys of a page outside the pool are passed over)
        for h in range(hq):
            g = h // (hq // hkv)
            x = np.where(ok, scale * (q[a:b, h] @ k[:, g].T), -np.inf)
            top = x.max(axis=1)
            live = top > -np.inf
            e = np.exp(x - np.where(live, top, 0.0)[:, None])
            z = np.where(live, e.sum(axis=1), 1.0)[:, None]
            p = np.where(ok, e, 0.0) / z
            seen = ok.any(axis=0)
            vv = np.where(seen[:, None], v[:, g], 0.0)
            out[a:b, h], size[a:b, h] = p @ vv, p @ np.abs(vv)
            lse[h, a:b] = np.where(live, top + np.log(z[:, 0]), -np.inf)
            reach[h, a:b] = scale * (np.abs(q[a:b, h]) @ np.abs(np.where(seen[:, None], k[:, g], 0.0)).T).max(axis=1)
    return out, lse, size, reach


def fork(table, lens, refs, parents, grow, page):
    """(table, lens, refs, src, dst, left) of the next step, as lists; tables of the pages alone, without -1."""
    outside = list(refs)
    for row, x in zip(table, lens):
        for p in row[:-(-x // page)]:
            outside[p] -= 1
    size = [lens[p] if p >= 0 else 0 for p in parents]
    whole = {p for r, x in zip(parents, size) if r >= 0 for p in table[r][:x // page]}
    count, rows, copies, kept = list(outside), [], [], set()
    for r, x in zip(parents, size):
        rows.append(list(table[r][:x // page]) if r >= 0 else [])
        for p in rows[-1]:
            count[p] += 1
    for s, (r, x) in enumerate(zip(parents, size)):
        copies.append(-1)
        if x % page:
            p = table[r][x // page]
            if outside[p] == 0 and p not in whole and p not in kept:
                kept.add(p)
                count[p] += 1
                rows[s].append(p)
            else:
                copies[s] = p
    free = [i for i, n in enumerate(count) if n == 0]
    need = [-(-(x + g) // page) - len(row) for x, g, row in zip(size, grow, rows)]
    if sum(need) > len(free):
        none = [-1] * len(parents)
        return [[] for _ in parents], [0] * len(parents), list(refs), none, none, len(free) - sum(need)
    dst = []
    for s, n in enumerate(need):
        new, free = free[:n], free[n:]
        dst.append(new[0] if copies[s] >= 0 else -1)
        for p in new:
            count[p] = 1
        rows[s] += new
    return rows, [x + g for x, g in zip(size, grow)], count, copies, dst, len(free)


def compact(table, refs):
    """(table, refs, to, src, dst, used), as lists."""
    used = sum(n > 0 for n in refs)
    src = [i for i in range(used, len(refs)) if refs[i] > 0]
    dst = [i for i in range(used) if refs[i] <= 0]
    to = [i if n > 0 else -1 for i, n in enumerate(refs)]
    count = [max(n, 0) if i < used else 0 for i, n in enumerate(refs)]
    for a, b in zip(src, dst):
        to[a], count[b] = b, refs[a]
    rows = [[to[p] if 0 <= p < len(refs) else -1 for p in row] for row in table]
    return rows, count, to, src, dst, used
