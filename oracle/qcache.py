"""Oracle of the quantised paged cache and the operators around it (TEST INFRASTRUCTURE ONLY).

Plain numpy statements of include/qcache.h: the head norm with the position rotation, the three code
formats (int8, e4m3, e2m1 with e4m3 block scales), the page layout and the attention of drafted tokens; of a serving
step, the plan of pages, the rotation by several axes, the attention of chunks and the verification of drafts. What the header defines in float32 (scales and codes) is computed in float32, operation by operation;
everything else in float64, sums of probabilities in exact fractions.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# codes 0 .. 126 of e4m3: 4 exponent bits of bias 7, 3 fraction bits; 127 is its NaN
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])
TOP = {"int8": 127.0, "e4m3": 448.0, "e2m1": 2688.0}


def norm_rope(x, w, eps, pos, table, rot, interleaved) -> np.ndarray:
    """x [n, heads, d] -> float64 [n, heads, d]; w None: no norm."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    if not rot:
        return y
    t = np.asarray(table, dtype=np.float64)[pos][:, None]
    half = rot // 2
    z = t[..., :half] + 1j * t[..., half:]
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    out = y.copy()
    turned = (y[..., first] + 1j * y[..., second]) * z      # multiplication by exp(i angle)
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def nearest(levels, y) -> np.ndarray:
    """Index of the nearest of ascending `levels` to each y >= 0 (beyond the last: the last); ties to the
    even index. Exact: y are float32 values, levels have few bits."""
    y = np.asarray(y, dtype=np.float64)
    i = np.clip(np.searchsorted(levels, y), 1, len(levels) - 1)
    lo, hi = y - levels[i - 1], levels[i] - y
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)


def quantise(x, fmt):
    """Rows x [..., d] -> codes (int8 values, or codes with their sign in the top bit), scale float32 [...],
    block-scale codes [..., d / 16] or None."""
    x = np.asarray(x, dtype=np.float32)
    f = np.float32
    A = np.abs(x).max(-1)
    ok = np.isfinite(x).all(-1) & (np.where(np.isfinite(A), A, 0) >= f(2.0 ** -100))
    A = np.where(ok, A, f(1))
    x = np.where(ok[..., None], x, f(0))
    scale = np.where(ok, A / f(TOP[fmt]), f(0)).astype(f)
    up = (f(TOP[fmt]) / A)[..., None]
    if fmt == "int8":
        return np.rint(x * up).astype(np.int64), scale, None
    if fmt == "e4m3":
        y = x * up
        return nearest(E4M3, np.abs(y)) + 128 * np.signbit(y), scale, None
    b = x.reshape(*x.shape[:-1], -1, 16)
    sb = nearest(E4M3, np.abs(b).max(-1) * (f(448) / A)[..., None])
    s = E4M3[sb].astype(f)
    by = np.where(s > 0, up / np.where(s > 0, s, f(1)), f(0)).astype(f)
    y = (b * by[..., None]).reshape(x.shape)
    return nearest(E2M1, np.abs(y)) + 8 * np.signbit(y), scale, sb


def values(codes, scale, block, fmt) -> np.ndarray:
    """float64 values of codes (products of the exact code values and the scales)."""
    codes = np.asarray(codes)
    scale = np.asarray(scale, dtype=np.float64)[..., None]
    if fmt == "int8":
        return codes * scale
    if fmt == "e4m3":
        return np.where(codes & 128, -1.0, 1.0) * E4M3[codes & 127] * scale
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(E4M3[block], 16, axis=-1) * scale


def page_bytes(fmt, d, heads, page) -> int:
    row = d // 2 + d // 16 if fmt == "e2m1" else d
    return heads * 2 * page * (row + 4)


def pack(pages, slots, k, v, fmt, page) -> None:
    """Writes k, v [n, heads, d] into pages uint8 [n_pages, page_bytes] at `slots` (-1: skipped)."""
    n, heads, d = k.shape
    rb = d // 2 if fmt == "e2m1" else d
    bb = d // 16 if fmt == "e2m1" else 0
    part = 2 * page * (rb + 4 + bb)
    for which, x in enumerate((k, v)):
        codes, scale, block = quantise(x, fmt)
        raw = (codes & 255).astype(np.uint8)
        if fmt == "e2m1":
            raw = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
        for i in range(n):
            if slots[i] < 0 or slots[i] >= len(pages) * page:
                continue
            p, t = divmod(int(slots[i]), page)
            for h in range(heads):
                run = pages[p, h * part + which * page * rb:][:page * rb].reshape(-1, 16)
                for c in range(rb // 16):
                    at = t * (rb // 16) + c
                    run[at ^ ((at >> 3) & 7)] = raw[i, h, 16 * c:16 * c + 16]
                s0 = h * part + 2 * page * rb + which * page * 4 + 4 * t
                pages[p, s0:s0 + 4] = np.frombuffer(np.float32(scale[i, h]).tobytes(), dtype=np.uint8)
                if bb:
                    b0 = h * part + 2 * page * (rb + 4) + which * page * bb + t * bb
                    pages[p, b0:b0 + bb] = block[i, h]


def attend(q, K, V, lens, nodes, sees, scale):
    """q [n_seq, n_nodes, hq, d]; K[b], V[b] float64 [places, heads, d] of sequence b; sees [n_seq, n_nodes,
    n_nodes] truth values. Returns out, lse and weight = sum_t p_t |v_t| / sum_t p_t (for error bounds)."""
    n_seq, n_nodes, hq, d = q.shape
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for b in range(n_seq):
        heads = K[b].shape[1]
        for i in range(nodes[b]):
            seen = np.concatenate([np.arange(lens[b]), lens[b] + np.flatnonzero(sees[b, i, :nodes[b]])]).astype(int)
            if not len(seen):
                continue
            for h in range(hq):
                kv = h // (hq // heads)
                s = scale * (K[b][seen, kv] @ q[b, i, h].astype(np.float64))
                p = np.exp(s - s.max())
                out[b, i, h] = p @ V[b][seen, kv] / p.sum()
                weight[b, i, h] = p @ np.abs(V[b][seen, kv]) / p.sum()
                lse[b, i, h] = s.max() + np.log(p.sum())
    return out, lse, weight


def norm_rope_axes(x, w, eps, pos, table, sections, interleaved) -> np.ndarray:
    """norm_rope with positions pos [axes, n]: sections[a] pairs turn by axis a's."""
    half = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    t = np.asarray(table, dtype=np.float64)
    rows = np.stack([np.concatenate([t[pos[axis, i], np.arange(half)], t[pos[axis, i], half + np.arange(half)]]) for i in range(x.shape[0])])
    return norm_rope(x, w, eps, np.arange(x.shape[0]), rows, 2 * half, interleaved)


def plan(lens, news, free_pages, taken, table, n_tokens, page, held=None):
    """table (a copy, with the new pages), starts, slots, pos, taken after it, and whether pages were wanting or
    something was out of range. held (a list): updated in place."""
    table, n_free = np.array(table), len(free_pages)
    width = table.shape[1]
    starts, slots, pos, lack, odd = [0], [], [], False, not 0 <= taken <= n_free
    taken = min(max(taken, 0), n_free)
    for b, (n, t) in enumerate(zip(lens, news)):
        odd |= n < 0 or t < 0 or max(n, 0) + max(t, 0) > width * page
        n, t = max(n, 0), max(t, 0)
        have = -(-n // page)
        if held is not None:
            odd |= not 0 <= held[b] <= width
            have = held[b] = min(max(held[b], min(have, width)), width)
        for k in range(have, min(-(-(n + t) // page), width)):
            if held is not None and taken < n_free:           # a page that is wanting is not held
                held[b] = k + 1
            lack |= taken >= n_free
            table[b, k] = free_pages[taken] if taken < n_free else -1
            taken += taken < n_free
        for place in range(n, n + t):
            p = table[b, place // page] if place < width * page else -1
            slots.append(p * page + place % page if p >= 0 else -1)
            pos.append(place)
        starts.append(starts[-1] + t)
    odd |= len(slots) > n_tokens
    pad = max(n_tokens - len(slots), 0)
    return (table, np.minimum(starts, n_tokens), np.array(slots[:n_tokens] + [-1] * pad), np.array(pos[:n_tokens] + [0] * pad), taken,
            lack, odd)


def verify(p, q, tokens, parents, nodes, u):
    """One sequence: p [n_nodes + 1, vocab], q [n_nodes, vocab] (float64 of the values as they are). Returns the accepted
    nodes and the token drawn after them (-1: nothing to draw from)."""
    from fractions import Fraction
    vocab = p.shape[1]
    clean = [np.where(np.isfinite(x) & (x > 0), x, 0.0) for x in (p, q)]
    at, came = -1, []
    while True:
        w = [Fraction(x) for x in clean[0][at + 1]]
        total, taken, over = Fraction(1), None, False
        for c in range(nodes):
            x = tokens[c]
            if parents[c] != at or not -1 <= parents[c] < c or not 0 <= x < vocab:
                continue
            row = clean[1][at + 1]
            if Fraction(float(u[c])) * Fraction(row[x]) * total < w[x]:
                taken = c
                break
            w = [max(a - total * Fraction(b), Fraction(0)) for a, b in zip(w, row)]
            total = sum(w)
            if total == 0:
                w = [Fraction(x) for x in clean[0][at + 1]]
                break
        if taken is None:
            break
        came.append(taken)
        at = taken
    mark, run = Fraction(float(u[-1])) * sum(w), Fraction(0)
    for k, x in enumerate(w):
        run += x
        if run > mark:
            return came, k
    return came, -1


def seen_by(t, places, prefix, window):
    """The places that the row at place t of a sequence of `places` sees: lo, hi."""
    return max(0, t + 1 - window) if window else 0, max(t + 1, min(max(prefix, 0), places))


def attend_chunk(q, K, V, lens, news, scale, cap=0.0, window=0, prefix=None, slopes=None, missing=None):
    """q [n_tokens, hq, d], the new tokens of all sequences one after another; K[b], V[b] float64 [places, heads, d];
    missing[b]: places that are not there. Returns out, lse, weight = sum p |v| / sum p, and top = the largest over the
    places of p max|v| / sum p (for error bounds)."""
    n, hq, d = q.shape
    out, weight, lse, top = np.zeros(q.shape), np.zeros(q.shape), np.full((n, hq), -np.inf), np.zeros((n, hq))
    row = 0
    for b, (ln, t) in enumerate(zip(lens, news)):
        for i in range(t):
            lo, hi = seen_by(ln + i, ln + t, 0 if prefix is None else prefix[b], window)
            at = np.setdiff1d(np.arange(lo, hi), [] if missing is None else missing[b])
            if len(at):
                for h in range(hq):
                    kv = h // (hq // K[b].shape[1])
                    s = scale * (K[b][at, kv] @ q[row, h].astype(np.float64))
                    if cap:
                        s = cap * np.tanh(s / cap)
                    if slopes is not None:
                        s = s + slopes[h] * (at - (ln + i))
                    p = np.exp(s - s.max())
                    v = V[b][at, kv]
                    out[row, h] = p @ v / p.sum()
                    weight[row, h] = p @ np.abs(v) / p.sum()
                    top[row, h] = (p * np.abs(v).max(-1)).max() / p.sum()
                    lse[row, h] = s.max() + np.log(p.sum())
            row += 1
    return out, lse, weight, top
