"""Plain implementations, in 64 bits on the CPU, of the operators for long sequences and shaped answers: attention under
a window with sinks, weights of cached slots, eviction, logits processing.  They share nothing with the library."""
from __future__ import annotations

import math

import numpy as np

import serve_reference as ref

P = 16


def _chain(parents, node):
    """A node and its ancestors, from the node up (parents None: a chain)."""
    out = []
    while node >= 0:
        out.append(node)
        node = node - 1 if parents is None else int(parents[node])
    return out


def sees(n, t, parents, window, sinks):
    """[t][n + t]: what each new token sees of n cached slots and of the new tokens (window 0: everything)."""
    m = np.zeros((t, n + t), bool)
    depth = [len(_chain(parents, i)) - 1 for i in range(t)]
    for i in range(t):
        place = n + depth[i]
        ok = lambda p: window == 0 or p < sinks or p > place - window  # noqa: E731
        slots = np.arange(n)
        m[i, :n] = True if window == 0 else (slots < sinks) | (slots > place - window)
        for j in _chain(parents, i):
            m[i, n + j] = ok(n + depth[j])
    return m


def window_attn64(c, window, sinks, scale):
    """(out, sum p |v|, lse) of every new token, [B][T][Hq](..D); a sequence of negative length gives NaN.  Slots that
    nobody sees are not looked at."""
    q, kn, vn = (c[n].double().numpy() for n in ("q", "kn", "vn"))
    b, t, hq, d = q.shape
    hkv = kn.shape[2]
    g = hq // hkv
    out, mag, lse = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    for i in range(b):
        n = int(c["lens"][i])
        if n < 0:
            continue
        see = sees(n, t, None if c["parents"] is None else c["parents"][i], window, sinks)
        use = np.flatnonzero(see.any(0))
        slots = use[use < n]
        page, at = c["table"][i][slots // P], slots % P
        for h in range(hkv):
            kv = []
            for cache, sc, new in ((c["k"], c["ks"], kn), (c["v"], c["vs"], vn)):
                rows = [ref.decode(cache[page, h, at]) * sc[page, h][:, None].astype(np.float64)]
                for j in range(0, t, P):
                    codes, s = ref.block_codes(new[i, j:j + P, h])
                    rows.append(ref.decode(codes) * s)
                kv.append(np.concatenate(rows))
            k, v = kv
            m = np.concatenate([see[:, slots], see[:, n:]], 1)
            for j in range(h * g, (h + 1) * g):
                z = np.where(m, q[i, :, j] @ k.T * scale, -np.inf)
                top = z.max(1, keepdims=True)
                e = np.exp(z - top)
                total = e.sum(1, keepdims=True)
                p = e / total
                lse[i, :, j] = (top + np.log(total))[:, 0]
                # a value with a NaN reaches its own column of the rows that see it, and no other row
                out[i, :, j] = p @ np.nan_to_num(v)
                mag[i, :, j] = p @ np.abs(np.nan_to_num(v))
                odd = np.isnan(v)
                if odd.any():
                    out[i, :, j][(m.astype(float) @ odd) > 0] = np.nan
    return out, mag, lse


def weights64(c, weights, lse, lens, prev, nodes_of, decay, scale):
    """(weights after the call, their tolerance), [pages][Hkv][16] in 64 bits.  nodes_of(b): the nodes whose rows count.
    Tolerance, by term: a score in 32 bits is off by 2 D 2^-24 sum |q k| scale (D products and sums, which tensor cores
    may truncate), score - lse by 2^-22 (|score| + |lse|) more (the units, the constants, one subtraction), the
    exponential by 2^-21 of itself, each sum and product of weights by 2^-20 of what it adds up."""
    q = c["q"].double().numpy()
    b, t, hq, d = q.shape
    hkv = c["k"].shape[1]
    g = hq // hkv
    out, tol = weights.astype(np.float64).copy(), np.zeros(weights.shape)
    for i in range(b):
        n = int(lens[i])
        if n < 1:
            continue
        slots = np.arange(n)
        page, at = c["table"][i][slots // P], slots % P
        for h in range(hkv):
            k = ref.decode(c["k"][page, h, at]) * c["ks"][page, h][:, None].astype(np.float64)
            had = np.where(slots < prev[i], out[page, h, at], 0.0) * decay
            got, off = had.copy(), 2.0 ** -20 * np.abs(had)
            for a in nodes_of(i):
                for j in range(h * g, (h + 1) * g):
                    z = k @ q[i, a, j] * scale
                    p = np.exp(z - lse[i, a, j])
                    got += p
                    off += p * (2 * d * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[i, a, j])) + 2.0 ** -22 * (np.abs(z) + abs(lse[i, a, j])) + 2.0 ** -19)
            out[page, h, at], tol[page, h, at] = got, off
    return out, tol


def kept_slots(weights, budget, sinks, recent):
    """The slots that stay of one head's weights [L], ascending."""
    n = len(weights)
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sinks, n - recent)
    w = weights[middle].astype(np.float64)
    w = np.where(np.isnan(w), -np.inf, w)
    order = np.lexsort((middle, ~np.isnan(weights[middle]) * -1, -w))  # heavier; a number before a NaN; lower slot
    best = middle[order[:budget - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)]))


def evict(kind, caches, scales, weights, table, lens, new_tables, budget, sinks, recent):
    """Changes the host arrays as kv_evict does; returns kept.  caches: [k, v] as raw arrays [pages][Hkv][16][..]; scales:
    [k, v] in 64 bits for `block8`."""
    hkv = weights.shape[1]
    kept = np.full((len(lens), hkv, budget), -1, np.int64)
    for b, n in enumerate(lens):
        if n < 1:
            continue
        page, at = table[b][np.arange(n) // P], np.arange(n) % P
        for h in range(hkv):
            stay = kept_slots(weights[page, h, at], budget, sinks, recent)
            kept[b, h, :len(stay)] = stay
            rows = [c[page[stay], h, at[stay]].copy() for c in caches]
            w = weights[page[stay], h, at[stay]].copy()
            old = [s[page[stay], h].copy() for s in scales] if kind == "block8" else None
            for j in range(0, len(stay), P):
                m, to = min(P, len(stay) - j), new_tables[b][j // P]
                weights[to, h, :m] = w[j:j + m]
                for x in range(2):
                    block = rows[x][j:j + m]
                    if kind == "block8":
                        top = old[x][j:j + m].max()
                        f = (old[x][j:j + m] / top)[:, None]
                        block = np.where(f == 1, block, ref.encode(ref.decode(block) * f))
                        scales[x][to, h] = top
                    caches[x][to, h, :m] = block
    return kept


def logits64(x, history, lens, starts, rep, pres, freq, bias, mask, mask_index, tokens, parents):
    """(logits [B][T][V] in 64 bits after the call, magnitudes that entered each, which were touched).  history [B][H] or
    None; bias: (tokens, values) or None; mask: truth values [M][V] or None; a sequence of negative length is left."""
    out = np.array(x, np.float64)
    b, t, v = out.shape
    mag, touched = np.abs(out), np.zeros(out.shape, bool)
    for i in range(b):
        n = 0 if lens is None else int(lens[i])
        if n < 0:
            continue
        words = [] if history is None else [int(w) for w in history[i][:min(n, len(history[i]))]]
        start = 0 if starts is None else int(starts[i])
        for a in range(t):
            path = [] if tokens is None else [int(tokens[i][j]) for j in _chain(None if parents is None else parents[i], a)]
            count = {}
            for w in words[max(start, 0):] + path:
                count[w] = count.get(w, 0) + 1
            for w in set(words) | set(path):
                if not 0 <= w < v:
                    continue
                y = out[i, a, w]
                if rep is not None:
                    y = y / float(rep[i]) if y > 0 else y * float(rep[i])
                m = max(abs(out[i, a, w]), abs(y))
                c = count.get(w, 0)
                if c and freq is not None:
                    y, m = y - float(freq[i]) * c, m + abs(float(freq[i])) * c
                if c and pres is not None:
                    y, m = y - float(pres[i]), m + abs(float(pres[i]))
                out[i, a, w], mag[i, a, w], touched[i, a, w] = y, m, True
            if bias is not None:
                for w, y in {int(w): float(y) for w, y in zip(bias[0][i], bias[1][i])}.items():
                    if 0 <= w < v:
                        out[i, a, w] += y
                        mag[i, a, w] += abs(y)
                        touched[i, a, w] = True
            if mask is not None:
                m = i * t + a if mask_index is None else int(mask_index[i][a])
                if m >= 0:
                    no = ~mask[m] if m < len(mask) else np.ones(v, bool)
                    out[i, a, no], mag[i, a, no], touched[i, a, no] = -np.inf, 0.0, True
    return out, mag, touched
