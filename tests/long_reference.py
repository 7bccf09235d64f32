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
