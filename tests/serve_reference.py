"""Plain implementations, in 64 bits on the CPU, of the serving operators around the verify step.  They share
nothing with the library: codes are found in a table of the E4M3 values, scales by counting up powers of two,
masks by walking up the tree, tokens by sorting."""
from __future__ import annotations

import math

import numpy as np
import torch

P = 16
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def e4m3_values():
    """The value of every non-negative finite code 0 .. 126."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


VALUES = e4m3_values()


def encode(x):
    """Codes (uint8) of a float64 array: nearest value, ties to the even code, saturated; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0, a)
    hi = np.clip(np.searchsorted(VALUES, a), 0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - VALUES[lo], VALUES[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(VALUES[hi] == a, hi, code)
    code = (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def decode(codes):
    codes = np.asarray(codes, np.uint8)
    mag = np.append(VALUES, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def scale_of(amax):
    """Smallest power of two 2^k, k in [-64, 119], with amax <= 448 * 2^k."""
    k = -64
    while k < 119 and amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def block_codes(x):
    """(codes, scale) of one block."""
    finite = np.abs(x[~np.isnan(x)])
    s = scale_of(finite.max() if finite.size else 0.0)
    return encode(x / s), s


def rope_table(base, d, n):
    """cos and sin of n positions as the library stores them: from 64 bits, rounded to 32."""
    inv = np.array([math.pow(base, -(2.0 * j) / d) for j in range(d // 2)])
    a = np.arange(n, dtype=np.float64)[:, None] * inv
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()


def rotate32(x, cos, sin):
    """The rotation of float32 rows with every product and sum rounded on its own; x [..., D], cos/sin [..., D/2]."""
    lo, hi = x.float().chunk(2, -1)
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def norm_rope64(x, w, eps, cos, sin):
    """(result in 64 bits, bound on the magnitudes that enter each of its elements)."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    mag = y.abs()
    if cos is not None:
        c, s = cos.double(), sin.double()
        lo, hi = y.chunk(2, -1)
        y = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
        l, h = mag.chunk(2, -1)
        mag = torch.cat([l + h, l + h], -1)
    return y, mag


def ancestors(parents, t):
    """sees[i][j]: node j is i or an ancestor of i (parents None: a chain)."""
    m = np.zeros((t, t), bool)
    for i in range(t):
        n = i
        while n >= 0:
            m[i, n] = True
            n = n - 1 if parents is None else int(parents[n])
    return m


def attn64(q, k_cache, v_cache, ks, vs, table, lens, parents, k_new, v_new, scale):
    """(out, weighted magnitude sum_j p_j |v_j|), both [B][T][Hq][D] in 64 bits.  q, k_new, v_new: float64 arrays;
    caches: codes (uint8) with scales [pages][Hkv]; a sequence of negative length gives NaN."""
    b, t, hq, d = q.shape
    hkv = k_new.shape[2]
    g = hq // hkv
    out = np.full(q.shape, np.nan)
    mag = np.full(q.shape, np.nan)
    for i in range(b):
        n = int(lens[i])
        if n < 0:
            continue
        tree = ancestors(None if parents is None else parents[i], t)
        sees = np.concatenate([np.ones((t, n), bool), tree], 1)
        for h in range(hkv):
            kv = []
            for cache, sc, new in ((k_cache, ks, k_new), (v_cache, vs, v_new)):
                rows = [decode(cache[table[i][p // P], h, p % P]) * float(sc[table[i][p // P], h]) for p in range(n)]
                for j in range(0, t, P):
                    codes, s = block_codes(new[i, j:j + P, h])
                    rows.extend(decode(codes) * s)
                kv.append(np.array(rows).reshape(n + t, d))
            k, v = kv
            for j in range(h * g, (h + 1) * g):
                z = q[i, :, j] @ k.T * scale
                z = np.where(sees, z, -np.inf)
                e = np.exp(z - z.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
                out[i, :, j] = p @ v
                mag[i, :, j] = p @ np.abs(v)
    return out, mag


def sample64(x, u, t, top_k, top_p, min_p):
    """The token of one row (float64 logits), -1 for a row without anything above -inf."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    m = x.max()
    if m == -np.inf:
        return -1
    if not t > 0:
        return int(np.argmax(x))
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / t))
    w[w < 2.0 ** -44] = 0  # the definition: such a token is never drawn, not for u = 0 either
    order = np.lexsort((np.arange(len(x)), -x))
    keep = np.ones(len(x), bool)  # by rank
    if 0 < top_k < len(x):
        keep[top_k:] = False
    ws = w[order]
    if top_p < 1:
        before = np.cumsum(ws) - ws
        keep &= before < float(top_p) * ws[keep].sum()
    if min_p > 0:
        keep &= ws >= min_p
    keep[0] = True
    kept = np.sort(order[keep])
    mass = np.cumsum(w[kept])
    return int(kept[min(len(kept) - 1, np.searchsorted(mass, min(max(float(u), 0.0), 1.0) * mass[-1], side="right"))])
