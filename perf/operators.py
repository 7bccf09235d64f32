"""Cases of the serving operators around the verify step: their inputs, their plain form in elementary
torch operations (32 bits, 64 where 32 lose what matters), the framework's calls, and their definition in
64 bits.

  norm_rope  qk_norm_rope: per-head norms of queries and keys and the position rotation
  append     kv_append_paged: ragged new keys and values into the paged cache
  attn       tree_attn_paged_block8: tree attention over an 8-bit cache with a scale per page and head
  sample     sample_tokens: temperature, top-k, top-p and min-p from given uniform numbers
"""
import math

import numpy as np
import torch

own = False

P = 16  # slots per page
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ROPE_BASE = 10000.0
EPS = 1e-6
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence decoding its next token: latency alone
        dict(name="attn_decode_b1", op="attn", dtype="f16", B=1, T=1, Hq=32, Hkv=32, D=128, lo=2048, hi=2048, scale=0.0),
        # a decoding batch of ragged lengths, one token each: the cache's bytes
        dict(name="attn_decode_b64", op="attn", dtype="bf16", B=64, T=1, Hq=32, Hkv=8, D=128, lo=256, hi=8192, scale=0.0),
        # a serving batch's 64-node trees (the bench's serving workload)
        dict(name="attn_tree_b16", op="attn", dtype="bf16", B=16, T=64, Hq=32, Hkv=8, D=128, lo=512, hi=8192, scale=0.0),
        # long contexts with 26-node trees (the bench's 32k workload)
        dict(name="attn_tree_32k", op="attn", dtype="bf16", B=8, T=26, Hq=64, Hkv=8, D=128, lo=32768, hi=32768, scale=0.0),
        # the decoding batch's new tokens, one a sequence, into the block-scaled cache
        dict(name="append_decode_b64", op="append", dtype="bf16", cache="block8", B=64, lo=1, hi=1, past=4096, Hkv=8, D=128, rope=True),
        # ragged prompts into the block-scaled cache, rotated on the way
        dict(name="append_prompt_block8", op="append", dtype="bf16", cache="block8", B=16, lo=100, hi=4000, past=0, Hkv=8, D=128, rope=True),
        # prompts of many heads into a 16-bit cache, behind earlier turns
        dict(name="append_prompt_f16", op="append", dtype="f16", cache="act", B=8, lo=512, hi=1500, past=1000, Hkv=32, D=128, rope=True),
        # a tree batch's queries and keys: 16 sequences of 64 nodes, views of one projection
        dict(name="norm_rope_tree", op="norm_rope", dtype="bf16", N=1024, Hq=32, Hkv=8, D=128, norm=True, rope=True, packed=True),
        # a prompt batch's queries and keys
        dict(name="norm_rope_prompt", op="norm_rope", dtype="bf16", N=16384, Hq=32, Hkv=8, D=128, norm=True, rope=True, packed=True),
        # one row at the tests' vocabulary
        dict(name="sample_b1", op="sample", dtype="f32", N=1, V=32000, kind="top"),
        # a serving batch, each row with parameters of its own
        dict(name="sample_b64", op="sample", dtype="bf16", N=64, V=128000, kind="mixed"),
        # a large batch drawn from whole tempered distributions
        dict(name="sample_b256_full", op="sample", dtype="f16", N=256, V=32000, kind="full"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "append", "norm_rope", "sample"])
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 16])
        g = rng.choice([1, 2, 3, 4, 7, 8])
        t = rng.choice([1, 1, 2, 5, rng.randint(3, 64)])
        b = _log(rng, 1, 64)
        d = rng.choice([64, 128, 128])
        hi = _log(rng, 16, 16384)
        cap = 2e8 // (hkv * d)  # cache elements of K
        hi = int(max(1, min(hi, cap // b, 4e10 // (4 * t * hkv * g * d * b))))
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), B=b, T=t, Hq=hkv * g, Hkv=hkv, D=d, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                    scale=rng.choice([0.0, 0.05]))
    if op == "append":
        hkv = rng.choice([1, 2, 3, 8, 8, 32])
        b = _log(rng, 1, 128)
        hi = _log(rng, 1, 8192)
        hi = int(max(1, min(hi, 250000 // (b * hkv) + 1)))
        return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]), cache=rng.choice(["act", "e4m3", "block8", "block8"]), B=b, lo=rng.choice([0, hi]), hi=hi,
                    past=rng.choice([0, 37, 500, 5000]), Hkv=hkv, D=rng.choice([64, 128]), rope=rng.random() < 0.8)
    if op == "norm_rope":
        hkv = rng.choice([1, 4, 8, 32])
        return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]), N=max(1, min(_log(rng, 1, 16384), 300000 // (hkv * 5))), Hq=hkv * rng.choice([1, 3, 4]), Hkv=hkv,
                    D=rng.choice([64, 128]), norm=rng.random() < 0.8, rope=rng.random() < 0.8, packed=rng.random() < 0.5)
    v = _log(rng, 1000, 200000)
    if rng.random() < 0.5:
        v = v // 8 * 8
    return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), N=max(1, min(_log(rng, 1, 512), 8000000 // v)), V=v, kind=rng.choice(["top", "mixed", "full", "greedy"]))


# ---------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rope_table(max_pos, d):
    """(cos, sin) of every position, from angles in 64 bits."""
    inv = ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos(), a.sin()


_ropes = {}


def _handles(max_pos, d):
    """The rotation as a program keeps it: the plain form's table and the framework's, one for each size."""
    max_pos = -(-max_pos // 4096) * 4096
    if (max_pos, d) not in _ropes:
        cos, sin = _rope_table(max_pos, d)
        _ropes[max_pos, d] = [cos.float(), sin.float(), None]
    h = _ropes[max_pos, d]
    if own and h[2] is None:
        import medusa_tree_speculative_attn_gb300 as mt
        h[2] = mt.Rope(ROPE_BASE, d, max_pos)
    return h


def _lengths(b, lo, hi):
    """b lengths of [lo, hi], the largest of them hi: the same ones for every seed, which orders them."""
    n = np.random.default_rng(1).integers(lo, hi + 1, size=b)
    n[0] = hi
    return n


def _tables(rng, lens):
    """A block table over shuffled pages, and the number of pages."""
    need = (np.asarray(lens) + P - 1) // P
    pages = int(need.sum()) + 3
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(need), max(1, int(need.max()))), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b, n in enumerate(need):
        table[b, :n] = perm[at[b]:at[b + 1]]
    return torch.from_numpy(table).cuda(), pages


def _exponent(amax):
    """k of the smallest scale 2^k with amax <= 448 * 2^k, within [-64, 119]."""
    f, e = torch.frexp(amax)
    return torch.where(f <= 0.875, e - 9, e - 8).clamp(-64, 119)


def _pow2(k):
    return torch.ldexp(torch.ones_like(k, dtype=torch.float32), k)


def _codes(x):
    return x.clamp(-448, 448).to(F8)


def _block_cache(g, pages, hkv, d, dtype, outliers):
    """A block-scaled cache of seeded values: codes [pages][Hkv][16][D] and scales [pages][Hkv]."""
    size = torch.exp(0.5 * _randn(g, pages, hkv, 1, 1))
    channel = torch.ones(hkv, 1, d, device="cuda")
    if outliers:  # keys have a few large channels
        channel[:, :, torch.randint(d, (3,), generator=g, device="cuda")] = 4.0
    x = torch.randn(pages, hkv, P, d, generator=g, device="cuda", dtype=dtype).float() * size * channel
    s = _pow2(_exponent(x.abs().amax((2, 3))))
    return _codes(x / s[:, :, None, None]), s


def _tree(rng, t):
    parents = np.full(t, -1, np.int32)
    for i in range(1, t):
        parents[i] = rng.integers(max(0, i - 12), i)
    return parents


def prepare(case, seed):
    return {"attn": _prepare_attn, "append": _prepare_append, "norm_rope": _prepare_norm_rope, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_attn(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, t, hq, hkv, d, dt = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    lens = rng.permutation(_lengths(b, c["lo"], c["hi"]))
    table, pages = _tables(rng, lens)
    k, ks = _block_cache(g, pages, hkv, d, dt, True)
    v, vs = _block_cache(g, pages, hkv, d, dt, False)
    s = dict(c, k_cache=k, v_cache=v, k_scales=ks, v_scales=vs, table=table, lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
             parents=torch.from_numpy(np.stack([_tree(rng, t) for _ in range(b)])).cuda(), q=_randn(g, b, t, hq, d).to(dt),
             k_new=_randn(g, b, t, hkv, d).to(dt), v_new=_randn(g, b, t, hkv, d).to(dt))
    s["out"] = torch.zeros_like(s["q"])
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        s["workspace"] = mt.alloc_block8_workspace(s["q"], s["k_cache"], s["table"])
    return s


def _prepare_append(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, hkv, d, dt = c["B"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    order = rng.permutation(b)
    new, past = _lengths(b, c["lo"], c["hi"])[order], np.random.default_rng(2).integers(0, c["past"] + 1, size=b)[order]
    table, pages = _tables(rng, past + new)
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(offsets[-1])
    kv = _randn(g, n, 2, hkv, d).to(dt)  # the projection's output: keys and values of a row side by side
    s = dict(c, k=kv[:, 0], v=kv[:, 1], table=table, lens=torch.from_numpy(past.astype(np.int32)).cuda(), offsets=torch.from_numpy(offsets).cuda())
    if c["cache"] == "block8":
        s["k_cache"], s["k_scales"] = _block_cache(g, pages, hkv, d, dt, True)
        s["v_cache"], s["v_scales"] = _block_cache(g, pages, hkv, d, dt, False)
    else:
        s["k_cache"], s["v_cache"] = (_randn(g, pages, hkv, P, d).to(dt) for _ in range(2))
        if c["cache"] == "e4m3":
            s["k_cache"], s["v_cache"] = _codes(s["k_cache"].float() * 32), _codes(s["v_cache"].float() * 32)
    s["rot"] = _handles(c["past"] + c["hi"] + 1, d) if c["rope"] else None
    if own:
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _prepare_norm_rope(c, seed):
    g = _generator(seed)
    n, hq, hkv, d, dt = c["N"], c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    x = (_randn(g, n, hq + 2 * hkv, d) * torch.exp(0.3 * _randn(g, n, 1, 1))).to(dt)  # a projection's rows: queries, keys, values
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    if not c["packed"]:
        q, k = q.contiguous(), k.contiguous()
    s = dict(c, q=q, k=k, q_out=torch.empty(n, hq, d, dtype=dt, device="cuda"), k_out=torch.empty(n, hkv, d, dtype=dt, device="cuda"),
             positions=torch.randint(32768, (n,), generator=g, device="cuda", dtype=torch.int32), rot=_handles(32768, d) if c["rope"] else None, qw=None, kw=None)
    if c["norm"]:
        s["qw"], s["kw"] = ((1 + 0.1 * _randn(g, d)).to(dt) for _ in range(2))
    if own:
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    n, v, kind = c["N"], c["V"], c["kind"]
    x = 2.5 * _randn(g, n, v)
    x.scatter_add_(1, torch.randint(v, (n, 8), generator=g, device="cuda"), 6 * torch.rand(n, 8, generator=g, device="cuda"))
    temperature, top_k, top_p, min_p = np.ones(n), np.zeros(n), np.ones(n), np.zeros(n)
    if kind == "top":
        temperature[:], top_k[:], top_p[:] = 0.8, 50, 0.95
    elif kind == "mixed":
        temperature[:] = rng.choice([0.0, 0.6, 0.8, 1.0, 1.3], size=n)
        top_k[:] = rng.choice([0, 0, 1, 20, 64, 1000], size=n)
        top_p[:] = rng.choice([1.0, 0.9, 0.95, 0.5], size=n)
        min_p[:] = rng.choice([0.0, 0.0, 0.05, 0.1], size=n)
    elif kind == "greedy":
        temperature[:] = 0
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    return dict(c, logits=x.to(TYPES[c["dtype"]]), uniforms=torch.rand(n, generator=g, device="cuda"), temperature=f32(temperature),
                top_k=torch.from_numpy(top_k.astype(np.int32)).cuda(), top_p=f32(top_p), min_p=f32(min_p), tokens=torch.empty(n, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------- one pass

def run(s):
    return {"attn": _run_attn, "append": _run_append, "norm_rope": _run_norm_rope, "sample": _run_sample}[s["op"]](s)


def _run_attn(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        return mt.tree_attn_paged_block8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["lens"], s["parents"], s["out"],
                                         k_new=s["k_new"], v_new=s["v_new"], workspace=s["workspace"], sm_scale=s["scale"])
    b, t, hq, hkv, d = s["B"], s["T"], s["Hq"], s["Hkv"], s["D"]
    g, pages = hq // hkv, s["table"].clamp(min=0).long()

    def past(cache, scales):
        x = cache[pages].float() * scales[pages][..., None, None]  # [B][blocks][Hkv][16][D]
        return x.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)

    def new(x):
        blocks = torch.zeros(b, -(-t // P) * P, hkv, d, device=x.device)
        blocks[:, :t] = x
        blocks = blocks.view(b, -1, P, hkv, d)
        sc = _pow2(_exponent(blocks.abs().amax((2, 4))))[:, :, None, :, None]
        return (_codes(blocks / sc).float() * sc).view(b, -1, hkv, d)[:, :t].permute(0, 2, 1, 3)

    k, v = (torch.cat([past(s[n + "_cache"], s[n + "_scales"]), new(s[n + "_new"])], 2) for n in "kv")
    q = s["q"].float().view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    slots = k.shape[2] - t
    up = torch.zeros(b, t, t + 1, dtype=torch.float64, device=q.device)
    up.scatter_(2, torch.where(s["parents"] < 0, t, s["parents"]).long()[:, :, None], 1.0)
    up = torch.linalg.matrix_power(up[:, :, :t] + torch.eye(t, dtype=torch.float64, device=q.device), 64) > 0
    sees = torch.cat([(torch.arange(slots, device=q.device) < s["lens"][:, None])[:, None, :].expand(b, t, slots), up], 2)
    sees = sees[:, None, :, None, :].expand(b, 1, t, g, slots + t).reshape(b, 1, t * g, slots + t)
    scores = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] or d ** -0.5)
    scores = scores.masked_fill(~sees, -math.inf)
    p = torch.exp(scores - scores.amax(3, keepdim=True))
    out = torch.matmul(p, v) / p.sum(3, keepdim=True)
    return out.view(b, hkv, t, g, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(s["q"].dtype)


def _rotate(x, cos, sin):
    lo, hi = x.chunk(2, -1)
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _run_append(s):
    caches = [s["k_cache"], s["v_cache"]] + ([s["k_scales"], s["v_scales"]] if s["cache"] == "block8" else [])
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        block = s["cache"] == "block8"
        mt.kv_append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["offsets"], status_ws=s["status"],
                           rope=s["rot"][2] if s["rot"] else None, k_scales=s["k_scales"] if block else None, v_scales=s["v_scales"] if block else None,
                           k_scale=1 / 32, v_scale=1 / 32)
        return caches
    row = torch.arange(s["k"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["offsets"], row, right=True) - 1
    slot = (s["lens"][b] + row - s["offsets"][b]).long()
    page, at = s["table"][b, slot // P].long(), slot % P
    k, v, dt = s["k"].float(), s["v"].float(), s["k"].dtype
    if s["rot"]:
        k = _rotate(k, s["rot"][0][slot][:, None], s["rot"][1][slot][:, None]).to(dt).float()
    for x, cache, scales in ((k, s["k_cache"], s.get("k_scales")), (v, s["v_cache"], s.get("v_scales"))):
        if s["cache"] == "act":
            cache[page, :, at] = x.to(dt)
        elif s["cache"] == "e4m3":
            cache.view(torch.uint8)[page, :, at] = _codes(x / (1 / 32)).view(torch.uint8)
        else:
            new = torch.full_like(scales, -1.0).scatter_reduce_(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
            first = torch.full((cache.shape[0],), P, device="cuda").scatter_reduce_(0, page, at, "amin")  # a page's first new slot
            fresh = torch.where(new < 0, 0.0, _pow2(_exponent(new.clamp(min=0))))
            grown = torch.where((first > 0)[:, None], torch.maximum(scales, fresh), fresh)
            # pages that were partly full: their earlier rows under the new scale
            part = s["table"].gather(1, (s["lens"] // P).clamp(max=s["table"].shape[1] - 1).long()[:, None])[:, 0]
            part = part[(s["offsets"][1:] > s["offsets"][:-1]) & (s["lens"] % P > 0)].long()
            again = _codes(cache[part].float() * (scales[part] / grown[part])[:, :, None, None])
            keep = (torch.arange(P, device="cuda") < first[part][:, None])[:, None, :, None]
            cache.view(torch.uint8)[part] = torch.where(keep, again.view(torch.uint8), cache[part].view(torch.uint8))
            scales.copy_(grown)
            cache.view(torch.uint8)[page, :, at] = _codes(x / scales[page][..., None]).view(torch.uint8)
    return caches


def _run_norm_rope(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        return mt.qk_norm_rope(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], rope=s["rot"][2] if s["rot"] else None, q_weight=s["qw"],
                               k_weight=s["kw"], eps=EPS, status_ws=s["status"])
    outs = []
    for x, w in ((s["q"].float(), s["qw"]), (s["k"].float(), s["kw"])):
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        if s["rot"]:
            p = s["positions"].long()
            x = _rotate(x, s["rot"][0][p][:, None], s["rot"][1][p][:, None])
        outs.append(x.to(s["q"].dtype))
    return outs


def _run_sample(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        return mt.sample_tokens(s["logits"], s["uniforms"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    x = s["logits"].double()  # a draw lies next to some border: sums in 64 bits
    n, v = x.shape
    t = s["temperature"].double()[:, None]
    x, index = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    mass = w.cumsum(1)
    rank = torch.arange(v, device="cuda")
    k = torch.where((s["top_k"] <= 0) | (s["top_k"] > v), v, s["top_k"])[:, None]
    k = torch.where(t > 0, k, 1)
    p = s["top_p"].double()[:, None]
    whole = mass.gather(1, k.long() - 1)
    keep = (rank < k) & ((mass - w < p * whole) | (p >= 1)) & (w >= s["min_p"].double()[:, None])
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, index, torch.where(keep, w, 0.0)).cumsum(1)
    at = (kept <= s["uniforms"].double()[:, None] * kept[:, -1:]).sum(1)
    return at.to(torch.int32)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "attn":
        lens = _lengths(c["B"], c["lo"], c["hi"])
        e, t, d = BYTES[c["dtype"]], c["T"], c["D"]
        cache = int(lens.sum()) * c["Hkv"] * d * 2 + int((-(-lens // P)).sum()) * (c["Hkv"] * 8 + 4)
        rows = c["B"] * t * d * e * (2 * c["Hq"] + 2 * c["Hkv"]) + c["B"] * (4 * t + 4)
        return {"bytes": cache + rows, "flops": 4 * t * c["Hq"] * d * int((lens + t).sum())}
    if op == "append":
        n = int(_lengths(c["B"], c["lo"], c["hi"]).sum())
        e = BYTES[c["dtype"]]
        out = e if c["cache"] == "act" else 1
        pages = n / P + c["B"]
        return {"bytes": n * c["Hkv"] * c["D"] * 2 * (e + out) + n * c["D"] * 4 * c["rope"] + pages * 4 + pages * c["Hkv"] * 8 * (c["cache"] == "block8") + 8 * c["B"],
                "flops": n * c["Hkv"] * c["D"] * 4}
    if op == "norm_rope":
        h = (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": c["N"] * (h * 2 * BYTES[c["dtype"]] + 4 + c["D"] * 4 * c["rope"]), "flops": c["N"] * h * 7}
    return {"bytes": c["N"] * (c["V"] * BYTES[c["dtype"]] + 24), "flops": c["N"] * c["V"] * 4}


# ---------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "norm_rope": _exact_norm_rope, "sample": _exact_sample}[case["op"]](s)


def _scale_of(largest):
    """The block scale of one largest magnitude, from the definition."""
    k = -64
    while k < 119 and largest > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def _to_code(x):
    """x to the nearest 8-bit value (3 bits of fraction, exponents from -6, steps of 2^-9 below; ties to even), as 64 bits."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))) / 8
    return torch.round(x / step) * step


def _exact_attn(s):
    b, t, hq, hkv, d = s["B"], s["T"], s["Hq"], s["Hkv"], s["D"]
    g, lens, parents, table = hq // hkv, s["lens"].tolist(), s["parents"].tolist(), s["table"].tolist()
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device="cuda")
    for i in range(b):
        sees = torch.zeros(t, t, dtype=torch.bool)
        for a in range(t):
            node = a
            while node >= 0:
                sees[a, node] = True
                node = parents[i][node]
        sees = torch.cat([torch.ones(t, lens[i], dtype=torch.bool), sees], 1).cuda()
        both = []
        for n in "kv":
            pages = torch.tensor(table[i][:-(-lens[i] // P)], dtype=torch.long, device="cuda")
            x = s[n + "_cache"][pages].double() * s[n + "_scales"][pages].double()[:, :, None, None]
            x = x.transpose(1, 2).reshape(-1, hkv, d)[:lens[i]]
            new = s[n + "_new"][i].double()
            parts = [x]
            for a in range(0, t, P):
                block = new[a:a + P]
                sc = torch.tensor([_scale_of(m) for m in block.abs().amax((0, 2)).tolist()], dtype=torch.float64, device="cuda")[:, None]
                parts.append(_to_code(block / sc) * sc)
            both.append(torch.cat(parts))
        k, v = both
        for h in range(hkv):
            q = s["q"][i, :, h * g:(h + 1) * g].double()
            z = torch.einsum("tgd,nd->tgn", q, k[:, h]) * (s["scale"] or 1 / math.sqrt(d))
            z = torch.softmax(z.masked_fill(~sees[:, None, :], -math.inf), 2)
            out[i, :, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", z, v[:, h])
    return out


def _exact_append(s):
    if s["k"].shape[0] * s["Hkv"] * s["D"] > 60e6 or s["k"].shape[0] / P + s["B"] > 5000:
        return None
    offsets, lens, table = s["offsets"].tolist(), s["lens"].tolist(), s["table"].tolist()
    caches, scales = [s["k_cache"].double(), s["v_cache"].double()], [s["k_scales"].double(), s["v_scales"].double()] if s["cache"] == "block8" else []
    n, d, dt = s["k"].shape[0], s["D"], s["k"].dtype
    k = s["k"].double()
    if s["rot"]:
        slot = torch.cat([torch.arange(lens[b], lens[b] + offsets[b + 1] - offsets[b]) for b in range(s["B"])]).cuda().double()
        angle = slot[:, None, None] * ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        lo, hi = k[..., :d // 2], k[..., d // 2:]
        k = torch.cat([lo * angle.cos() - hi * angle.sin(), hi * angle.cos() + lo * angle.sin()], 2)
        if s["cache"] != "act":  # the codes are those of the rotated key in the activations' type
            k = k.to(dt).double()
    for w, x in enumerate((k, s["v"].double())):
        for b in range(s["B"]):
            i, end = 0, offsets[b + 1] - offsets[b]
            while i < end:
                slot = lens[b] + i
                page, at = table[b][slot // P], slot % P
                m = min(P - at, end - i)
                rows = x[offsets[b] + i:offsets[b] + i + m].transpose(0, 1)  # [Hkv][m][D]
                if s["cache"] == "act":
                    caches[w][page, :, at:at + m] = rows
                elif s["cache"] == "e4m3":
                    caches[w][page, :, at:at + m] = _to_code(rows * 32)
                else:
                    sc = torch.tensor([_scale_of(v) for v in rows.abs().amax((1, 2)).tolist()], dtype=torch.float64, device="cuda")
                    if at:
                        old = scales[w][page].clone()
                        sc = torch.maximum(sc, old)
                        caches[w][page, :, :at] = _to_code(caches[w][page, :, :at] * (old / sc)[:, None, None])
                    scales[w][page] = sc
                    caches[w][page, :, at:at + m] = _to_code(rows / sc[:, None, None])
                i += m
    return caches + scales


def _exact_norm_rope(s):
    d, outs = s["D"], []
    for x, w in ((s["q"].double(), s["qw"]), (s["k"].double(), s["kw"])):
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w.double()
        if s["rot"]:
            angle = s["positions"].double()[:, None, None] * ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
            lo, hi = x[..., :d // 2], x[..., d // 2:]
            x = torch.cat([lo * angle.cos() - hi * angle.sin(), hi * angle.cos() + lo * angle.sin()], -1)
        outs.append(x)
    return outs


def _exact_sample(s):
    tokens = []
    for i in range(s["N"]):
        x, t = s["logits"][i].double().cpu().numpy(), float(s["temperature"][i])
        if not t > 0:
            tokens.append(int(np.argmax(x)))
            continue
        w = np.exp((x - x.max()) / t)
        order = np.lexsort((np.arange(len(x)), -x))
        k = int(s["top_k"][i])
        order = order[:k] if k > 0 else order
        ws = w[order]
        before = np.cumsum(ws) - ws
        keep = w[order] >= float(s["min_p"][i])
        if float(s["top_p"][i]) < 1:
            keep &= before < float(s["top_p"][i]) * ws.sum()
        keep[0] = True
        kept = np.sort(order[keep])
        mass = np.cumsum(w[kept])
        tokens.append(int(kept[min(len(kept) - 1, np.searchsorted(mass, float(s["uniforms"][i]) * mass[-1], side="right"))]))
    return torch.tensor(tokens, dtype=torch.int32)
