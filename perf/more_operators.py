"""Cases of the operators that keep a long-running sequence's cache small and shape its answers: their inputs, their
plain form in elementary torch operations (32 bits, 64 where 32 lose what matters), the framework's calls, and their
definition in 64 bits.

  window   tree_attn_paged_block8 with a sliding window and sinks, and the rows' log-sum-exp
  weights  kv_attn_weights: the attention weight that every cached slot has received
  evict    kv_evict: the slots worth keeping, by weight, into new pages
  logits   process_logits: penalties for repeated tokens, biases, grammar masks
"""
import math

import numpy as np
import torch

own = False

P = 16  # slots per page
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one long conversation's next token under a window: latency alone
        dict(name="window_decode_b1", op="window", dtype="f16", B=1, T=1, Hq=32, Hkv=32, D=128, lo=32768, hi=32768, window=2048, sinks=4, chain=True),
        # a decoding batch of long ragged conversations, one token each
        dict(name="window_decode_b64", op="window", dtype="bf16", B=64, T=1, Hq=32, Hkv=8, D=128, lo=256, hi=100000, window=4096, sinks=4, chain=True),
        # 64-node trees over long conversations
        dict(name="window_tree_b16", op="window", dtype="bf16", B=16, T=64, Hq=32, Hkv=8, D=128, lo=512, hi=32768, window=4096, sinks=16, chain=False),
        # one sequence's step, weighed
        dict(name="weights_decode_b1", op="weights", dtype="f16", B=1, T=1, Hq=32, Hkv=8, D=128, lo=4096, hi=4096, path=0, decay=1.0),
        # a decoding batch's step, older weights fading
        dict(name="weights_decode_b64", op="weights", dtype="bf16", B=64, T=1, Hq=32, Hkv=8, D=128, lo=256, hi=8192, path=0, decay=0.99),
        # the accepted paths of a serving batch's 64-node trees
        dict(name="weights_path_b16", op="weights", dtype="bf16", B=16, T=64, Hq=32, Hkv=8, D=128, lo=512, hi=8192, path=5, decay=1.0),
        # chunks of 64 prompt tokens, every token's row weighed
        dict(name="weights_chunk_b8", op="weights", dtype="bf16", B=8, T=64, Hq=32, Hkv=8, D=128, lo=4096, hi=16384, path=0, decay=1.0),
        # one sequence back to its budget
        dict(name="evict_b1", op="evict", dtype="bf16", cache="block8", B=1, Hkv=8, D=128, lo=4224, hi=4224, budget=4096, sinks=4, recent=512),
        # a batch back to its budget, block-scaled cache
        dict(name="evict_b64", op="evict", dtype="bf16", cache="block8", B=64, Hkv=8, D=128, lo=3000, hi=4224, budget=4096, sinks=4, recent=512),
        # long prompts cut to an eighth, 16-bit cache
        dict(name="evict_prompt_b16", op="evict", dtype="bf16", cache="act", B=16, Hkv=8, D=128, lo=4000, hi=16384, budget=2048, sinks=16, recent=256),
        # one row at the tests' vocabulary
        dict(name="logits_b1", op="logits", dtype="f32", B=1, T=1, V=32000, hist=1000, bias=0, masks=0),
        # trees of a serving batch, a third of the rows under a grammar
        dict(name="logits_tree_b16", op="logits", dtype="bf16", B=16, T=64, V=32000, hist=4096, bias=20, masks=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "weights", "evict", "logits"])
    if op == "window":
        hkv, g, t = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([1, 1, 2, 5, rng.randint(3, 64)])
        b, d, window = _log(rng, 1, 64), rng.choice([64, 128, 128]), _log(rng, 1, 8192)
        hi = _log(rng, 16, 100000)
        window = int(max(1, min(window, 1.5e8 // (hkv * d * b), 3e10 // (4 * t * hkv * g * d * b))))
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), B=b, T=t, Hq=hkv * g, Hkv=hkv, D=d, lo=rng.choice([0, hi // 2, hi]), hi=hi, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 37]), chain=rng.random() < 0.4)
    if op == "weights":
        hkv, g, t = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([1, 1, 2, 5, rng.randint(3, 64)])
        b, d = _log(rng, 1, 64), rng.choice([64, 128, 128])
        hi = _log(rng, 16, 32768)
        hi = int(max(1, min(hi, 2e8 // (hkv * d * b), 2e10 // (4 * t * hkv * g * d * b))))
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), B=b, T=t, Hq=hkv * g, Hkv=hkv, D=d, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                    path=rng.choice([0, min(t, 4)]), decay=rng.choice([1.0, 0.95]))
    if op == "evict":
        hkv, b, d = rng.choice([1, 2, 3, 8, 8, 32]), _log(rng, 1, 64), rng.choice([64, 128])
        hi = _log(rng, 16, 32768)
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        hi = int(max(16, min(hi, 2.4e8 // (hkv * d * b * BYTES[dtype]))))
        budget = max(1, int(hi * rng.choice([0.1, 0.5, 0.9, 0.98])))
        return dict(op=op, dtype=dtype, cache=rng.choice(["act", "e4m3", "block8", "block8"]), B=b, Hkv=hkv, D=d, lo=rng.choice([0, hi]), hi=hi,
                    budget=budget, sinks=rng.choice([0, min(4, budget // 4)]), recent=rng.choice([0, budget // 8, budget // 2]))
    v = _log(rng, 1000, 200000)
    if rng.random() < 0.5:
        v = v // 8 * 8
    t = rng.choice([1, 1, 1, 5, 26, 64])
    return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), B=max(1, min(_log(rng, 1, 128), 20000000 // (v * t))), T=t, V=v, hist=rng.choice([0, 50, _log(rng, 10, 10000)]),
                bias=rng.choice([0, 20]), masks=rng.choice([0, 3, 20]))


# ---------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(b, lo, hi):
    """b lengths of [lo, hi], the largest of them hi: the same ones for every seed, which orders them."""
    n = np.random.default_rng(1).integers(lo, hi + 1, size=b)
    n[0] = hi
    return n


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _fill(rng, table, first, last, pages, at):
    """Entries first .. last - 1 of each row from a shuffled pool of pages; returns how many are used."""
    for b in range(len(table)):
        n = last[b] - first[b]
        table[b, first[b]:last[b]] = pages[at:at + n]
        at += n
    return at


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
    return {"window": _prepare_window, "weights": _prepare_weights, "evict": _prepare_evict, "logits": _prepare_logits}[case["op"]](case, seed)


def _prepare_window(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, t, hq, hkv, d, dt = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    lens = rng.permutation(_lengths(b, c["lo"], c["hi"]))
    # only the pages that the window and the sinks reach are still held
    blocks = -(-lens // P)
    sink_blocks = -(-np.minimum(lens, c["sinks"]) // P)
    first = np.maximum(np.maximum(lens - c["window"] + 1, 0) // P, sink_blocks)
    table = np.full((b, max(1, int(blocks.max()))), -1, np.int32)
    pages = int((sink_blocks + blocks - first).sum()) + 3
    pool = rng.permutation(pages)
    _fill(rng, table, first, blocks, pool, _fill(rng, table, np.zeros_like(blocks), sink_blocks, pool, 0))
    k, ks = _block_cache(g, pages, hkv, d, dt, True)
    v, vs = _block_cache(g, pages, hkv, d, dt, False)
    s = dict(c, k_cache=k, v_cache=v, k_scales=ks, v_scales=vs, table=_i32(table), lens=_i32(lens), host_lens=lens, q=_randn(g, b, t, hq, d).to(dt),
             parents=None if c["chain"] else _i32(np.stack([_tree(rng, t) for _ in range(b)])), k_new=_randn(g, b, t, hkv, d).to(dt), v_new=_randn(g, b, t, hkv, d).to(dt))
    # slots that the first node sees, side by side: what the plain form gathers
    reach = [np.concatenate([np.arange(min(c["sinks"], max(n - c["window"] + 1, 0))), np.arange(max(n - c["window"] + 1, 0), n)]) for n in lens]
    most = max(1, max(len(r) for r in reach))
    s["reach"] = _i32(np.stack([np.pad(r, (0, most - len(r)), constant_values=-1) for r in reach])).long()
    s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(b, t, hq, device="cuda")
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        s["workspace"] = mt.alloc_block8_workspace(s["q"], s["k_cache"], s["table"])
    return s


def _prepare_weights(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, t, hq, hkv, d, dt = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    lens = rng.permutation(_lengths(b, c["lo"], c["hi"]))
    blocks = -(-lens // P)
    table = np.full((b, max(1, int(blocks.max()))), -1, np.int32)
    pages = int(blocks.sum()) + 3
    _fill(rng, table, np.zeros_like(blocks), blocks, rng.permutation(pages), 0)
    k, ks = _block_cache(g, pages, hkv, d, dt, True)
    s = dict(c, k_cache=k, k_scales=ks, table=_i32(table), lens=_i32(lens), host_lens=lens, q=_randn(g, b, t, hq, d).to(dt))
    s["path"] = s["path_len"] = None
    if c["path"]:
        s["path"] = _i32(np.sort(np.stack([np.concatenate([[0], 1 + rng.permutation(t - 1)[:c["path"] - 1]]) for _ in range(b)]), 1))
        s["path_len"] = _i32(rng.integers(0, c["path"], b))
    s["weights"] = torch.rand(pages, hkv, P, generator=g, device="cuda") * 0.1
    s["prev"] = _i32(np.maximum(lens - 1 - rng.integers(0, 70, b), 0))  # slots that were weighed before
    s["out"] = torch.zeros_like(s["weights"])
    # the attention's log-sum-exp, over the cached slots
    s["lse"] = torch.zeros(b, t, hq, device="cuda")
    for i in range(b):
        n = int(lens[i])
        if n:
            at = s["table"][i, :blocks[i]].long()
            x = (k[at].float() * ks[at][:, :, None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, :n]
            z = torch.matmul(s["q"][i].float().view(t, hkv, hq // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d), x.transpose(1, 2)) * d ** -0.5
            s["lse"][i] = torch.logsumexp(z, 2).view(hkv, t, hq // hkv).permute(1, 0, 2).reshape(t, hq)
    if own:
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _prepare_evict(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, hkv, d, dt = c["B"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    lens = rng.permutation(_lengths(b, c["lo"], c["hi"]))
    blocks, after = -(-lens // P), -(-np.minimum(lens, c["budget"]) // P)
    pages = int((blocks + after).sum()) + 3
    pool = rng.permutation(pages)
    table, to = np.full((b, max(1, int(blocks.max()))), -1, np.int32), np.full((b, -(-c["budget"] // P)), -1, np.int32)
    zero = np.zeros_like(blocks)
    _fill(rng, to, zero, after, pool, _fill(rng, table, zero, blocks, pool, 0))
    s = dict(c, table=_i32(table), new_table=_i32(to), lens=_i32(lens), host_lens=lens, k_scales=None, v_scales=None)
    if c["cache"] == "block8":
        s["k_cache"], s["k_scales"] = _block_cache(g, pages, hkv, d, dt, True)
        s["v_cache"], s["v_scales"] = _block_cache(g, pages, hkv, d, dt, False)
    else:
        s["k_cache"], s["v_cache"] = (torch.randn(pages, hkv, P, d, generator=g, device="cuda", dtype=dt) for _ in range(2))
        if c["cache"] == "e4m3":
            s["k_cache"], s["v_cache"] = _codes(s["k_cache"].float() * 32), _codes(s["v_cache"].float() * 32)
    # most slots have received next to nothing, some of them nothing at all
    w = torch.exp(2 * _randn(g, pages, hkv, P) - 4)
    s["weights"] = torch.where(torch.rand(pages, hkv, P, generator=g, device="cuda") < 0.1, 0.0, w)
    s["kept"] = torch.zeros(b, hkv, c["budget"], dtype=torch.int32, device="cuda")
    if own:
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _prepare_logits(c, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    b, t, v = c["B"], c["T"], c["V"]
    x = 2.5 * _randn(g, b, t, v)
    hist_lens = rng.integers(c["hist"] // 2, c["hist"] + 1, b)
    # tokens repeat as words do: rank r about 1 / r of the time
    zipf = lambda *shape: np.minimum((v ** rng.random(shape)).astype(np.int64) * 7919 % v, v - 1)  # noqa: E731
    s = dict(c, logits=x.to(TYPES[c["dtype"]]), history=_i32(zipf(b, max(1, c["hist"]))), history_lens=_i32(hist_lens), output_starts=_i32(hist_lens * rng.random(b)))
    f32 = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    s["repetition"], s["presence"], s["frequency"] = f32(rng.choice([1.0, 1.1, 1.3], b)), f32(rng.choice([0.0, 0.5, 1.5], b)), f32(rng.choice([0.0, 0.1, 0.7], b))
    s["bias_tokens"] = s["bias_values"] = s["mask"] = s["mask_index"] = s["tree_tokens"] = s["tree_parents"] = None
    if c["bias"]:
        s["bias_tokens"], s["bias_values"] = _i32(np.where(rng.random((b, c["bias"])) < 0.2, -1, zipf(b, c["bias"]))), f32(5 * rng.standard_normal((b, c["bias"])))
    if c["masks"]:  # a grammar's states allow few tokens or most; two rows in three are free
        share = rng.choice([0.001, 0.05, 0.9], (c["masks"], 1))
        bits = rng.random((c["masks"], -(-v // 32) * 32), dtype=np.float32) < share
        s["mask"] = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).cuda()
        s["mask_index"] = _i32(np.where(rng.random((b, t)) < 1 / 3, rng.integers(0, c["masks"], (b, t)), -1))
    if t > 1:
        s["tree_tokens"], s["tree_parents"] = _i32(zipf(b, t)), _i32(np.stack([_tree(rng, t) for _ in range(b)]))
    s["out"] = torch.empty_like(s["logits"])
    if own:
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    return {"window": _run_window, "weights": _run_weights, "evict": _run_evict, "logits": _run_logits}[s["op"]](s)


def _ancestors(parents, t):
    """[B][T][T]: node j is i or above it."""
    up = torch.zeros(len(parents), t, t + 1, dtype=torch.float64, device="cuda")
    up.scatter_(2, torch.where(parents < 0, t, parents).long()[:, :, None], 1.0)
    return torch.linalg.matrix_power(up[:, :, :t] + torch.eye(t, dtype=torch.float64, device="cuda"), 64) > 0


def _run_window(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        mt.tree_attn_paged_block8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["lens"], s["parents"], s["out"], k_new=s["k_new"],
                                  v_new=s["v_new"], workspace=s["workspace"], window=s["window"], sinks=s["sinks"], lse=s["lse"])
        return s["out"], s["lse"]
    b, t, hq, hkv, d, w = s["B"], s["T"], s["Hq"], s["Hkv"], s["D"], s["window"]
    g, reach, n = hq // hkv, s["reach"], s["reach"].shape[1]
    page, at = s["table"].gather(1, reach.clamp(min=0) // P).clamp(min=0).long(), reach % P

    def past(cache, scales):
        return (cache.view(torch.uint8)[page, :, at].view(F8).float() * scales[page][..., None]).transpose(1, 2)  # [B][Hkv][n][D]

    def new(x):
        blocks = torch.zeros(b, -(-t // P) * P, hkv, d, device=x.device)
        blocks[:, :t] = x
        blocks = blocks.view(b, -1, P, hkv, d)
        sc = _pow2(_exponent(blocks.abs().amax((2, 4))))[:, :, None, :, None]
        return (_codes(blocks / sc).float() * sc).view(b, -1, hkv, d)[:, :t].transpose(1, 2)

    k, v = (torch.cat([past(s[x + "_cache"], s[x + "_scales"]), new(s[x + "_new"])], 2) for x in "kv")
    above = torch.ones(t, t, device="cuda").tril().bool().expand(b, t, t) if s["parents"] is None else _ancestors(s["parents"], t)
    place = s["lens"][:, None].long() + above.sum(2) - 1  # [B][T] a node's position
    seen = lambda pos: (pos < s["sinks"]) | (pos > place[:, :, None] - w)  # noqa: E731
    sees = torch.cat([(reach >= 0)[:, None, :] & seen(reach[:, None, :]), above & seen(place[:, None, :])], 2)[:, None, :, None, :]
    q = s["q"].float().view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    z = (torch.matmul(q, k.transpose(2, 3)) * d ** -0.5).view(b, hkv, t, g, n + t).masked_fill(~sees, -math.inf)
    top = z.amax(4, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(4, keepdim=True)
    out = torch.matmul(p.view(b, hkv, t * g, n + t), v).view(b, hkv, t, g, d) / total
    lse = (top + torch.log(total)).squeeze(4)
    return out.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(b, t, hq)


def _run_weights(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        return mt.kv_attn_weights(s["q"], s["k_cache"], s["k_scales"], s["table"], s["lens"], s["lse"], s["weights"], out=s["out"], prev_lens=s["prev"],
                                  accept_path=s["path"], accept_len=s["path_len"], decay=s["decay"], status_ws=s["status"])
    b, t, hq, hkv, d = s["B"], s["T"], s["Hq"], s["Hkv"], s["D"]
    g, pages = hq // hkv, s["table"].clamp(min=0).long()
    q, lse = s["q"].float(), s["lse"]
    counts = torch.ones(b, t, device="cuda")
    if s["path"] is not None:
        q = q.gather(1, s["path"].long()[:, :, None, None].expand(-1, -1, hq, d))
        lse = lse.gather(1, s["path"].long()[:, :, None].expand(-1, -1, hq))
        t = q.shape[1]
        counts = (torch.arange(t, device="cuda") <= s["path_len"][:, None]).float()
    k = (s["k_cache"][pages].float() * s["k_scales"][pages][..., None, None]).transpose(1, 2).reshape(b, hkv, -1, d)
    q = q.view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    z = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    p = torch.exp(z - lse.view(b, t, hkv, g).permute(0, 2, 1, 3).reshape(b, hkv, t * g, 1)) * counts[:, None, :, None].expand(b, hkv, t, g).reshape(b, hkv, t * g, 1)
    slot = torch.arange(k.shape[2], device="cuda")
    old = torch.where((slot < s["prev"][:, None])[:, None, :], s["weights"][pages].transpose(1, 2).reshape(b, hkv, -1), 0.0)
    new = (old * s["decay"] + p.sum(2)).transpose(1, 2)  # [B][slots][Hkv]
    live = slot < s["lens"][:, None]
    at = (pages[:, :, None] * P + torch.arange(P, device="cuda")).view(b, -1)
    out = s["out"].transpose(1, 2).reshape(-1, hkv)
    out[at[live]] = new[live]
    s["out"].copy_(out.view(-1, P, hkv).transpose(1, 2))
    return s["out"]


def _run_evict(s):
    outs = [s["kept"], s["weights"], s["k_cache"], s["v_cache"]] + ([s["k_scales"], s["v_scales"]] if s["cache"] == "block8" else [])
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        mt.kv_evict(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["lens"], s["new_table"], s["kept"], sinks=s["sinks"], recent=s["recent"], k_scales=s["k_scales"],
                    v_scales=s["v_scales"], status_ws=s["status"])
        return outs
    b, hkv, budget = s["B"], s["Hkv"], s["budget"]
    pages, n = s["table"].clamp(min=0).long(), s["lens"][:, None, None]
    slot = torch.arange(max(pages.shape[1] * P, budget), device="cuda")
    w = s["weights"][pages].transpose(1, 2).reshape(b, hkv, -1)
    w = torch.nn.functional.pad(w, (0, len(slot) - w.shape[2]))
    w = torch.where((slot < s["sinks"]) | (slot >= n - s["recent"]) | (n <= budget), math.inf, w)
    w = torch.where(slot < n, w, -math.inf)
    order = torch.sort(w, dim=2, descending=True, stable=True)[1][:, :, :budget]
    kept = torch.where(order < n, order, len(slot)).sort(2)[0]
    there = kept < len(slot)
    s["kept"].copy_(torch.where(there, kept, -1))
    bi = torch.arange(b, device="cuda")[:, None, None].expand_as(kept)[there]
    hi = torch.arange(hkv, device="cuda")[None, :, None].expand_as(kept)[there]
    to = slot[:budget].expand_as(kept)[there]
    src, dst, here, there = pages[bi, kept[there] // P], s["new_table"][bi, to // P].long(), kept[there] % P, to % P
    s["weights"][dst, hi, there] = s["weights"][src, hi, here]
    for name in "kv":
        cache, scales = s[name + "_cache"], s[name + "_scales"]
        if scales is None:
            raw = cache.view(torch.uint8) if s["cache"] == "e4m3" else cache
            raw[dst, hi, there] = raw[src, hi, here]
            continue
        old = scales[src, hi]
        top = torch.zeros_like(scales).view(-1).scatter_reduce_(0, dst * hkv + hi, old, "amax").view(-1, hkv)
        moved = cache.view(torch.uint8)[src, hi, here].view(F8).float() * (old / top[dst, hi])[:, None]
        cache.view(torch.uint8)[dst, hi, there] = _codes(moved).view(torch.uint8)
        scales[dst, hi] = top[dst, hi]
    return outs


def _run_logits(s):
    if own:
        import medusa_tree_speculative_attn_gb300 as mt
        return mt.process_logits(s["logits"], s["out"], history=s["history"], history_lens=s["history_lens"], output_starts=s["output_starts"], repetition=s["repetition"],
                                 presence=s["presence"], frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], mask=s["mask"],
                                 mask_index=s["mask_index"], tree_tokens=s["tree_tokens"], tree_parents=s["tree_parents"], status_ws=s["status"])
    b, t, v = s["B"], s["T"], s["V"]
    row = torch.arange(b, device="cuda")[:, None] * v
    at = torch.arange(s["history"].shape[1], device="cuda")
    live = at < s["history_lens"][:, None]
    late = (live & (at >= s["output_starts"][:, None])).float()
    flat = (row + s["history"]).view(-1)
    seen = torch.zeros(b * v, device="cuda").index_add_(0, flat, live.float().view(-1)).view(b, 1, v)
    made = torch.zeros(b * v, device="cuda").index_add_(0, flat, late.view(-1)).view(b, 1, v)
    if s["tree_tokens"] is not None:
        above = _ancestors(s["tree_parents"], t).float()
        path = torch.zeros(b, t, v, device="cuda").scatter_add_(2, s["tree_tokens"].long()[:, None, :].expand(b, t, t), above)
        seen, made = seen + path, made + path
    per = lambda a: a[:, None, None]  # noqa: E731
    x = s["logits"].float()
    x = torch.where(seen > 0, torch.where(x > 0, x / per(s["repetition"]), x * per(s["repetition"])), x)
    x = x - per(s["frequency"]) * made - per(s["presence"]) * (made > 0)
    if s["bias_tokens"] is not None:  # of a token named twice the last entry counts
        n = s["bias_tokens"].shape[1]
        entry = torch.where(s["bias_tokens"] < 0, 0, torch.arange(1, n + 1, device="cuda"))
        last = torch.zeros(b * v, dtype=torch.long, device="cuda").scatter_reduce_(0, (row + s["bias_tokens"].clamp(min=0)).view(-1), entry.view(-1), "amax").view(b, v)
        x = x + torch.nn.functional.pad(s["bias_values"], (1, 0)).gather(1, last)[:, None]
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).view(s["mask"].shape[0], -1)[:, :v] > 0
        allowed = bits[s["mask_index"].clamp(min=0).long()] | (s["mask_index"] < 0)[:, :, None]
        x = x.masked_fill(~allowed, -math.inf)
    return s["out"].copy_(x.to(s["logits"].dtype))


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "logits":
        rows, e = c["B"] * c["T"], BYTES[c["dtype"]]
        masked = rows / 3 * c["V"] / 8 if c["masks"] else 0
        return {"bytes": rows * c["V"] * 2 * e + c["B"] * (3 * c["hist"] + 8 * c["bias"] + 20) + masked + rows * 12, "flops": rows * c["V"]}
    lens = _lengths(c["B"], c["lo"], c["hi"])
    if op == "window":
        far = np.maximum(lens - c["window"] + 1, 0)
        n = int((lens - far + np.minimum(far, c["sinks"])).sum())
        rows = c["B"] * c["T"] * (c["D"] * 2 * (2 * c["Hq"] + 2 * c["Hkv"]) + c["Hq"] * 4 + 4)
        return {"bytes": n * c["Hkv"] * (c["D"] * 2 + 0.5) + n / P * 4 + rows, "flops": 4 * c["T"] * c["Hq"] * c["D"] * (n + c["B"] * c["T"] // 2)}
    if op == "weights":
        n, t = int(lens.sum()), (c["path"] + 1) / 2 if c["path"] else c["T"]
        return {"bytes": n * c["Hkv"] * (c["D"] + 8 + 0.25) + n / P * 4 + c["B"] * t * c["Hq"] * (2 * c["D"] + 4), "flops": 2 * t * c["Hq"] * c["D"] * n}
    n, m = int(lens.sum()), int(np.minimum(lens, c["budget"]).sum())
    e = BYTES[c["dtype"]] if c["cache"] == "act" else 1
    return {"bytes": n * c["Hkv"] * 4 + m * c["Hkv"] * (4 * c["D"] * e + 8 + (c["cache"] == "block8")) + (n + m) / P * 4, "flops": n * c["Hkv"] * 4}


# ---------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_window, "weights": _exact_weights, "evict": _exact_evict, "logits": _exact_logits}[case["op"]](s)


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


def _exact_window(s):
    b, t, hq, hkv, d, w, sinks = s["B"], s["T"], s["Hq"], s["Hkv"], s["D"], s["window"], s["sinks"]
    g, lens = hq // hkv, s["lens"].tolist()
    table = s["table"].cpu()
    out, lse = torch.zeros(b, t, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(b, t, hq, dtype=torch.float64, device="cuda")
    for i in range(b):
        n = lens[i]
        parents = list(range(-1, t - 1)) if s["parents"] is None else s["parents"][i].tolist()
        chains, depth = [], []
        for a in range(t):
            node, chain = a, []
            while node >= 0:
                chain.append(node)
                node = parents[node]
            chains.append(chain)
            depth.append(len(chain) - 1)
        slots = [p for p in range(n) if p < sinks or p > n - w]
        sees = torch.zeros(t, len(slots) + t, dtype=torch.bool)
        pos = torch.tensor(slots, dtype=torch.long)
        for a in range(t):
            sees[a, :len(slots)] = (pos < sinks) | (pos > n + depth[a] - w)
            for node in chains[a]:
                sees[a, len(slots) + node] = n + depth[node] < sinks or depth[node] > depth[a] - w
        sees, both = sees.cuda(), []
        page, at = table[i][pos // P].long().cuda(), (pos % P).cuda()
        for x in "kv":
            parts = [s[x + "_cache"].view(torch.uint8)[page, :, at].view(F8).double() * s[x + "_scales"][page].double()[:, :, None]]
            new = s[x + "_new"][i].double()
            for a in range(0, t, P):
                block = new[a:a + P]
                sc = torch.tensor([_scale_of(m) for m in block.abs().amax((0, 2)).tolist()], dtype=torch.float64, device="cuda")[:, None]
                parts.append(_to_code(block / sc) * sc)
            both.append(torch.cat(parts))
        k, v = both
        for h in range(hkv):
            z = torch.einsum("tgd,nd->tgn", s["q"][i, :, h * g:(h + 1) * g].double(), k[:, h]) / math.sqrt(d)
            z = z.masked_fill(~sees[:, None, :], -math.inf)
            lse[i, :, h * g:(h + 1) * g] = torch.logsumexp(z, 2)
            out[i, :, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", torch.softmax(z, 2), v[:, h])
    return out, lse


def _exact_weights(s):
    hq, hkv, d = s["Hq"], s["Hkv"], s["D"]
    g, out = hq // hkv, torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        nodes = list(range(s["T"])) if s["path"] is None else s["path"][i].tolist()[:int(s["path_len"][i]) + 1]
        pages = s["table"][i, :-(-n // P)].long()
        k = (s["k_cache"][pages].double() * s["k_scales"][pages].double()[:, :, None, None]).transpose(1, 2).reshape(-1, hkv, d)[:n]
        w = s["weights"][pages].double().transpose(1, 2).reshape(-1, hkv)[:n] * s["decay"]
        w[int(s["prev"][i]):] = 0
        for h in range(hkv):
            z = torch.einsum("tgd,nd->tgn", s["q"][i, nodes, h * g:(h + 1) * g].double(), k[:, h]) / math.sqrt(d)
            w[:, h] += torch.exp(z - s["lse"][i, nodes, h * g:(h + 1) * g].double()[:, :, None]).sum((0, 1))
        slot = torch.arange(n, device="cuda")
        out[pages[slot // P], :, slot % P] = w
    return out


def _exact_evict(s):
    b, hkv, budget, lens = s["B"], s["Hkv"], s["budget"], s["lens"].tolist()
    weights, caches = s["weights"].double(), [s["k_cache"].double(), s["v_cache"].double()]
    scales = [s["k_scales"].double(), s["v_scales"].double()] if s["cache"] == "block8" else []
    kept = np.full((b, hkv, budget), -1, np.int32)
    for i in range(b):
        n = lens[i]
        if not n:
            continue
        pages = s["table"][i, :-(-n // P)].long()
        w = s["weights"][pages].transpose(1, 2).reshape(-1, hkv)[:n].cpu().numpy()
        m = min(n, budget)
        for h in range(hkv):
            if n <= budget:
                pick = np.arange(n)
            else:
                middle = np.arange(s["sinks"], n - s["recent"])
                best = middle[np.lexsort((middle, -w[middle, h].astype(np.float64)))][:budget - s["sinks"] - s["recent"]]
                pick = np.sort(np.concatenate([np.arange(s["sinks"]), best, np.arange(n - s["recent"], n)]))
            kept[i, h, :m] = pick
            at = torch.from_numpy(pick).cuda()
            src, here = pages[at // P], at % P
            to = torch.arange(m, device="cuda")
            dst, there = s["new_table"][i].long()[to // P], to % P
            weights[dst, h, there] = weights[src, h, here]
            for c, cache in enumerate(caches):
                rows = cache[src, h, here]
                if scales:
                    old = scales[c][src, h]
                    top = torch.nn.functional.pad(old, (0, -m % P)).view(-1, P).amax(1)
                    scales[c][s["new_table"][i].long()[:len(top)], h] = top
                    rows = _to_code(rows * (old / top[to // P])[:, None])
                cache[dst, h, there] = rows
    return [torch.from_numpy(kept), weights] + caches + scales


def _exact_logits(s):
    b, t, v = s["B"], s["T"], s["V"]
    if b * t * (v + 10 * s["hist"]) > 1e8:  # a row at a time on the host
        return None
    out = s["logits"].double().cpu().numpy().copy()
    history, hist_lens, starts = s["history"].cpu().numpy(), s["history_lens"].tolist(), s["output_starts"].tolist()
    rep, pres, freq = (s[n].double().tolist() for n in ("repetition", "presence", "frequency"))
    mask = None if s["mask"] is None else np.unpackbits(s["mask"].cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :v]
    for i in range(b):
        words = history[i, :hist_lens[i]]
        for a in range(t):
            path, node = [], a if s["tree_tokens"] is not None else -1
            while node >= 0:
                path.append(int(_host(s, "tree_tokens")[i][node]))
                node = int(_host(s, "tree_parents")[i][node])
            said = np.concatenate([words[starts[i]:], np.array(path, np.int64)]).astype(np.int64)
            every, x = np.unique(np.concatenate([words, path]).astype(np.int64)), out[i, a]
            x[every] = np.where(x[every] > 0, x[every] / rep[i], x[every] * rep[i])
            tokens, counts = np.unique(said, return_counts=True)
            x[tokens] -= freq[i] * counts + pres[i]
            if s["bias_tokens"] is not None:
                last = {int(k): float(y) for k, y in zip(_host(s, "bias_tokens")[i], _host(s, "bias_values")[i]) if k >= 0}
                for k, y in last.items():
                    x[k] += y
            if mask is not None and _host(s, "mask_index")[i][a] >= 0:
                x[mask[_host(s, "mask_index")[i][a]] == 0] = -math.inf
    return torch.from_numpy(out)


def _host(s, name):
    """A state's tensor as an array on the host, brought there once."""
    if ("host", name) not in s:
        s["host", name] = s[name].cpu().numpy()
    return s["host", name]
