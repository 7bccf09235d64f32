"""The serving operators on the GPU against plain implementations in 64 bits (serve_reference).

Tolerances (u = half a step of the output's type relative to the value: bf16 2^-8, fp16 2^-11, fp32 2^-24):
  norms and rotation  u |y| for the rounding at the end, and 2^-19 of the magnitudes that enter y: a chain of six
                      rounded 32-bit operations (2^-24 each), the reciprocal square root (2^-22), the sum of D
                      squares (a tree of depth <= 16: 2^-20) and the table (2^-24);
  attention           u |out| (output; a split segment's pieces stay in 32 bits) + 2^-11 A (fp16 weights) + 2 E A,
                      A = sum p |v|, E the error of a score in the exponent: D products and sums in 32 bits, which
                      tensor cores may truncate, 2 D 2^-24 sum |q k| scale <= 2^-9 for these inputs;
  codes, scales, values, tokens: equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import medusa_tree_speculative_attn_gb300 as mt
import serve_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
P = 16
BASE = 10000.0


def _status():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _rand(rng, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype)


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32))


def _codes(t):
    return t.cpu().view(torch.uint8).numpy()


def _table(rng, need, pages):
    """A block table with need[b] shuffled pages each, -1 behind them."""
    perm = rng.permutation(pages)
    out = np.full((len(need), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        out[b, :n] = perm[at:at + n]
        at += n
    return out


def _graph(fn):
    """fn captured on a side stream, then replayed once."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fn()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            fn()
    torch.cuda.synchronize()
    return g


# ---- norms and rotation ----------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n, hq, hkv, d", [(1, 1, 1, 64), (3, 8, 2, 128), (17, 5, 5, 64), (64, 32, 8, 128), (5, 9, 3, 128)])
@pytest.mark.parametrize("norm, rope", [(True, True), (True, False), (False, True)])
def test_norm_rope(dtype, n, hq, hkv, d, norm, rope):
    rng = np.random.default_rng(n * 100 + hq)
    dt = DT[dtype]
    x = _rand(rng, n, hq + 2 * hkv, d, dtype=dt, scale=3.0)
    if n > 1:
        x[1] = 0  # a row of zeros
    w = [(1 + 0.2 * _rand(rng, d)).to(dt) for _ in range(2)] if norm else [None, None]
    pos = rng.integers(0, 500, n)
    if n > 2:
        pos[2] = -1  # no token
    pos[0] = 499
    xd = x.cuda()
    q, k = xd[:, :hq], xd[:, hq:hq + hkv]  # views of a projection's rows
    qo, ko = torch.full((n, hq, d), 7.0, dtype=dt, device="cuda"), torch.full((n, hkv, d), 7.0, dtype=dt, device="cuda")
    table = mt.Rope(BASE, d, 500) if rope else None
    ws = _status()
    mt.qk_norm_rope(q, k, _i32(pos).cuda(), qo, ko, rope=table, q_weight=w[0].cuda() if norm else None,
                    k_weight=w[1].cuda() if norm else None, eps=1e-5, status_ws=ws)
    assert mt.read_status(ws) == 0
    cos, sin = ref.rope_table(BASE, d, 500)
    at = np.maximum(pos, 0)
    c, s = (cos[at][:, None], sin[at][:, None]) if rope else (None, None)
    for got, src, wt in ((qo, x[:, :hq], w[0]), (ko, x[:, hq:hq + hkv], w[1])):
        want, mag = ref.norm_rope64(src, wt, 1e-5, c, s)
        got = got.cpu().double()
        tol = ref.HALF_STEP[dt] * want.abs() + 2.0 ** -19 * mag + (2.0 ** -25 if dt == torch.float16 else 0)
        live = torch.from_numpy(pos >= 0)
        assert bool(((got - want).abs() <= tol)[live].all())
        assert bool((got[~live] == 7.0).all())
        if not norm:  # the same bits as the tree attention's own rotation
            assert torch.equal(got[live], ref.rotate32(src, c, s).to(dt).double()[live])


def test_norm_rope_in_place_and_in_a_graph():
    rng = np.random.default_rng(5)
    x = _rand(rng, 40, 6, 128, dtype=torch.bfloat16).cuda()
    want_q, want_k = torch.empty_like(x[:, :4]), torch.empty_like(x[:, 4:])
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos, rope, ws = torch.arange(40, dtype=torch.int32, device="cuda"), mt.Rope(BASE, 128, 64), _status()
    mt.qk_norm_rope(x[:, :4], x[:, 4:], pos, want_q, want_k, rope=rope, q_weight=w, k_weight=w, status_ws=ws)
    y = x.clone()
    mt.qk_norm_rope(y[:, :4], y[:, 4:], pos, y[:, :4], y[:, 4:], rope=rope, q_weight=w, k_weight=w, status_ws=ws)
    assert torch.equal(y[:, :4], want_q) and torch.equal(y[:, 4:], want_k)
    a, b = torch.empty_like(want_q), torch.empty_like(want_k)
    g = _graph(lambda: mt.qk_norm_rope(x[:, :4], x[:, 4:], pos, a, b, rope=rope, q_weight=w, k_weight=w, status_ws=ws))
    a.zero_(), b.zero_()
    g.replay()
    assert torch.equal(a, want_q) and torch.equal(b, want_k)


def test_norm_rope_position_past_the_table():
    x = torch.ones(2, 2, 64, dtype=torch.float16, device="cuda")
    out, ws = torch.full_like(x, 3.0), _status()
    mt.qk_norm_rope(x, x, _i32([10, 3]).cuda(), out, torch.empty_like(x), rope=mt.Rope(BASE, 64, 10), status_ws=ws)
    assert mt.read_status(ws) == -7
    assert bool((out[0] == 3.0).all()) and not bool((out[1] == 3.0).any())


# ---- appending to the cache ------------------------------------------------

class Cache:
    """A seeded cache of one kind, on the GPU, and its copy on the host."""

    def __init__(self, rng, kind, pages, hkv, d, dt):
        self.kind = kind
        if kind == "act":
            k, v = (_rand(rng, pages, hkv, P, d, dtype=dt) for _ in range(2))
        else:  # any code, NaN included, may lie in slots that no sequence holds
            k, v = (torch.from_numpy(rng.integers(0, 256, (pages, hkv, P, d)).astype(np.uint8)).view(torch.float8_e4m3fn) for _ in range(2))
        self.host = [k.clone(), v.clone()]
        self.k, self.v = k.cuda(), v.cuda()
        self.scales = [None, None]
        if kind == "block8":
            self.host_scales = [2.0 ** rng.integers(-8, 3, (pages, hkv)).astype(np.float64) for _ in range(2)]
            self.scales = [torch.from_numpy(s).float().cuda() for s in self.host_scales]

    def args(self):
        return dict(k_scales=self.scales[0], v_scales=self.scales[1], k_scale=0.03, v_scale=0.05)

    def append(self, which, x, page, head, r0):
        """The rows x [m][D] (in the act dtype) into slots r0 .. of a page."""
        m = x.shape[0]
        if self.kind == "act":
            self.host[which][page, head, r0:r0 + m] = x
            return
        codes = self.host[which].view(torch.uint8).numpy()[page, head]
        x = x.double().numpy()
        if self.kind == "e4m3":
            scale = np.float32(0.03 if which == 0 else 0.05)
            codes[r0:r0 + m] = ref.encode((x.astype(np.float32) / scale).astype(np.float64))
            return
        finite = np.abs(x[~np.isnan(x)])
        s = ref.scale_of(finite.max() if finite.size else 0.0)
        if r0:
            old = self.host_scales[which][page, head]
            s = max(s, old)
            if s > old:
                codes[:r0] = ref.encode(ref.decode(codes[:r0]) * (old / s))
        self.host_scales[which][page, head] = s
        codes[r0:r0 + m] = ref.encode(x / s)

    def check(self):
        for got, want in ((self.k, self.host[0]), (self.v, self.host[1])):
            assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
        if self.kind == "block8":
            for got, want in zip(self.scales, self.host_scales):
                assert np.array_equal(got.cpu().double().numpy(), want)


def _append_on_host(cache, k, v, rows_of, lens, table, rot):
    """rows_of(b): the new rows of sequence b."""
    for b in range(len(lens)):
        rows, n = rows_of(b), int(lens[b])
        if n < 0:
            continue
        i = 0
        while i < len(rows):
            slot = n + i
            r0 = slot % P
            m = min(P - r0, len(rows) - i)
            for h in range(k.shape[1]):
                x = k[rows[i:i + m], h]
                if rot is not None:
                    x = ref.rotate32(x, rot[0][slot:slot + m], rot[1][slot:slot + m]).to(k.dtype)
                cache.append(0, x, table[b, slot // P], h, r0)
                cache.append(1, v[rows[i:i + m], h], table[b, slot // P], h, r0)
            i += m


APPENDS = [  # past lengths, new rows
    ([0], [1]), ([0], [16]), ([15], [1]), ([16], [17]), ([5], [60]),
    ([0, 7, -1, 31, 16], [3, 0, 0, 33, 1]), ([100, 3, 47], [1, 1, 1]), ([12, 0], [50, 2]),
]


@pytest.mark.parametrize("kind", ["act", "e4m3", "block8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(kind, dtype, case):
    past, new = APPENDS[case]
    rng = np.random.default_rng(case * 10 + len(dtype))
    dt, hkv, d = DT[dtype], [1, 3, 8][case % 3], [64, 128][case % 2]
    need = [-(-(max(p, 0) + n) // P) for p, n in zip(past, new)]
    table = _table(rng, need, sum(need) + 2)
    cache = Cache(rng, kind, sum(need) + 2, hkv, d, dt)
    off = np.concatenate([[0], np.cumsum(new)])
    n = int(off[-1]) + 2  # two rows behind the last sequence's
    kv = _rand(rng, n, 2, hkv, d, dtype=dt, scale=float(rng.choice([0.01, 1.0, 30.0])))
    rope = mt.Rope(BASE, d, 256) if case % 4 else None
    rot = ref.rope_table(BASE, d, 256) if case % 4 else None
    ws, dev = _status(), kv.cuda()
    mt.kv_append_paged(dev[:, 0], dev[:, 1], cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(), _i32(off).cuda(),
                       status_ws=ws, rope=rope, **cache.args())
    assert mt.read_status(ws) == 0
    _append_on_host(cache, kv[:, 0], kv[:, 1], lambda b: list(range(off[b], off[b + 1])), past, table, rot)
    cache.check()


def test_append_again_and_again_to_one_page():
    # one row at a time, each larger than all before: the scale grows with every row
    rng = np.random.default_rng(3)
    cache = Cache(rng, "block8", 2, 2, 64, torch.bfloat16)
    table, ws = _i32([[1, 0]]).cuda(), _status()
    for i in range(20):
        kv = _rand(rng, 1, 2, 2, 64, dtype=torch.bfloat16, scale=2.0 ** (i % 7))
        d = kv.cuda()
        mt.kv_append_paged(d[:, 0], d[:, 1], cache.k, cache.v, table, _i32([i]).cuda(), _i32([0, 1]).cuda(), status_ws=ws, **cache.args())
        _append_on_host(cache, kv[:, 0], kv[:, 1], lambda b: [0], [i], np.array([[1, 0]]), None)
        cache.check()
    assert mt.read_status(ws) == 0


def test_append_extreme_values():
    rng = np.random.default_rng(4)
    cache = Cache(rng, "block8", 3, 1, 64, torch.bfloat16)
    x = torch.zeros(48, 2, 1, 64, dtype=torch.bfloat16)  # a page of zeros
    x[16:32] = _rand(rng, 16, 2, 1, 64, dtype=torch.bfloat16)
    x[17, 0, 0, 5] = float("nan")
    x[18, 1, 0, 6] = float("inf")
    x[32:48] = _rand(rng, 16, 2, 1, 64, dtype=torch.bfloat16, scale=1e-25)
    x[33, 0, 0, 0] = 3e38
    d, ws, table = x.cuda(), _status(), np.array([[2, 0, 1]])
    mt.kv_append_paged(d[:, 0], d[:, 1], cache.k, cache.v, _i32(table).cuda(), _i32([0]).cuda(), _i32([0, 48]).cuda(), status_ws=ws, **cache.args())
    _append_on_host(cache, x[:, 0], x[:, 1], lambda b: list(range(48)), [0], table, None)
    cache.check()


@pytest.mark.parametrize("kind", ["act", "block8"])
def test_append_accepted(kind):
    rng = np.random.default_rng(8)
    b, t, hkv, d, dt = 4, 20, 3, 128, torch.bfloat16
    past, lens = [14, 0, -1, 33], [3, 0, 2, 4]
    path = np.full((b, 6), -1)
    for i, n in enumerate(lens):
        path[i, :n + 1] = np.sort(rng.choice(np.arange(1, t), n + 1, replace=False))
        path[i, 0] = 0
    need = [2, 1, 1, 3]
    table = _table(rng, need, 8)
    cache = Cache(rng, kind, 8, hkv, d, dt)
    k, v = (_rand(rng, b, t, hkv, d, dtype=dt) for _ in range(2))
    ws = _status()
    rope = mt.Rope(BASE, d, 64)
    mt.kv_append_accepted(k.cuda(), v.cuda(), _i32(path).cuda(), _i32(lens).cuda(), cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(),
                          status_ws=ws, rope=rope, **cache.args())
    assert mt.read_status(ws) == 0
    _append_on_host(cache, k.view(b * t, hkv, d), v.view(b * t, hkv, d), lambda i: [i * t + int(path[i, j]) for j in range(lens[i] + 1)], past,
                    table, ref.rope_table(BASE, d, 64))
    cache.check()


@pytest.mark.parametrize("bad", ["page", "table", "offsets", "rows", "position", "node"])
def test_append_reports_and_leaves_the_rest(bad):
    rng = np.random.default_rng(11)
    hkv, d, dt = 2, 64, torch.float16
    past, new = [0, 10, 4], [20, 20, 5]
    table = _table(rng, [2, 2, 1], 6)
    off = np.array([0, 20, 40, 45])
    cache = Cache(rng, "block8", 6, hkv, d, dt)
    kv = _rand(rng, 45, 2, hkv, d, dtype=dt)
    dev, ws, want = kv.cuda(), _status(), -4
    skip = {"page": [(1, 1)], "table": [(1, 0), (1, 1)], "position": [(1, 1)]}.get(bad, [])
    rope = None
    if bad == "page":
        table = table.copy()
        table[1, 1] = 6
    elif bad == "table":
        past[1] = 13
    elif bad == "position":
        rope, want = mt.Rope(BASE, d, 29), -7
    elif bad == "offsets":
        off = np.array([0, 20, 10, 45])
    elif bad == "rows":
        off = np.array([0, 20, 40, 46])
    if bad == "node":
        path = np.array([[0, 45], [0, 1], [0, 2]])
        x = kv.view(3, 15, 2, hkv, d)
        mt.kv_append_accepted(x[:, :, 0].contiguous().cuda(), x[:, :, 1].contiguous().cuda(), _i32(path).cuda(), _i32([1, 1, 1]).cuda(), cache.k,
                              cache.v, _i32(table).cuda(), _i32(past).cuda(), status_ws=ws, **cache.args())
        assert mt.read_status(ws) == -4
        return
    mt.kv_append_paged(dev[:, 0], dev[:, 1], cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(), _i32(off).cuda(), status_ws=ws, rope=rope,
                       **cache.args())
    assert mt.read_status(ws) == want
    if not skip:
        return
    rot = ref.rope_table(BASE, d, 64) if rope else None
    before = [t.clone() for t in cache.host], [s.copy() for s in cache.host_scales]
    if bad == "page":
        table[1, 1] = table[1, 0]  # any place: its rows are put back below
    if bad == "table":
        past[1] = -1
    keep = table[1, 1]
    _append_on_host(cache, kv[:, 0], kv[:, 1], lambda b: list(range(off[b], off[b + 1] - (14 if bad == "page" and b == 1 else 0))), past, table, rot)
    if bad == "position":
        for w in range(2):
            cache.host[w].view(torch.uint8)[keep] = before[0][w].view(torch.uint8)[keep]
            cache.host_scales[w][keep] = before[1][w][keep]
    cache.check()


# ---- attention over the block-scaled cache ---------------------------------

def _attn_case(rng, b, t, hq, hkv, d, lens, dtype, tree="tree", spread=2.0):
    dt = DT[dtype]
    need = [-(-max(n, 0) // P) for n in lens]
    pages = sum(need) + 2
    table = _table(rng, need, pages)
    k, v = (rng.integers(0, 256, (pages, hkv, P, d)).astype(np.uint8) for _ in range(2))  # stale slots hold anything
    ks, vs = (2.0 ** rng.integers(-3, 2, (pages, hkv)).astype(np.float64) for _ in range(2))
    for i, n in enumerate(lens):
        for p in range(max(n, 0)):
            for c, s in ((k, ks), (v, vs)):
                pg = table[i, p // P]
                c[pg, :, p % P] = ref.encode(rng.standard_normal((hkv, d)) / s[pg][:, None])
    parents = None
    if tree == "tree":
        parents = np.full((b, t), -1)
        for i in range(b):
            for j in range(1, t):
                parents[i, j] = rng.integers(max(0, j - 9), j)
    q, kn, vn = (_rand(rng, b, t, h, d, dtype=dt, scale=s) for h, s in ((hq, spread), (hkv, 1.0), (hkv, 1.0)))
    return dict(q=q, kn=kn, vn=vn, k=k, v=v, ks=ks, vs=vs, table=table, lens=lens, parents=parents)


def _attn_run(c, out=None, ws=None, sm_scale=0.0):
    f8 = lambda x: torch.from_numpy(x).cuda().view(torch.float8_e4m3fn)  # noqa: E731
    q, kc, table = c["q"].cuda(), f8(c["k"]), _i32(c["table"]).cuda()
    out = torch.full_like(q, 5.0) if out is None else out
    ws = mt.alloc_block8_workspace(q, kc, table) if ws is None else ws
    args = (q, kc, f8(c["v"]), torch.from_numpy(c["ks"]).float().cuda(), torch.from_numpy(c["vs"]).float().cuda(), table, _i32(c["lens"]).cuda(),
            None if c["parents"] is None else _i32(c["parents"]).cuda(), out)
    kw = dict(k_new=c["kn"].cuda(), v_new=c["vn"].cuda(), workspace=ws, sm_scale=sm_scale)
    mt.tree_attn_paged_block8(*args, **kw)
    return out, ws, args, kw


def _attn_check(c, out, sm_scale=0.0):
    q = c["q"].double().numpy()
    d = q.shape[-1]
    want, mag = ref.attn64(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["parents"], c["kn"].double().numpy(),
                           c["vn"].double().numpy(), sm_scale or d ** -0.5)
    got = out.cpu().double().numpy()
    u = ref.HALF_STEP[c["q"].dtype]
    live = np.array([n >= 0 for n in c["lens"]])
    tol = u * np.abs(want) + (2.0 ** -11 + 2.0 ** -8) * mag + 1e-7
    assert np.isfinite(got[live]).all()
    bad = np.abs(got - want)[live] > tol[live]
    assert not bad.any(), (np.abs(got - want)[live] / tol[live]).max()
    assert (got[~live] == 5.0).all()


ATTN = [  # T, Hq, Hkv, D, lengths
    (1, 1, 1, 64, [0]), (1, 1, 1, 64, [1]), (1, 4, 1, 128, [16]), (1, 8, 2, 128, [17, 0, 300]),
    (1, 7, 1, 128, [63, 64, 65]), (2, 3, 3, 64, [5, 40]), (5, 12, 4, 128, [200, -1, 31]),
    (16, 2, 2, 128, [100, 3]), (17, 2, 1, 64, [90]), (64, 4, 1, 128, [250, 0]), (64, 8, 8, 64, [33]),
    (26, 8, 1, 128, [500]), (33, 3, 1, 128, [129, 64]), (64, 32, 4, 128, [100]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tree", ["tree", "chain"])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_block8_attention(dtype, tree, case):
    t, hq, hkv, d, lens = ATTN[case]
    rng = np.random.default_rng(case)
    c = _attn_case(rng, len(lens), t, hq, hkv, d, lens, dtype, tree)
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


def test_block8_attention_scale_and_empty_batch():
    c = _attn_case(np.random.default_rng(50), 3, 4, 8, 2, 128, [70, 20, 33], "bf16")
    out, ws, _, _ = _attn_run(c, sm_scale=0.02)
    _attn_check(c, out, 0.02)
    c["lens"] = [-1, -1, -1]
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0 and bool((out == 5.0).all())


def test_block8_attention_many_sequences():
    rng = np.random.default_rng(60)
    lens = [int(n) for n in rng.integers(-1, 40, 300)]
    c = _attn_case(rng, 300, 1, 2, 1, 64, lens, "f16", "chain")
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("batch, t, d, longest", [(500, 8, 128, 50), (300, 8, 64, 330), (200, 40, 128, 100), (150, 40, 64, 400)])
def test_block8_attention_many_pieces(dtype, batch, t, d, longest):
    # 32 or 160 rows a head: a CTA walks several pieces, of one tile and of more
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(-1, longest, batch)]
    c = _attn_case(rng, batch, t, 8, 2, d, lens, dtype, "tree")
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


def test_block8_attention_of_widely_spread_scales():
    # pages whose value scales differ by 2^40 and more, a page of zeros, one dominant key
    rng = np.random.default_rng(70)
    c = _attn_case(rng, 1, 3, 4, 2, 128, [160], "bf16")
    for p, k in zip(c["table"][0], (-64, -20, 0, 10, -3, 4, 20, -40, 0, 1)):
        c["vs"][p] = 2.0 ** k
    c["v"][c["table"][0][0]] = 0
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


def test_block8_attention_of_a_dominant_first_key():
    # the first key takes most of the mass and its value is small: what is left of the output is the others'
    rng = np.random.default_rng(71)
    c = _attn_case(rng, 1, 2, 4, 1, 128, [600], "bf16", spread=1.0)
    q = c["q"].double().numpy()
    first = c["table"][0][0]
    c["k"][first, 0, 0] = ref.encode(np.sign(q[0, 0].sum(0)) * 8 / c["ks"][first, 0])
    c["v"][first, 0, 0] = 0
    out, ws, _, _ = _attn_run(c)
    _attn_check(c, out)


def test_block8_attention_reports_bad_pages_and_trees():
    rng = np.random.default_rng(80)
    c = _attn_case(rng, 2, 4, 4, 2, 64, [50, 20], "f16")
    good = c["table"].copy()
    c["table"][0, 2] = 99
    assert mt.read_status(_attn_run(c)[1]) == -4
    c["table"] = good
    c["lens"] = [50, 100]
    assert mt.read_status(_attn_run(c)[1]) == -4
    c["lens"] = [50, 20]
    c["parents"][1, 2] = 3
    assert mt.read_status(_attn_run(c)[1]) == -3


def test_block8_attention_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(90)
    c = _attn_case(rng, 4, 3, 8, 2, 128, [700, 20, 64, 333], "bf16")
    want, ws, args, kw = _attn_run(c)
    _attn_check(c, want)
    out = args[-1]
    want = out.clone()
    g = _graph(lambda: mt.tree_attn_paged_block8(*args, **kw))
    out.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the lengths are read at replay: a shorter batch with the same graph
    args[6].copy_(_i32([100, 20, -1, 5]))
    out.fill_(5.0)
    g.replay()
    c["lens"] = [100, 20, -1, 5]
    _attn_check(c, out)


# ---- sampling ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", [(3, 4, 2), (4, 6, 2), (8, 8, 2), (40, 8, 2)])  # both kernels, split and whole segments
def test_block8_attention_nan_in_and_out_of_sight(dtype, t, hq, hkv):
    rng = np.random.default_rng(90 + t)
    lens = [900, 3, 70]
    c = _attn_case(rng, 3, t, hq, hkv, 128, lens, dtype, None)
    c["parents"] = np.tile(np.maximum(np.arange(t) - 1, 0), (3, 1))  # a chain that leaves node 2 out: a leaf under node 0
    c["parents"][:, 0], c["parents"][:, 2] = -1, 0
    if t > 3:
        c["parents"][:, 3] = 1
    c["vn"][:, 2, :, 5] = c["kn"][:, 1, 0, 7] = 0
    c["q"][2, 0] = c["q"][1, t - 1, 1] = 0
    clean = _attn_run(c)[0].cpu()
    c["vn"][:, 2, 0, 5] = float("nan")  # seen by node 2 alone, under KV head 0
    c["q"][2, 0, 0, 3] = float("nan")
    c["q"][1, t - 1, 1, 9] = float("inf")
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    touched = np.zeros((3, t, hq), bool)
    touched[:, 2, :hq // hkv] = touched[2, 0, 0] = touched[1, t - 1, 1] = True
    touched = torch.from_numpy(touched)
    assert out.cpu()[touched].isnan().all()
    assert torch.equal(out.cpu()[~touched], clean[~touched])
    c["kn"][0, 1, 0, 7] = float("nan")  # sequence 0, KV head 0: node 1 and what comes below it
    touched[0, 1, :hq // hkv] = touched[0, 3:, :hq // hkv] = True
    out = _attn_run(c)[0].cpu()
    assert out[touched].isnan().all()
    assert torch.equal(out[~touched], clean[~touched])


def test_block8_attention_one_workspace_for_all_sizes():
    rng = np.random.default_rng(95)
    cases = [_attn_case(rng, b, t, hq, hkv, d, lens, dtype) for b, t, hq, hkv, d, lens, dtype in
             [(2, 1, 8, 2, 128, [3000, 40], "bf16"), (2, 20, 8, 2, 128, [800, 33], "f16"), (3, 2, 6, 2, 64, [500, -1, 900], "f16"),
              (1, 64, 16, 4, 128, [300], "bf16"), (1, 9, 3, 1, 128, [1000], "bf16")]]
    own = [_attn_run(c)[:2] for c in cases]
    ws = torch.zeros(max(w.numel() for _, w in own), dtype=torch.uint8, device="cuda")
    for i in [0, 1, 2, 3, 4, 2, 0, 3, 1, 4, 0]:
        assert torch.equal(_attn_run(cases[i], ws=ws)[0], own[i][0])
    assert mt.read_status(ws) == 0


def test_block8_attention_two_graphs_and_eager_calls_share_a_workspace():
    rng = np.random.default_rng(96)
    cases = [_attn_case(rng, 2, t, 8, 2, 128, [1500, 200], "bf16") for t in (1, 12)]
    own = [_attn_run(c) for c in cases]
    ws = torch.zeros(max(w.numel() for _, w, _, _ in own), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _, _, args, kw in own:
        outs.append(torch.zeros_like(args[8]))
        call = (*args[:8], outs[-1])
        graphs.append(_graph(lambda call=call, kw=kw: mt.tree_attn_paged_block8(*call, **{**kw, "workspace": ws})))
    for i in (0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], own[i][0])
        assert torch.equal(_attn_run(cases[1 - i], ws=ws)[0], own[1 - i][0])
    assert mt.read_status(ws) == 0


FAR = 300000  # a page of 8 heads of 128 columns behind byte 2^32 and, in 16 bits, element 2^32


@pytest.mark.parametrize("t", [1, 20])
def test_block8_attention_far_pages(t):
    rng = np.random.default_rng(97)
    c = _attn_case(rng, 2, t, 16, 8, 128, [200, 77], "bf16")
    near, _, args, kw = _attn_run(c)
    n = c["k"].shape[0]
    far = []
    for x in args[1:5]:
        big = torch.empty((FAR + n, *x.shape[1:]), dtype=x.dtype, device="cuda")
        big.view(torch.uint8)[FAR:] = x.view(torch.uint8)
        far.append(big)
    table = torch.where(args[5] >= 0, args[5] + FAR, args[5])
    out = torch.empty_like(near)
    mt.tree_attn_paged_block8(args[0], *far, table, *args[6:8], out, **{**kw, "workspace": mt.alloc_block8_workspace(args[0], far[0], table)})
    assert torch.equal(out, near)


@pytest.mark.parametrize("kind", ["act", "block8"])
def test_append_far_pages(kind):
    rng = np.random.default_rng(98)
    n, table = 4, _i32([[2, 0], [3, 1]]).cuda()
    k, v = (_rand(rng, 30, 8, 128, dtype=torch.bfloat16).cuda() for _ in range(2))
    lens, off, ws = _i32([5, 0]).cuda(), _i32([0, 20, 30]).cuda(), _status()
    got = []
    for base in (0, FAR):
        caches = [torch.empty((base + n, 8, P, 128), dtype=torch.bfloat16 if kind == "act" else torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        scales = [torch.ones((base + n, 8), device="cuda") for _ in range(2)]
        for x in caches:
            x.view(torch.uint8)[base:] = 0
        kw = {} if kind == "act" else dict(k_scales=scales[0], v_scales=scales[1])
        mt.kv_append_paged(k, v, *caches, table + base, lens, off, status_ws=ws, **kw)
        got.append([x.view(torch.uint8)[base:].clone() for x in caches] + [x[base:].clone() for x in scales])
        del caches, scales
    assert mt.read_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert all(int(x.count_nonzero()) > 0 for x in got[0])


def test_norm_rope_far_tokens():
    rng = np.random.default_rng(99)
    x, pos, ws = _rand(rng, 3, 6, 64, dtype=torch.bfloat16).cuda(), _i32([4, 0, 9]).cuda(), _status()
    step = 3 * 2 ** 30 // 2  # elements from token to token: the last one is 3 * 2^30 elements away
    big = torch.empty(2 * step + 6 * 64, dtype=torch.bfloat16, device="cuda")
    view = big.as_strided((3, 6, 64), (step, 64, 1))
    view.copy_(x)
    rope = mt.Rope(BASE, 64, 16)
    near, far = x.clone(), view
    for y in (near, far):
        mt.qk_norm_rope(y[:, :4], y[:, 4:], pos, y[:, :4], y[:, 4:], rope=rope, q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                        k_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"), status_ws=ws)
    assert mt.read_status(ws) == 0
    assert torch.equal(far, near) and not torch.equal(near, x)


def test_sampling_far_rows_and_the_same_row_twice():
    rng = np.random.default_rng(100)
    n, v = 20000, 120000
    big = torch.empty(n, v, dtype=torch.float16, device="cuda")
    few = _rand(rng, 2, v, dtype=torch.float16, scale=2.0).cuda()
    big[n - 1], big[3] = few[0], few[1]
    u = torch.tensor([0.1, 0.9, 0.5, 0.5], device="cuda")
    near, far = (torch.full((4,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    mt.sample_tokens(few, u, near, row_index=_i32([0, 0, 1, -1]).cuda())
    mt.sample_tokens(big, u, far, row_index=_i32([n - 1, n - 1, 3, -1]).cuda())
    assert torch.equal(near, far) and int(near[3]) == -7 and int(near[0]) != int(near[1])


def _sample(x, u, t=None, k=None, p=None, m=None, index=None, tokens=None):
    n = len(u)
    f = lambda a: None if a is None else torch.as_tensor(np.asarray(a, np.float32)).cuda()  # noqa: E731
    tokens = torch.full((n,), -7, dtype=torch.int32, device="cuda") if tokens is None else tokens
    mt.sample_tokens(x, f(u), tokens, temperature=f(t), top_k=None if k is None else _i32(k).cuda(), top_p=f(p), min_p=f(m),
                     row_index=None if index is None else _i32(index).cuda())
    return tokens.cpu().numpy()


def _sample_check(x, u, t, k, p, m):
    got = _sample(x, u, t, k, p, m)
    h = x.cpu().double().numpy()
    f = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
    want = [ref.sample64(h[i], f(u)[i], f(t)[i], int(k[i]), f(p)[i], f(m)[i]) for i in range(len(u))]
    assert got.tolist() == want


def _params(rng, n):
    return (rng.choice([0.0, 0.5, 0.8, 1.0, 1.5], n), rng.choice([0, 1, 2, 17, 50, 1000], n), rng.choice([1.0, 0.9, 0.5, 0.99], n),
            rng.choice([0.0, 0.0, 0.02, 0.2], n))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n, v", [(1, 1), (4, 2), (33, 7), (16, 1000), (40, 4099), (24, 32000), (3, 32001), (12, 70003), (2, 200000), (1, 499999)])
def test_sampling(dtype, n, v):
    rng = np.random.default_rng(v)
    x = _rand(rng, n, v, scale=2.5)
    x.view(-1)[torch.from_numpy(rng.integers(0, n * v, 4 * n))] += 5
    t, k, p, m = _params(rng, n)
    _sample_check(x.to(DT[dtype]).cuda(), rng.random(n), t, k, p, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "two", "whole", "negative", "tiny", "huge", "masked"])
def test_sampling_ties_and_odd_ranges(dtype, kind):
    rng = np.random.default_rng(len(kind))
    n, v = 32, 5003
    x = {"equal": lambda: np.full((n, v), 0.25), "two": lambda: rng.integers(0, 2, (n, v)) * 1.0, "whole": lambda: np.round(rng.standard_normal((n, v)) * 2),
         "negative": lambda: -100 - rng.random((n, v)) * 10, "tiny": lambda: rng.standard_normal((n, v)) * 1e-6,
         "huge": lambda: rng.standard_normal((n, v)) * 1e4, "masked": lambda: np.where(rng.random((n, v)) < 0.9, -np.inf, rng.standard_normal((n, v)))}[kind]()
    t, k, p, m = _params(rng, n)
    _sample_check(torch.from_numpy(x).to(DT[dtype]).cuda(), rng.random(n), t, k, p, m)


def test_sampling_limits_of_the_parameters():
    rng = np.random.default_rng(7)
    v = 3001
    x = _rand(rng, 1, v, scale=2.0).repeat(20, 1).cuda()
    u = np.array([0.0, 1 - 2.0 ** -24] * 10, np.float32)
    t = np.repeat([1e-30, 1e-3, 1.0, 100.0, 1e30, 1.0, 1.0, 1.0, 1.0, 1.0], 2)
    k = np.repeat([0, 0, v, v + 5, -3, v - 1, 1, 0, 0, 0], 2)
    p = np.repeat([1.0, 1.0, 2.0, 1.0, 1.0, 1.0, 0.9, 0.0, 1e-9, 0.999999], 2)
    m = np.repeat([0.0, 0.0, -1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 1.0, 1.5], 2)
    _sample_check(x, u, t, k, p, m)
    top = int(x[0].argmax())
    assert _sample(x[:3], [2.0, -1.0, float("nan")], [1e-3] * 3).tolist() == [top] * 3  # numbers outside [0, 1)


def test_sampling_infinities_and_nan():
    rng = np.random.default_rng(9)
    v = 777
    x = _rand(rng, 6, v)
    x[0, :] = float("-inf")
    x[1, :] = float("nan")
    x[2, ::2] = float("nan")
    x[3, [5, 600]] = float("inf")
    x[4, :] = float("-inf")
    x[4, 31] = -3.0
    u = [0.3, 0.3, 0.4, 0.6, 0.9, 0.2]
    for k, p, m in ((0, 1.0, 0.0), (3, 0.9, 0.1), (700, 0.99, 0.0)):
        one = [1.0] * 6
        _sample_check(x.cuda(), u, one, [k] * 6, [p] * 6, [m] * 6)
    assert _sample(x.cuda(), u)[:2].tolist() == [-1, -1]
    assert _sample(x.cuda(), u)[3] == 600 and _sample(x.cuda(), u)[4] == 31


def test_sampling_rows_by_index_strides_and_places_without_a_row():
    rng = np.random.default_rng(12)
    big = _rand(rng, 10, 3, 1003, dtype=torch.bfloat16).cuda()
    x = big[:, 1]  # every third row, unaligned
    u = rng.random(6)
    index = [3, 0, -1, 9, 10, 3]
    got = _sample(x, u, index=index)
    h = x.cpu().double().numpy()
    want = [ref.sample64(h[r], np.float64(np.float32(v)), 1.0, 0, 1.0, 0.0) if 0 <= r < 10 else (-7 if r < 0 else -1) for r, v in zip(index, u)]
    assert got.tolist() == want


def test_sampling_whole_distribution():
    # 4096 evenly spread numbers draw each token as often as its probability says, within one
    v, n = 50, 4096
    x = _rand(np.random.default_rng(13), 1, v, scale=1.5)
    got = _sample(x.repeat(n, 1).cuda(), (np.arange(n) + 0.5) / n)
    w = np.exp(x[0].double().numpy() - float(x.max()))
    count = np.bincount(got, minlength=v)
    assert (np.abs(count - w / w.sum() * n) <= 1.0 + 1e-6).all()


def test_sampling_in_a_graph():
    rng = np.random.default_rng(14)
    x, u = _rand(rng, 5, 9000, scale=2.0).cuda(), torch.rand(5, device="cuda")
    tokens = torch.zeros(5, dtype=torch.int32, device="cuda")
    par = dict(temperature=torch.full((5,), 0.9, device="cuda"), top_p=torch.full((5,), 0.9, device="cuda"))
    g = _graph(lambda: mt.sample_tokens(x, u, tokens, **par))
    for _ in range(3):
        x.copy_(_rand(rng, 5, 9000, scale=2.0))
        u.copy_(torch.rand(5))
        tokens.zero_()
        g.replay()
        got = tokens.cpu().tolist()
        assert got == mt.sample_tokens(x, u, torch.zeros_like(tokens), **par).cpu().tolist()


# ---- together ----------------------------------------------------------------

def test_prompt_step_and_draw_together():
    """Two layers of one serving pass: prompts into a block-scaled cache, a tree step over it, acceptance, the
    accepted path appended, a token drawn from the end node's row; each result against the plain implementations."""
    rng = np.random.default_rng(100)
    b, t, hq, hkv, d, v, dt = 3, 8, 8, 2, 128, 500, torch.bfloat16
    prompts = [37, 5, 80]
    off = np.concatenate([[0], np.cumsum(prompts)])
    n = int(off[-1])
    table = _table(rng, [4, 2, 6], 14)
    rope, rot, ws = mt.Rope(BASE, d, 128), ref.rope_table(BASE, d, 128), _status()
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    w = (1 + 0.1 * _rand(rng, d)).to(dt)
    parents = np.array([[-1, 0, 0, 1, 1, 2, 3, 3]] * b)
    depths = np.array([0, 1, 1, 2, 2, 2, 3, 3])
    tokens = rng.integers(0, v, (b, t))
    logits = _rand(rng, b, t, v, scale=2.0)
    for i, path in enumerate(([0, 1, 3], [0], [0, 2, 5])):  # the accepted paths
        for a, c in zip(path, path[1:]):
            logits[i, a, tokens[i, c]] = 30.0
        logits[i, path[-1], :] += 0  # the end's argmax is none of its children's tokens but by chance
        for c in range(t):
            if parents[i, c] == path[-1]:
                logits[i, path[-1], tokens[i, c]] = -30.0
    dtab = _i32(table).cuda()
    states = []
    for layer in range(2):
        cache = Cache(rng, "block8", 14, hkv, d, dt)
        qkv = _rand(rng, n, hq + 2 * hkv, d, dtype=dt).cuda()
        pos = torch.cat([torch.arange(p) for p in prompts]).int().cuda()
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
        mt.qk_norm_rope(q, k, pos, q, k, rope=rope, q_weight=w.cuda(), k_weight=w.cuda(), status_ws=ws)
        mt.kv_append_paged(k, qkv[:, hq + hkv:], cache.k, cache.v, dtab, lens, _i32(off).cuda(), status_ws=ws, **cache.args())
        _append_on_host(cache, k.cpu(), qkv[:, hq + hkv:].cpu(), lambda i: list(range(off[i], off[i + 1])), [0] * b, table, None)
        cache.check()
        states.append(cache)
    lens += _i32(prompts).cuda()
    rows = [_rand(rng, b, t, hq + 2 * hkv, d, dtype=dt) for _ in range(2)]
    kept = []
    for cache, x in zip(states, rows):
        y = x.cuda().view(b * t, -1, d)
        pos = (lens[:, None] + _i32(depths).cuda()).view(-1).int()
        q, k = torch.empty(b * t, hq, d, dtype=dt, device="cuda"), torch.empty(b * t, hkv, d, dtype=dt, device="cuda")
        mt.qk_norm_rope(y[:, :hq], y[:, hq:hq + hkv], pos, q, k, rope=rope, q_weight=w.cuda(), k_weight=w.cuda(), status_ws=ws)
        q, k, vn = q.view(b, t, hq, d), k.view(b, t, hkv, d), y[:, hq + hkv:].contiguous().view(b, t, hkv, d)
        out = torch.empty_like(q)
        aws = mt.alloc_block8_workspace(q, cache.k, dtab)
        mt.tree_attn_paged_block8(q, cache.k, cache.v, *cache.scales, dtab, lens, _i32(parents).cuda(), out, k_new=k, v_new=vn, workspace=aws)
        assert mt.read_status(aws) == 0
        _attn_check(dict(q=q.cpu(), kn=k.cpu(), vn=vn.cpu(), k=_codes(cache.k), v=_codes(cache.v), ks=cache.host_scales[0], vs=cache.host_scales[1],
                         table=table, lens=prompts, parents=parents), out)
        kept.append((k, vn))
    alen, path = torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros(b, 4, dtype=torch.int32, device="cuda")
    mt.tree_accept_greedy(_i32(tokens).cuda(), logits.cuda(), _i32(parents).cuda(), alen, path, argmax_out=torch.zeros(b, t, dtype=torch.int32, device="cuda"),
                          next_token=torch.zeros(b, dtype=torch.int32, device="cuda"), workspace=mt.alloc_accept_workspace(b, t))
    assert alen.tolist() == [2, 0, 2]
    for cache, (k, vn) in zip(states, kept):
        mt.kv_append_accepted(k, vn, path, alen, cache.k, cache.v, dtab, lens, status_ws=ws, **cache.args())
        _append_on_host(cache, k.cpu().view(b * t, hkv, d), vn.cpu().view(b * t, hkv, d),
                        lambda i: [i * t + int(path[i, j]) for j in range(int(alen[i]) + 1)], prompts, table, None)
        cache.check()
    lens += alen + 1
    end = path.gather(1, alen[:, None].long())[:, 0] + torch.arange(b, device="cuda", dtype=torch.int32) * t
    u = rng.random(b)
    got = _sample(logits.cuda().view(b * t, v), u, [0.8] * b, [40] * b, [0.95] * b, [0.0] * b, index=end.cpu().numpy())
    f = lambda a: np.float64(np.float32(a))  # noqa: E731
    assert got.tolist() == [ref.sample64(logits.view(b * t, v)[int(end[i])].double().numpy(), f(u[i]), f(0.8), 40, f(0.95), 0.0) for i in range(b)]
    assert mt.read_status(ws) == 0


def test_block8_attention_wait_bound():
    """A pipeline wait that only its bound ends: the status says so, and the next call is right."""
    rng = np.random.default_rng(95)
    c = _attn_case(rng, 2, 32, 8, 2, 128, [100, 40], "bf16")
    out, ws, args, kw = _attn_run(c)
    _attn_check(c, out)
    try:
        mt.debug_set_wait(20_000_000, stall=True)
        mt.tree_attn_paged_block8(*args, **kw)
        assert mt.read_status(ws) == -6
    finally:
        mt.debug_set_wait()
    out.fill_(5.0)
    mt.tree_attn_paged_block8(*args, **kw)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv, lens", [(1, 1, 1, [0, 1, 40]), (1, 8, 2, [5, 900, 0]), (4, 8, 2, [900, 3, 70]), (4, 18, 2, [33, 0, 200]), (9, 8, 2, [900, 3, 70])])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_block8_attention_infinite_query_among_keys_of_one_sign(dtype, t, hq, hkv, lens, sign):
    # every product with the infinity has the same sign: all scores +inf, or all -inf
    c = _attn_case(np.random.default_rng(110), 3, t, hq, hkv, 128, lens, dtype, "chain")
    c["k"][:, :, :, 9] = ref.encode(1.0)
    c["kn"][..., 9] = 1.0
    c["q"][..., 9] = 0.5
    clean = _attn_run(c)[0].cpu()
    c["q"][1, 0, 0, 9] = c["q"][:, t - 1, hq - 1, 9] = sign * float("inf")
    touched = torch.zeros(3, t, hq, dtype=torch.bool)
    touched[1, 0, 0] = touched[:, t - 1, hq - 1] = True
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    out = out.cpu()
    assert out[touched].isnan().all()
    assert torch.equal(out[~touched], clean[~touched])


def _leaf_2(parents):
    """Every node the child of the one before it, but node 2, a leaf under node 0, and node 3, under node 1."""
    t = parents.shape[1]
    parents[:] = np.arange(t) - 1
    parents[:, 2:3], parents[:, 3:4] = 0, 1


def _attn_check_nodes(c, out, nodes=slice(None)):
    """As _attn_check, of some of the nodes, with two more terms.  A weight below 2^-14 is a subnormal fp16, off by up
    to 2^-25 where the row's largest weight times value scale stands for 2^3: together sum |code| 2^-28 max(p scale),
    which counts where the scales in sight differ by much.  And what is past the output type's largest value is
    infinite (or, within the tolerance, is not yet)."""
    q, kn, vn = (c[n].double().numpy() for n in ("q", "kn", "vn"))
    b, t, hq, d = q.shape
    hkv = kn.shape[2]
    got, top = out.cpu().double().numpy(), torch.finfo(c["q"].dtype).max
    for i in range(b):
        n = c["lens"][i]
        tree = ref.ancestors(None if c["parents"] is None else c["parents"][i], t)
        sees = np.concatenate([np.ones((t, n), bool), tree], 1)
        at = [(c["table"][i][s // P], s % P) for s in range(n)]
        for h in range(hkv):
            both = []
            for cache, scales, new in ((c["k"], c["ks"], kn), (c["v"], c["vs"], vn)):
                code, scale = [ref.decode(cache[pg, h, s]) for pg, s in at], [float(scales[pg, h]) for pg, s in at]
                for j in range(0, t, P):
                    block, s = ref.block_codes(new[i, j:j + P, h])
                    code.extend(ref.decode(block))
                    scale.extend([s] * len(block))
                both.append((np.array(code), np.array(scale)[:, None]))
            (k, ks), (v, vs) = both
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                z = np.where(sees, q[i, :, j] @ (k * ks).T * d ** -0.5, -np.inf)
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                want, mag = w @ (v * vs), w @ np.abs(v * vs)
                tol = ref.HALF_STEP[c["q"].dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -8) * mag + 1e-7
                tol += 2.0 ** -28 * (w * vs.T).max(1, keepdims=True) * (sees @ np.abs(v))
                with np.errstate(invalid="ignore"):
                    fine = np.abs(got[i, :, j] - want) <= tol
                    fine |= (np.abs(want) + tol >= top) & (got[i, :, j] == np.sign(want) * np.inf)
                assert fine[nodes].all(), (i, j, np.argwhere(~fine)[:3])


ROWS = [(1, 1, 1), (1, 8, 1), (4, 8, 2), (4, 18, 2), (6, 16, 4), (40, 8, 2), (64, 4, 1)]  # T, Hq, Hkv: 1 to 256 rows a KV head, both kernels


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", ROWS)
@pytest.mark.parametrize("at, power", [(0, 24), (0, 40), (3, 28), (18, 60)])
def test_block8_attention_large_values_of_no_weight(dtype, t, hq, hkv, at, power):
    # a page whose value scale is 2^power times the others' and whose scores are 120 lower, in powers of two: what
    # is left of it is below 2^-50, and the other pages' weights keep their bits
    c = _attn_case(np.random.default_rng(120 + at), 1, t, hq, hkv, 128, [333], dtype, spread=1.0)
    c["q"][..., 9], c["kn"][..., 9], c["k"][:, :, :, 9] = 120.0, 0, 0
    page = c["table"][0][at]
    c["ks"][page] = 1.0
    c["k"][page, :, :, 9] = ref.encode(-9.0)
    c["vs"][page] = 2.0 ** power
    c["v"][page] = ref.encode(np.random.default_rng(1).standard_normal((hkv, P, 128)))
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", [r for r in ROWS if r[0] > 1])
def test_block8_attention_large_values_out_of_sight(dtype, t, hq, hkv):
    # they raise the scale of their block of new tokens, and so cost its other rows precision; nothing else
    c = _attn_case(np.random.default_rng(130), 2, t, hq, hkv, 128, [100, 0], dtype)
    _leaf_2(c["parents"])
    c["vn"][:, 2, 0, 5], c["kn"][0, 2, hkv - 1, 7] = 30000.0, -30000.0
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check_nodes(c, out, np.arange(t) != 2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", ROWS)
def test_block8_attention_of_spread_scales_in_every_kernel(dtype, t, hq, hkv):
    # as the tests of widely spread scales and of a dominant key, for every number of rows
    c = _attn_case(np.random.default_rng(140), 1, t, hq, hkv, 128, [160], dtype, spread=1.0)
    for p, k in zip(c["table"][0], (-64, -20, 0, 10, -3, 4, 20, -40, 0, 1)):
        c["vs"][p] = 2.0 ** k
    c["v"][c["table"][0][0]] = 0
    _attn_check_nodes(c, _attn_run(c)[0])
    c = _attn_case(np.random.default_rng(141), 1, t, hq, hkv, 128, [600], dtype, spread=1.0)
    first = c["table"][0][0]
    c["q"][..., 9], c["kn"][..., 9], c["k"][:, :, :, 9] = 8.0, 0, 0
    c["k"][first, 0, 0, 9], c["v"][first, 0, 0] = ref.encode(16 / c["ks"][first, 0]), 0
    _attn_check_nodes(c, _attn_run(c)[0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", [r for r in ROWS if r[0] > 1])
@pytest.mark.parametrize("where", ["value", "key", "both"])
def test_block8_attention_infinity_in_and_out_of_sight(dtype, t, hq, hkv, where):
    # as a NaN: the nodes that see it are NaN, the others as if it were 0
    c = _attn_case(np.random.default_rng(150), 2, t, hq, hkv, 128, [100, 0], dtype)
    _leaf_2(c["parents"])
    places = ([(c["vn"], 2, 0, 5)] if where != "key" else []) + ([(c["kn"], 2, hkv - 1, 7), (c["kn"], 1, hkv - 1, 100)] if where != "value" else [])
    for x, node, h, col in places:
        x[:, node, h, col] = 0
    clean = _attn_run(c)[0].cpu()
    _attn_check_nodes(c, clean)
    touched = torch.zeros(2, t, hq, dtype=torch.bool)
    for i, (x, node, h, col) in enumerate(places):
        x[:, node, h, col] = (-1) ** i * float("inf")
        sees = torch.from_numpy(ref.ancestors(c["parents"][0], t)[:, node])
        touched[:, sees, h * (hq // hkv):(h + 1) * (hq // hkv)] = True
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    assert out.cpu()[touched].isnan().all()
    assert torch.equal(out.cpu()[~touched], clean[~touched])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v, gap, t", [(400000, 23.0, 1.0), (200000, 22.0, 1.0), (300000, 11.5, 0.5), (70000, 20.0, 1.0), (400000, 15.0, 1.0)])
def test_sampling_top_p_of_a_long_flat_tail(dtype, v, gap, t):
    # one token of weight 1 and v - 1 of e^(-gap / t), far below it but together worth a cut.  A weight is good to 1e-9
    # of itself and 2^-44: all together to E, which is E / w tail tokens; the cut and the draw each compare such a sum
    # with a multiple of another
    p = np.float32([0.99999, 0.999995, 0.999999, 0.9, 0.99999, 0.99999])
    u = np.float32([0.99999, 0.999998, 1 - 2.0 ** -24, 0.99999, 0.5, 0.999999])
    x = torch.full((1, v), -gap)
    x[0, 0] = 0
    got = _sample(x.to(DT[dtype]).cuda().expand(len(u), v), u, [t] * len(u), p=p)
    w = np.exp(-gap / t)
    slack = 2 + 4 * (v * (2.0 ** -44 + 1e-9 * w) + 1e-9) / w
    for a, b, token in zip(p.astype(np.float64), u.astype(np.float64), got):
        kept = min(max(np.ceil((a * (1 + (v - 1) * w) - 1) / w), 0), v - 1)
        want = (b * (1 + kept * w) - 1) / w + 1
        assert abs(token - max(want, 0)) <= slack, (a, b, token, want, slack)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m, low, t", [(7 * 2.0 ** -24, -8.0, 1.0), (-7 * 2.0 ** -24, -8.0, 1.0), (7 * 2.0 ** -24, -4.0, 0.5), (-2.0 ** -23, -2.0, 0.25),
                                       (0.0, -8.0, 1.0), (2.0 ** -11, -8.0, 1.0), (-2.0 ** -10, -16.0, 2.0), (0.0625, -8.0, 1.0)])
def test_sampling_next_to_a_border_of_a_nearly_certain_token(dtype, m, low, t):
    # e^8 tokens of weight about e^-8, then the maximum, next to 0: differences that 24 bits do not hold.  The draw is
    # the maximum from the border on, which lies where all weights are good to 1e-9 and 2^-44
    n = 2981
    x = torch.full((1, n + 1), low)
    x[0, n] = m
    x = x.to(DT[dtype])
    h = x.double().numpy()[0]
    w = np.exp((h[0] - h[n]) / t)
    border, slack = n * w / (1 + n * w), 1e-9 + n * 2.0 ** -44
    u = np.float32(border) + np.arange(-40, 41, dtype=np.float32) * np.float32(2.0 ** -24)
    got = _sample(x.cuda().expand(len(u), n + 1), u, [t] * len(u))
    want = np.where(u.astype(np.float64) >= border, n, n - 1)
    sure = np.abs(u.astype(np.float64) - border) > slack
    assert sure.sum() >= 79 and np.array_equal(got[sure], want[sure])


@pytest.mark.parametrize("kind", ["act", "e4m3", "block8"])
def test_append_accepted_writes_nothing_of_a_path_with_a_stray_node(kind):
    # the path spans two pages or more, and the node outside the tree falls in one of them
    rng = np.random.default_rng(160)
    b, t, hkv, d, dt = 5, 40, 2, 64, torch.float16
    past, lens = [14, 3, 14, 0, 30], [3, 35, 3, 39, 2]
    path = np.full((b, 40), -1)
    for i, n in enumerate(lens):
        path[i, :n + 1] = rng.permutation(t)[:n + 1]
    path[0, 3], path[1, 1], path[3, 39] = t, -1, 1 << 30
    table = _table(rng, [2, 3, 2, 3, 3], 14)
    cache = Cache(rng, kind, 14, hkv, d, dt)
    k, v = (_rand(rng, b, t, hkv, d, dtype=dt) for _ in range(2))
    ws = _status()
    mt.kv_append_accepted(k.cuda(), v.cuda(), _i32(path).cuda(), _i32(lens).cuda(), cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(),
                          status_ws=ws, **cache.args())
    assert mt.read_status(ws) == -4
    good = [p if i in (2, 4) else -1 for i, p in enumerate(past)]
    _append_on_host(cache, k.view(b * t, hkv, d), v.view(b * t, hkv, d), lambda i: [i * t + int(path[i, j]) for j in range(lens[i] + 1)], good, table, None)
    cache.check()


@pytest.mark.parametrize("bad", ["offsets", "rows", "node", "length"])
def test_append_of_a_bad_sequence_leaves_its_pages(bad):
    # what test_append_reports_and_leaves_the_rest reads the status of: the first sequence is written, the bad one is not
    rng = np.random.default_rng(170)
    hkv, d, dt = 2, 64, torch.float16
    past, table = [0, 10, 4], _table(rng, [2, 2, 1], 7)
    cache, ws = Cache(rng, "block8", 7, hkv, d, dt), _status()
    kv = _rand(rng, 45, 2, hkv, d, dtype=dt)
    dev, live = kv.cuda(), [0, -1, -1]
    if bad in ("offsets", "rows"):
        # offsets that fall, and after them 35 rows, more than the last sequence's table covers; or a row too many
        off = [0, 20, 10, 45] if bad == "offsets" else [0, 20, 40, 46]
        mt.kv_append_paged(dev[:, 0], dev[:, 1], cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(), _i32(off).cuda(), status_ws=ws, **cache.args())
        live = [0, -1, -1] if bad == "offsets" else [0, 10, -1]
        rows = lambda b: list(range(off[b], off[b + 1]))  # noqa: E731
    else:
        path, lens = np.array([[0, 1], [0, 3], [0, 2]]), [1, 1, 1]
        if bad == "node":
            path[1, 1] = 15
        else:
            lens[1] = 2
        x, live = kv.view(3, 15, 2, hkv, d), [0, -1, 4]
        mt.kv_append_accepted(x[:, :, 0].contiguous().cuda(), x[:, :, 1].contiguous().cuda(), _i32(path).cuda(), _i32(lens).cuda(), cache.k, cache.v,
                              _i32(table).cuda(), _i32(past).cuda(), status_ws=ws, **cache.args())
        rows = lambda b: [15 * b + int(n) for n in path[b]]  # noqa: E731
    assert mt.read_status(ws) == -4
    _append_on_host(cache, kv[:, 0], kv[:, 1], rows, live, table, None)
    cache.check()


@pytest.mark.parametrize("batch", [32, 33, 1024, 1025, 2000])
@pytest.mark.parametrize("kind", ["act", "block8"])
def test_append_of_large_batches(batch, kind):
    # an item's sequence is found in one, two or three rounds of 32; some sequences are empty, some absent
    rng = np.random.default_rng(batch)
    past = rng.integers(-3, 40, batch)
    new = rng.integers(-6, 12, batch).clip(0)
    new[rng.integers(0, batch, 3)] = 50
    if batch > 1000:
        new[200:260] = 0
    past = np.where(past < 0, -1, past)
    off = np.concatenate([[0], np.cumsum(new)]) + 5  # rows before the first sequence's, too
    need = [-(-(max(int(p), 0) + int(n)) // P) for p, n in zip(past, new)]
    table = _table(rng, need, sum(need) + 1)
    cache = Cache(rng, kind, sum(need) + 1, 1, 64, torch.bfloat16)
    kv = _rand(rng, int(off[-1]) + 3, 2, 1, 64, dtype=torch.bfloat16)
    dev, ws = kv.cuda(), _status()
    mt.kv_append_paged(dev[:, 0], dev[:, 1], cache.k, cache.v, _i32(table).cuda(), _i32(past).cuda(), _i32(off).cuda(), status_ws=ws, **cache.args())
    assert mt.read_status(ws) == 0
    _append_on_host(cache, kv[:, 0], kv[:, 1], lambda b: list(range(off[b], off[b + 1])), past, table, None)
    cache.check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("batch, t, hq, hkv, longest", [(330, 20, 32, 32, 16), (300, 17, 64, 64, 60)])
def test_block8_attention_more_pieces_than_a_list_holds(dtype, batch, t, hq, hkv, longest):
    # tens of whole segments for every CTA of the tensor-core kernel: each role walks the schedule by itself
    rng = np.random.default_rng(180)
    lens = [int(n) for n in rng.integers(-1, longest + 1, batch)]
    c = _attn_case(rng, batch, t, hq, hkv, 64, [0] * batch, dtype)
    need = [-(-max(n, 0) // P) for n in lens]
    c["lens"], pages = lens, 40  # sequences share the pages, which nothing writes
    c["k"], c["v"] = (ref.encode(rng.standard_normal((pages, hkv, P, 64))) for _ in range(2))
    c["ks"], c["vs"] = (2.0 ** rng.integers(-2, 2, (pages, hkv)).astype(np.float64) for _ in range(2))
    c["table"] = np.where(np.arange(max(need))[None] < np.array(need)[:, None], rng.integers(0, pages, (batch, max(need))), -1)
    top = max(float(c["vn"].abs().max()), float((np.abs(ref.decode(c["v"])) * c["vs"][:, :, None, None]).max()))
    out, ws, args, kw = _attn_run(c)
    assert mt.read_status(ws) == 0
    got = out.clone()
    # some sequences against the definition, and all of them against calls of a few at a time (each within its tolerance)
    few = rng.choice(batch, 4, replace=False)
    part = {n: c[n][few] for n in ("q", "kn", "vn", "table", "parents")}
    _attn_check({**c, **part, "lens": [lens[i] for i in few]}, got[torch.from_numpy(few).cuda()])
    for b0 in range(0, batch, 30):
        sub = [args[0][b0:b0 + 30], *args[1:5], *(x[b0:b0 + 30].contiguous() for x in args[5:8]), torch.full_like(args[0][b0:b0 + 30], 5.0)]
        new = {n: kw[n][b0:b0 + 30] for n in ("k_new", "v_new")}
        mt.tree_attn_paged_block8(*sub, **new, workspace=mt.alloc_block8_workspace(sub[0], sub[1], sub[5]))
        a, b = sub[8].double(), got[b0:b0 + 30].double()
        assert bool(((a - b).abs() <= 2 * (ref.HALF_STEP[out.dtype] * b.abs() + (2.0 ** -11 + 2.0 ** -8) * top)).all())


@pytest.mark.parametrize("t, hq, hkv", ROWS)
def test_block8_attention_under_a_wide_block_table(t, hq, hkv):
    # a serving loop's tables have the model's whole length, whatever the sequences have
    c = _attn_case(np.random.default_rng(190), 2, t, hq, hkv, 128, [700, 37], "bf16")
    near = _attn_run(c)[0]
    wide = np.full((2, 131072 // P), -1)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    out, ws, _, _ = _attn_run(c)
    assert mt.read_status(ws) == 0
    _attn_check(c, out)
    _attn_check(c, near)


@pytest.mark.parametrize("t, hq, hkv", ROWS)
def test_block8_attention_keeps_eleven_bits_of_a_weight(t, hq, hkv):
    # as _attn_check, with queries so small that scores are good to 2^-13 (2 D 2^-24 sum |q k| scale < 2^-14 with a sum
    # <= 3; elements to 2^-17.8 of a largest of 1.1, times sum |k| scale <= 9: < 2^-14): what is left is the rounding of
    # the weights and of the output
    c = _attn_case(np.random.default_rng(200), 2, t, hq, hkv, 128, [300, 20], "f16", spread=0.25)
    q = c["q"].double().numpy()
    want, mag = ref.attn64(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["parents"], c["kn"].double().numpy(), c["vn"].double().numpy(), 128 ** -0.5)
    out, ws, args, kw = _attn_run(c)
    tol = ref.HALF_STEP[torch.float16] * np.abs(want) + (2.0 ** -11 + 2 * 2.0 ** -13) * mag + 1e-7
    assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()
    again = out.clone()
    for _ in range(3):  # and the same bits every time
        out.zero_()
        mt.tree_attn_paged_block8(*args, **kw)
        assert torch.equal(out, again)


@pytest.mark.parametrize("t, hq, hkv", ROWS)
def test_block8_attention_of_value_scales_below_the_range(t, hq, hkv):
    # the documented floor, in either kernel
    c = _attn_case(np.random.default_rng(210), 1, t, hq, hkv, 128, [90], "bf16")
    low, floor = {**c, "vs": c["vs"].copy()}, {**c, "vs": c["vs"].copy()}
    for page, value in zip(c["table"][0], (2.0 ** -90, 1e-30, 2.0 ** -126)):
        low["vs"][page], floor["vs"][page] = value, 2.0 ** -64
    assert torch.equal(_attn_run(low)[0], _attn_run(floor)[0])
