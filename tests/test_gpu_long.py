"""The operators for long sequences on the GPU against plain implementations in 64 bits (long_reference).

Tolerances (u = half a step of the output's type relative to the value: bf16 2^-8, fp16 2^-11, fp32 2^-24):
  window attention    as the attention without one (test_gpu_serve): u |out| + 2^-11 A + 2 E A, A = sum p |v|, E = 2^-9 the
                      error of a score in the exponent (D products and sums in 32 bits, 2 D 2^-24 sum |q k| scale, and
                      what falls below a query's parts);
  log-sum-exp         E for the scores, and 2^-20 (1 + |lse|) for the sum's 32 bits, its logarithm and the units."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import long_reference as lref
import medusa_tree_speculative_attn_gb300 as mt
import serve_reference as ref
from test_gpu_serve import DT, P, Cache, _attn_case, _codes, _graph, _i32, _rand, _status, _table

pytestmark = pytest.mark.gpu


# ---- attention under a window ------------------------------------------------

def _f8(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().view(torch.float8_e4m3fn)


def _hide(c, window, sinks):
    """Table entries that no new token needs become nonsense."""
    t = c["q"].shape[1]
    for i, n in enumerate(c["lens"]):
        if n > 0:
            some = lref.sees(n, t, None if c["parents"] is None else c["parents"][i], window, sinks).any(0)
            for p in range(c["table"].shape[1]):
                if not some[p * P:min(n, (p + 1) * P)].any():
                    c["table"][i, p] = 2 ** 30 if (i + p) % 2 else -1


def _window_run(c, window, sinks, sm_scale=0.0, lse=True, ws=None):
    q, kc, table = c["q"].cuda(), _f8(c["k"]), _i32(c["table"]).cuda()
    out = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:3], 5.0, device="cuda") if lse else None
    ws = mt.alloc_block8_workspace(q, kc, table) if ws is None else ws
    args = (q, kc, _f8(c["v"]), torch.from_numpy(c["ks"]).float().cuda(), torch.from_numpy(c["vs"]).float().cuda(), table, _i32(c["lens"]).cuda(),
            None if c["parents"] is None else _i32(c["parents"]).cuda(), out)
    kw = dict(k_new=c["kn"].cuda(), v_new=c["vn"].cuda(), workspace=ws, sm_scale=sm_scale, window=window, sinks=sinks, lse=lse)
    mt.tree_attn_paged_block8(*args, **kw)
    return out, lse, ws, args, kw


def _window_check(c, out, lse, window, sinks, sm_scale=0.0):
    d = c["q"].shape[-1]
    want, mag, wlse = lref.window_attn64(c, window, sinks, sm_scale or d ** -0.5)
    live = np.array([n >= 0 for n in c["lens"]])
    got = out.cpu().double().numpy()
    tol = ref.HALF_STEP[c["q"].dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -8) * mag + 1e-7
    assert np.array_equal(np.isnan(got[live]), np.isnan(want[live]))
    bad = np.abs(got - want)[live] > tol[live]
    assert not bad.any(), np.argwhere(bad)[:4]
    assert (got[~live] == 5.0).all()
    if lse is not None:
        got = lse.cpu().double().numpy()
        bad = np.abs(got - wlse)[live] > (2.0 ** -9 + 2.0 ** -20 * (1 + np.abs(wlse)))[live]
        assert np.isfinite(got[live]).all() and not bad.any(), np.argwhere(bad)[:4]
        assert (got[~live] == 5.0).all()


WINDOWS = [  # T, Hq, Hkv, D, lengths
    (1, 1, 1, 64, [0, 1, 40]), (1, 8, 2, 128, [17, -1, 300]), (2, 3, 3, 64, [5, 140]), (5, 12, 4, 128, [200, -1, 31]), (16, 2, 2, 128, [100, 3]),
    (17, 2, 1, 64, [90, 16]), (64, 4, 1, 128, [250, 0]), (64, 8, 8, 64, [133]), (26, 8, 1, 128, [500]), (33, 3, 1, 128, [129, 64]), (40, 8, 2, 128, [70, 300]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tree", ["tree", "chain"])
@pytest.mark.parametrize("window, sinks", [(1, 0), (3, 20), (16, 0), (33, 4), (64, 16), (100, 1), (1000, 5), (2 ** 31 - 1, 2 ** 31 - 1), (0, 7)])
@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window_attention(dtype, tree, window, sinks, case):
    t, hq, hkv, d, lens = WINDOWS[case]
    c = _attn_case(np.random.default_rng(1000 + case), len(lens), t, hq, hkv, d, lens, dtype, tree)
    _hide(c, window, sinks)
    out, lse, ws, _, _ = _window_run(c, window, sinks)
    assert mt.read_status(ws) == 0
    _window_check(c, out, lse, window, sinks)


@pytest.mark.parametrize("t, hq, hkv", [(1, 8, 2), (4, 8, 2), (24, 8, 2), (64, 4, 1), (4, 18, 2)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (900, 4)])
def test_window_attention_long_sequences_in_pieces(t, hq, hkv, window, sinks):
    lens = [3000, 40, 1100, 2047]
    c = _attn_case(np.random.default_rng(20 + t), 4, t, hq, hkv, 128, lens, "bf16", "tree")
    _hide(c, window, sinks)
    out, lse, ws, _, _ = _window_run(c, window, sinks)
    assert mt.read_status(ws) == 0
    _window_check(c, out, lse, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv, d", [(6, 6, 2, 128), (44, 12, 4, 64), (64, 7, 1, 128), (61, 14, 2, 64), (9, 24, 1, 128), (3, 200, 2, 64),
                                           (64, 5, 1, 128), (26, 5, 1, 64), (64, 3, 1, 128), (33, 65, 1, 64), (2, 127, 1, 128)])
@pytest.mark.parametrize("lens", [[40, 0, 300], [2500, 700]])
def test_window_attention_of_trees_with_odd_groups(dtype, t, hq, hkv, d, lens):
    # query heads a KV head that do not divide a tile's 128 rows: tiles of whole nodes, one or more a head
    c = _attn_case(np.random.default_rng(63), len(lens), t, hq, hkv, d, lens, dtype, "tree")
    window = 200 if d == 64 else 1000
    _hide(c, window, 5)
    out, lse, ws, _, _ = _window_run(c, window, 5)
    assert mt.read_status(ws) == 0
    _window_check(c, out, lse, window, 5)
    other, lse2, _, _, _ = _window_run(c, window, 5, ws=ws)
    assert torch.equal(other, out) and torch.equal(lse, lse2)


@pytest.mark.parametrize("t, hq, hkv", [(20, 6, 2), (64, 7, 1)])
def test_a_log_sum_exp_leaves_the_output_of_odd_groups(t, hq, hkv):
    c = _attn_case(np.random.default_rng(64), 3, t, hq, hkv, 128, [700, 20, 64], "bf16")
    out, _, _, args, kw = _window_run(c, 0, 0)
    plain = torch.full_like(out, 5.0)
    mt.tree_attn_paged_block8(*args[:8], plain, **{k: kw[k] for k in ("k_new", "v_new", "workspace")})
    assert torch.equal(out, plain)


@pytest.mark.parametrize("t, hq, hkv", [(3, 8, 2), (24, 8, 2)])
def test_window_zero_is_the_call_without_one(t, hq, hkv):
    c = _attn_case(np.random.default_rng(31), 3, t, hq, hkv, 128, [700, 20, 64], "bf16")
    out, _, _, args, kw = _window_run(c, 0, 9)
    plain = torch.full_like(out, 5.0)
    mt.tree_attn_paged_block8(*args[:8], plain, **{k: kw[k] for k in ("k_new", "v_new", "workspace")})
    assert torch.equal(out, plain)


def test_window_attention_scale_many_sequences_and_no_lse():
    rng = np.random.default_rng(32)
    lens = [int(n) for n in rng.integers(-1, 150, 300)]
    for t, dtype in ((1, "f16"), (20, "bf16")):
        c = _attn_case(rng, 300, t, 2, 1, 64, lens, dtype, "chain")
        _hide(c, 37, 3)
        out, _, ws, _, _ = _window_run(c, 37, 3, sm_scale=0.05, lse=False)
        assert mt.read_status(ws) == 0
        _window_check(c, out, None, 37, 3, sm_scale=0.05)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", [(6, 4, 2), (8, 8, 4), (6, 18, 2), (40, 8, 2), (64, 16, 4)])  # both kernels
@pytest.mark.parametrize("lens", [[90], [300, 2000]])  # whole segments, and ones in pieces
def test_window_attention_nan_in_and_out_of_sight(dtype, t, hq, hkv, lens):
    # NaN codes in the keys and values of slots that nobody sees, and values' at the window's edge, which the deeper
    # nodes do not see; the sinks' page has both kinds too
    window, sinks = 40, 5
    c = _attn_case(np.random.default_rng(33), len(lens), t, hq, hkv, 128, lens, dtype, "chain")
    for i, n in enumerate(lens):
        far = n - window + 1
        for s in (sinks, 15, far - 1, far - 2):
            c["k"][c["table"][i, s // P], :, s % P, 3] = c["v"][c["table"][i, s // P], :, s % P, 70] = 0x7F
        for s, col in ((far, 9), (far + 2, 127), (far + 3, 0)):  # seen by nodes 0, 0 .. 2, 0 .. 3
            c["v"][c["table"][i, s // P], 0, s % P, col] = 0xFF
    _hide(c, window, sinks)
    out, lse, ws, _, _ = _window_run(c, window, sinks)
    assert mt.read_status(ws) == 0
    _window_check(c, out, lse, window, sinks)
    assert out.isnan().any() and not out[:, 4:].isnan().any()


def test_window_attention_reports_bad_pages_in_sight_alone():
    c = _attn_case(np.random.default_rng(34), 2, 4, 4, 2, 64, [150, 20], "f16")
    c["table"][0, 3] = 99  # out of sight
    assert mt.read_status(_window_run(c, 30, 4)[2]) == 0
    c["table"][0, 8] = 99
    assert mt.read_status(_window_run(c, 30, 4)[2]) == -4
    c["table"][0, 8] = 0
    c["lens"] = [161, 20]  # past the table, whatever the window
    assert mt.read_status(_window_run(c, 30, 4)[2]) == -4
    c["lens"] = [150, 20]
    c["parents"][1, 2] = 3
    assert mt.read_status(_window_run(c, 30, 4)[2]) == -3


@pytest.mark.parametrize("t", [1, 20])
def test_window_attention_in_a_graph_with_other_lengths(t):
    c = _attn_case(np.random.default_rng(35), 4, t, 8, 2, 128, [700, 20, 64, 333], "bf16")
    out, lse, ws, args, kw = _window_run(c, 100, 4)
    _window_check(c, out, lse, 100, 4)
    g = _graph(lambda: mt.tree_attn_paged_block8(*args, **kw))
    args[6].copy_(_i32([101, 20, -1, 5]))
    out.fill_(5.0)
    lse.fill_(5.0)
    g.replay()
    c["lens"] = [101, 20, -1, 5]
    _window_check(c, out, lse, 100, 4)
    assert mt.read_status(ws) == 0


def test_window_attention_shares_a_workspace_with_any_call():
    rng = np.random.default_rng(36)
    cases = [_attn_case(rng, 2, t, 8, 2, 128, [1500, 200], dt) for t, dt in ((1, "bf16"), (12, "f16"), (40, "bf16"))]
    sizes = [(0, 0), (64, 4), (700, 0)]
    own = [[_window_run(c, w, s) for w, s in sizes] for c in cases]
    ws = torch.zeros(max(x[2].numel() for o in own for x in o), dtype=torch.uint8, device="cuda")
    for i, j in ((0, 1), (1, 1), (2, 2), (0, 0), (2, 1), (1, 2), (0, 2), (2, 0), (1, 0), (0, 1)):
        out, lse, _, _, _ = _window_run(cases[i], *sizes[j], ws=ws)
        assert torch.equal(out, own[i][j][0]) and torch.equal(lse, own[i][j][1])
    assert mt.read_status(ws) == 0


@pytest.mark.parametrize("t", [1, 20])
def test_window_attention_of_a_very_long_sequence(t):
    # positions near 2^31 behind a table of as many entries; only the pages in sight exist
    n, window, sinks, d = 2 ** 31 - 4096 - 200, 50, 20, 64
    rng = np.random.default_rng(37)
    blocks = (n + 63) // P
    table = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    first = (n - window + 1) // P
    seen = [0, 1] + list(range(first, -(-n // P)))
    table[0, torch.tensor(seen, device="cuda")] = torch.arange(len(seen), dtype=torch.int32, device="cuda")
    short = _attn_case(rng, 1, t, 8, 2, d, [len(seen) * P], "bf16", "chain")
    short["table"] = np.arange(len(seen), dtype=np.int32)[None]
    short["k"], short["v"], short["ks"], short["vs"] = (short[x][:len(seen)] for x in ("k", "v", "ks", "vs"))
    short["k"] &= 0x77  # (no NaN)
    short["v"] &= 0x77
    # the same under a short numbering: 32 slots of sinks' pages, then the window
    short["lens"] = [n - 16 * (first - 2)]
    want, _, _, _, _ = _window_run(short, window, sinks)
    _window_check(short, want, None, window, sinks)
    q = short["q"].cuda()
    out, ws = torch.empty_like(q), mt.alloc_block8_workspace(q, _f8(short["k"]), table)
    mt.tree_attn_paged_block8(q, _f8(short["k"]), _f8(short["v"]), torch.from_numpy(short["ks"]).float().cuda(), torch.from_numpy(short["vs"]).float().cuda(),
                              table, _i32([n]).cuda(), None, out, k_new=short["kn"].cuda(), v_new=short["vn"].cuda(), workspace=ws, window=window, sinks=sinks)
    assert mt.read_status(ws) == 0
    tol = 2.0 ** -7 * want.abs().float() + 2.0 ** -7  # another split of the sum
    assert bool(((out.float() - want.float()).abs() <= tol).all())


# ---- weights of cached slots ---------------------------------------------------

def _lse_of(c, nodes=None):
    """The attention's log-sum-exp over the whole cache, from the call that returns it."""
    return _window_run(c, 0, 0)[1]


def _weights_check(c, prev, path, decay, in_place, seed=0, lse=None, sm_scale=0.0):
    """One call against the plain implementation; returns what it wrote."""
    rng = np.random.default_rng(seed)
    b, t, hq, d = c["q"].shape
    pages, hkv = c["k"].shape[:2]
    lse = _lse_of(c) if lse is None else lse
    old = rng.random((pages, hkv, P)).astype(np.float32) * 3
    w, ws = torch.from_numpy(old).cuda(), _status()
    out = w if in_place else torch.full_like(w, -7.0)
    kw = dict(prev_lens=None if prev is None else _i32(prev).cuda(), decay=decay, status_ws=ws, sm_scale=sm_scale)
    if path is not None:
        kw |= dict(accept_path=_i32(path[0]).cuda(), accept_len=_i32(path[1]).cuda())
    got = mt.kv_attn_weights(c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w,
                             out=None if in_place else out, **kw)
    assert got is out and mt.read_status(ws) == 0
    nodes = (lambda i: range(t)) if path is None else (lambda i: path[0][i][:path[1][i] + 1])
    want, tol = lref.weights64(c, old, lse.cpu().double().numpy(), c["lens"], c["lens"] if prev is None else prev, nodes, decay, sm_scale or d ** -0.5)
    got = got.cpu().double().numpy()
    live = np.zeros(old.shape, bool)
    for i, n in enumerate(c["lens"]):
        for s in range(max(n, 0)):
            live[c["table"][i][s // P], :, s % P] = True
    bad = np.abs(got - want) > tol
    assert not bad[live].any(), np.argwhere(bad & live)[:4]
    assert (got[~live] == (old.astype(np.float64)[~live] if in_place else -7.0)).all()
    return got


WEIGHTS = [  # T, Hq, Hkv, D, lengths
    (1, 1, 1, 64, [0, 1, 40]), (1, 8, 2, 128, [17, -1, 300]), (2, 3, 3, 64, [5, 140]), (5, 12, 4, 128, [200, -1, 31]), (1, 7, 1, 128, [15, 16, 33]),
    (17, 2, 1, 64, [90, 16]), (64, 4, 1, 128, [250, 0]), (64, 9, 1, 128, [70, 40]), (64, 8, 8, 64, [133]), (33, 3, 1, 128, [129, 64]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("which", ["all", "path", "decayed"])
@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_slot_weights(dtype, which, case):
    t, hq, hkv, d, lens = WEIGHTS[case]
    rng = np.random.default_rng(2000 + case)
    c = _attn_case(rng, len(lens), t, hq, hkv, d, lens, dtype, "tree")
    path = None
    if which == "path":
        depth = min(t, 6)
        rows = np.stack([np.concatenate([np.sort(rng.permutation(t)[:depth]), [-1]]) for _ in lens])  # one place more than the longest
        path = rows, rng.integers(0, depth, len(lens))
    prev = [max(n - 20, 0) for n in lens] if which == "decayed" else None
    _weights_check(c, prev, path, 0.9 if which == "decayed" else 1.0, in_place=case % 2 == 0, seed=case)


def test_slot_weights_long_batch_scale_and_sum():
    c = _attn_case(np.random.default_rng(41), 3, 1, 8, 2, 128, [3000, 40, 2047], "bf16", "chain")
    _weights_check(c, [0, 40, 5000], None, 0.5, True)
    lse = torch.randn(3, 1, 8, device="cuda")
    _weights_check(c, None, None, 1.0, False, lse=lse, sm_scale=0.03)
    # the weights of a step's rows, and of their own new token, are shares of 1
    got = _weights_check(c, [0, 0, 0], None, 1.0, True)
    for i, n in enumerate(c["lens"]):
        pages = c["table"][i][np.arange(n) // P]
        total = got[pages, :, np.arange(n) % P].sum(0)  # per KV head: 4 rows
        assert (total < 4.001).all() and (total > 3.0 * n / (n + 20)).all()


def test_slot_weights_of_many_rows_a_head():
    c = _attn_case(np.random.default_rng(42), 1, 64, 40, 2, 64, [100], "f16", "chain")  # 1280 rows: five passes
    _weights_check(c, [33], None, 0.7, True)
    _weights_check(c, [33], None, 0.7, False)


def test_slot_weights_status_and_what_errors_leave():
    c = _attn_case(np.random.default_rng(43), 2, 4, 4, 2, 64, [50, 20], "f16")
    lse = torch.zeros(2, 4, 4, device="cuda")
    run = lambda **kw: mt.kv_attn_weights(c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse,  # noqa: E731
                                          **{**dict(weights=w, status_ws=ws), **kw})
    for bad in ("page", "length", "path", "node"):
        w, ws, kw = torch.ones(c["k"].shape[0], 2, P, device="cuda"), _status(), {}
        table, lens, touched = c["table"].copy(), list(c["lens"]), set(c["table"][1][:2])
        if bad == "page":
            touched |= {c["table"][0][p] for p in (0, 1, 3)}
            c["table"][0, 2] = c["k"].shape[0]
        elif bad == "length":
            c["lens"][0] = 65
        else:
            kw = dict(accept_path=_i32([[0, 1], [0, 1]]).cuda(), accept_len=_i32([1, 1]).cuda())
            kw["accept_path" if bad == "node" else "accept_len"][0] = 4 if bad == "node" else 2
        run(**kw)
        assert mt.read_status(ws) == -4, bad
        left = torch.tensor([p not in touched for p in range(len(w))])
        assert bool((w.cpu()[left] == 1).all()) and not bool((w.cpu()[~left][:, :, 0] == 1).any()), bad
        c["table"], c["lens"] = table, lens


def test_slot_weights_infinities_and_nan():
    c = _attn_case(np.random.default_rng(44), 2, 3, 4, 2, 64, [50, 20], "bf16", "chain")
    c["k"][c["table"][0][1], 1, 4, 9] = 0x7F  # a cached key of one head
    c["q"][1, 2, 0, 5] = float("inf")
    lse = torch.zeros(2, 3, 4, device="cuda")
    lse[0, 1, 0] = float("inf")  # a row that gives nothing
    w, ws = torch.zeros(c["k"].shape[0], 2, P, device="cuda"), _status()
    mt.kv_attn_weights(c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w, status_ws=ws)
    want = np.zeros(w.shape, bool)
    want[c["table"][0][1], 1, 4] = True
    want[c["table"][1][0], 0, :] = want[c["table"][1][1], 0, :4] = True
    assert np.array_equal(w.isnan().cpu().numpy(), want)


def test_slot_weights_in_a_graph_on_another_stream_and_the_same_twice():
    c = _attn_case(np.random.default_rng(45), 4, 2, 8, 2, 128, [700, 20, 64, 333], "bf16", "chain")
    lse = _lse_of(c)
    w, ws, out = torch.rand(c["k"].shape[0], 2, P, device="cuda"), _status(), None
    out = torch.zeros_like(w)
    args = (c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w)
    mt.kv_attn_weights(*args, out=out, status_ws=ws)
    want = out.clone()
    g = _graph(lambda: mt.kv_attn_weights(*args, out=out, status_ws=ws))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.zeros_like(w)
    s.wait_stream(torch.cuda.current_stream())
    mt.kv_attn_weights(*args, out=other, status_ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(other, want)


@pytest.mark.parametrize("t", [1, 40])  # both kernels
def test_slot_weights_far_pages(t):
    c = _attn_case(np.random.default_rng(46), 2, t, 16, 8, 128, [200, 77], "bf16", "chain")
    lse, far, n = _lse_of(c), 300000, c["k"].shape[0]  # a page behind byte 2^32
    table, ws = _i32(c["table"]).cuda(), _status()
    k, ks = torch.empty((far + n, 8, P, 128), dtype=torch.uint8, device="cuda"), torch.empty((far + n, 8), device="cuda")
    k[far:], ks[far:] = torch.from_numpy(c["k"]).cuda(), torch.from_numpy(c["ks"]).float().cuda()
    w, v = torch.zeros(far + n, 8, P, device="cuda"), torch.zeros(n, 8, P, device="cuda")
    args = (c["q"].cuda(), _i32(c["lens"]).cuda(), lse)
    mt.kv_attn_weights(args[0], k.view(torch.float8_e4m3fn), ks, torch.where(table >= 0, table + far, table), *args[1:], w, status_ws=ws)
    mt.kv_attn_weights(args[0], _f8(c["k"]), ks[far:].contiguous(), table, *args[1:], v, status_ws=ws)
    assert torch.equal(w[far:], v) and not bool(w[:far].any()) and mt.read_status(ws) == 0


# ---- eviction -------------------------------------------------------------------

class Evict:
    """A cache of one kind with weights, tables and new pages, on both sides."""

    def __init__(self, rng, kind, dt, hkv, d, lens, budget, spread=2.0, width=1):
        self.cache, self.lens, self.budget, self.kind = None, lens, budget, kind
        need, after = [-(-max(n, 0) // P) for n in lens], [-(-min(max(n, 0), budget) // P) for n in lens]
        self.pages = sum(need) + sum(after) + 3
        perm, at = rng.permutation(self.pages), 0
        self.table, self.new = np.full((len(lens), max(width, *need)), -1, np.int32), np.full((len(lens), -(-budget // P) + 1), -1, np.int32)
        for b in range(len(lens)):
            for t, n in ((self.table, need[b]), (self.new, after[b])):
                t[b, :n] = perm[at:at + n]
                at += n
        self.cache = Cache(rng, kind, self.pages, hkv, d, dt)
        self.weights = np.exp(spread * rng.standard_normal((self.pages, hkv, P))).astype(np.float32)
        self.weights[rng.random(self.weights.shape) < 0.2] = 0  # ties

    def run(self, sinks, recent, status=0, **kw):
        self.w, self.ws = torch.from_numpy(self.weights).cuda(), _status()
        self.kept = torch.full((len(self.lens), self.weights.shape[1], self.budget), 77, dtype=torch.int32, device="cuda")
        c = self.cache
        self.args = (c.k, c.v, self.w, _i32(self.table).cuda(), _i32(self.lens).cuda(), _i32(self.new).cuda(), self.kept)
        self.kw = dict(sinks=sinks, recent=recent, k_scales=c.scales[0], v_scales=c.scales[1], status_ws=self.ws, **kw)
        assert mt.kv_evict(*self.args, **self.kw) is self.kept
        assert mt.read_status(self.ws) == status

    def check(self, sinks, recent):
        raw = [c.view(torch.uint8).numpy() for c in self.cache.host]  # the same memory; rows of bytes
        kept = lref.evict(self.kind, raw, getattr(self.cache, "host_scales", None), self.weights, self.table, self.lens, self.new, self.budget, sinks, recent)
        live = np.array([n >= 0 for n in self.lens])
        got = self.kept.cpu().numpy()
        assert np.array_equal(got[live], kept[live]) and (got[~live] == 77).all()
        self.cache.check()
        assert np.array_equal(self.w.cpu().numpy(), self.weights, equal_nan=True)


EVICTS = [  # heads, D, lengths, budget, sinks, recent
    (1, 64, [1], 1, 0, 0), (1, 64, [2], 1, 0, 1), (2, 128, [40, 0, 17], 16, 2, 5), (3, 64, [100, -1, 99, 33], 33, 33, 0), (2, 128, [500, 31, 32], 31, 0, 31),
    (2, 64, [70], 100, 10, 20), (8, 128, [300, 290, 1], 256, 4, 64), (1, 128, [1000], 999, 0, 0), (5, 128, [129], 64, 0, 0), (2, 64, [3000, 64], 65, 1, 1),
]


@pytest.mark.parametrize("kind, dtype", [("act", "f32"), ("act", "f16"), ("act", "bf16"), ("e4m3", "bf16"), ("block8", "bf16")])
@pytest.mark.parametrize("case", range(len(EVICTS)))
@pytest.mark.parametrize("width", [1, 400])  # few rows of short tables go through one kernel, of wide ones through two
def test_evict(kind, dtype, case, width):
    hkv, d, lens, budget, sinks, recent = EVICTS[case]
    e = Evict(np.random.default_rng(3000 + case), kind, DT[dtype], hkv, d, lens, budget, width=width)
    if kind == "block8":  # no NaN codes: a re-encoded one keeps no sign
        for c, h in zip((e.cache.k, e.cache.v), e.cache.host):
            h.view(torch.uint8).numpy()[...] &= 0xF7
            c.view(torch.uint8).copy_(h.view(torch.uint8).cuda())
    e.run(sinks, recent)
    e.check(sinks, recent)


@pytest.mark.parametrize("what", ["equal", "zero", "negative", "odd", "close", "two"])
@pytest.mark.parametrize("longest", [700, 44000, 60000])  # keys in shared memory, and more of them
def test_evict_ties_and_odd_weights(what, longest):
    rng = np.random.default_rng(50)
    e = Evict(rng, "e4m3", torch.bfloat16, 2, 64, [longest, 600], 500)
    w = e.weights
    if what == "equal":
        w[...] = 0.7
    elif what == "zero":
        w[...] = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
    elif what == "negative":
        w[...] = -w
    elif what == "odd":
        w[...] = rng.choice(np.array([np.nan, np.inf, -np.inf, 0, 1, -1e-42, 1e-42, 3e38], np.float32), w.shape)
    elif what == "close":
        w[...] = (np.float32(1).view(np.int32) + rng.integers(0, 40, w.shape).astype(np.int32)).view(np.float32)
    else:
        w[...] = np.where(rng.random(w.shape) < 0.05, 2.0, 1.0)
    e.run(4, 100)
    e.check(4, 100)


def test_evict_scales_far_apart():
    rng = np.random.default_rng(51)
    e = Evict(rng, "block8", torch.bfloat16, 2, 128, [400], 100)
    for x in range(2):
        e.cache.host[x].view(torch.uint8).numpy()[...] &= 0xF7
        (e.cache.k, e.cache.v)[x].view(torch.uint8).copy_(e.cache.host[x].view(torch.uint8).cuda())
        e.cache.host_scales[x][...] = 2.0 ** rng.integers(-64, 120, e.cache.host_scales[x].shape)
        e.cache.scales[x].copy_(torch.from_numpy(e.cache.host_scales[x]).float())
    e.run(3, 10)
    e.check(3, 10)


def test_evict_keeps_nan_codes():
    rng = np.random.default_rng(52)
    e = Evict(rng, "block8", torch.bfloat16, 1, 64, [200], 64)
    e.run(0, 0)
    kept = e.kept.cpu().numpy()[0, 0]
    src = e.cache.host[0].view(torch.uint8).numpy()[e.table[0][kept // P], 0, kept % P]
    got = _codes(e.cache.k)[e.new[0][np.arange(64) // P], 0, np.arange(64) % P]
    assert np.array_equal(np.isnan(ref.decode(got)), np.isnan(ref.decode(src))) and np.isnan(ref.decode(src)).any()


def test_evict_pages_of_a_prefix_that_two_sequences_share():
    rng = np.random.default_rng(53)
    e = Evict(rng, "act", torch.float16, 2, 64, [100, 140], 60)
    e.table[1, :4] = e.table[0, :4]
    e.run(2, 20)
    e.check(2, 20)  # the shared pages are where they were


@pytest.mark.parametrize("bad", ["length", "page", "new"])
def test_evict_status_and_what_errors_leave(bad):
    rng = np.random.default_rng(54)
    e = Evict(rng, "act", torch.bfloat16, 2, 64, [70, 60], 40)
    before, table, new, lens = [c.clone() for c in e.cache.host], e.table.copy(), e.new.copy(), list(e.lens)
    untouched = set(range(e.pages)) - set(new[1][:3])
    if bad == "length":
        e.lens[0] = 81
    elif bad == "page":  # the recent rows' page: slots 64 .. 69 are new slots 34 .. 39, of the third new page
        e.table[0, 4] = e.pages
        untouched -= set(new[0][:2])
    else:
        e.new[0, 1] = -1
        untouched -= {new[0][0], new[0][2]}
    e.run(0, 6, status=-4)
    for c, h in zip((e.cache.k, e.cache.v), before):
        for p in untouched:
            assert torch.equal(c[p].cpu(), h[p]), (bad, p)
    # the other sequence is as it should be
    e.table, e.new, e.lens = table, new, lens
    kept = lref.evict("act", [h.view(torch.uint8).numpy() for h in e.cache.host], None, e.weights, table, [-1, 60], new, 40, 0, 6)
    assert np.array_equal(e.kept.cpu().numpy()[1], kept[1])
    for p in new[1][:2]:
        assert torch.equal(e.cache.k[p].cpu(), e.cache.host[0][p])


def test_evict_in_a_graph_with_other_lengths_and_twice_the_same():
    rng = np.random.default_rng(55)
    e = Evict(rng, "block8", torch.bfloat16, 2, 64, [200, 170, 64], 64)
    for c, h in zip((e.cache.k, e.cache.v), e.cache.host):
        h.view(torch.uint8).numpy()[...] &= 0xF7
        c.view(torch.uint8).copy_(h.view(torch.uint8).cuda())
    e.run(4, 16)
    first = e.kept.clone()
    mt.kv_evict(*e.args, **e.kw)  # the old pages are still there
    assert torch.equal(e.kept, first)
    e.check(4, 16)
    g = _graph(lambda: mt.kv_evict(*e.args, **e.kw))
    e.lens = [100, 30, -1]
    e.args[4].copy_(_i32(e.lens))
    e.kept.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    e.check(4, 16)
    assert mt.read_status(e.ws) == 0


@pytest.mark.parametrize("kind", ["act", "block8"])
def test_evict_far_pages(kind):
    rng = np.random.default_rng(56)
    hkv, d, far = 8, 128, 300000  # a page behind byte 2^32 and, in 16 bits, element 2^32
    e = Evict(rng, kind, torch.bfloat16, hkv, d, [100, 37], 48)
    e.run(2, 8)
    n, c = e.pages, e.cache
    big = [torch.empty((far + n, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in (c.k, c.v, e.w)]
    for x, y in zip(big, (c.k, c.v, e.w)):
        x.view(torch.uint8)[far:] = y.view(torch.uint8)
        x.view(torch.uint8)[torch.from_numpy(far + e.new[e.new >= 0]).cuda()] = 0
    scales = [None, None]
    if kind == "block8":
        scales = [torch.ones(far + n, hkv, device="cuda") for _ in range(2)]
        for x, y in zip(scales, c.scales):
            x[far:] = y
    move = lambda t: torch.where(t >= 0, t + far, t)  # noqa: E731
    kept = torch.zeros_like(e.kept)
    mt.kv_evict(*big, move(e.args[3]), e.args[4], move(e.args[5]), kept, sinks=2, recent=8, k_scales=scales[0], v_scales=scales[1], status_ws=e.ws)
    assert mt.read_status(e.ws) == 0 and torch.equal(kept, e.kept)
    for b, m in enumerate([48, 37]):
        for j in range(0, m, P):
            p, rows = int(e.new[b, j // P]), min(P, m - j)
            for x, y in zip(big, (c.k, c.v, e.w)):
                assert torch.equal(x[far + p, :, :rows].view(torch.uint8), y[p, :, :rows].view(torch.uint8))


# ---- logits ----------------------------------------------------------------------

def _logits_case(rng, b, t, v, dtype, history=0, bias=0, masks=0, tree="tree", per_row=False):
    """Inputs on the host; every kind of token id out of the vocabulary among them."""
    c = dict(x=_rand(rng, b, t, v, dtype=DT[dtype], scale=4.0), history=None, lens=None, starts=None, rep=None, pres=None, freq=None, bias=None, mask=None,
             index=None, tokens=None, parents=None)
    few = lambda *shape: np.minimum((v ** rng.random(shape)).astype(np.int64), v - 1)  # noqa: E731
    if history:
        c["history"] = np.where(rng.random((b, history)) < 0.05, rng.choice([-1, v, -2 ** 31, 2 ** 31 - 1], (b, history)), few(b, history))
        c["lens"], c["starts"] = rng.integers(0, history + 5, b), rng.integers(-2, history, b)
        c["rep"], c["pres"], c["freq"] = (rng.choice(a, b).astype(np.float32) for a in ([1.0, 1.3, 0.8], [0.0, 0.7, -0.4], [0.0, 0.31, -0.2]))
    if bias:
        c["bias"] = np.where(rng.random((b, bias)) < 0.2, rng.choice([-1, v], (b, bias)), few(b, bias)), (3 * rng.standard_normal((b, bias))).astype(np.float32)
    if masks:
        n = b * t if per_row else masks
        c["mask"] = rng.random((n, v)) < rng.choice([0.0, 0.01, 0.5, 0.99, 1.0], (n, 1))
        c["index"] = None if per_row else rng.integers(-1, masks + 1, (b, t))
    if tree:
        c["tokens"] = np.where(rng.random((b, t)) < 0.1, rng.choice([-1, v], (b, t)), few(b, t))
        c["parents"] = None if tree == "chain" else np.array([[-1] + [int(rng.integers(max(0, j - 9), j)) for j in range(1, t)] for _ in range(b)])
    return c


def _bits(mask):
    pad = np.pad(mask, ((0, 0), (0, -mask.shape[1] % 32)))
    return torch.from_numpy(np.packbits(pad, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def _logits_kw(c, ws, two=False):
    i32 = lambda x: None if x is None else _i32(x).cuda()  # noqa: E731
    f32 = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    flat = lambda x: x if x is None or not two else x[:, 0]  # noqa: E731
    return dict(history=i32(c["history"]), history_lens=i32(c["lens"]), output_starts=i32(c["starts"]), repetition=f32(c["rep"]), presence=f32(c["pres"]), frequency=f32(c["freq"]),
                bias_tokens=i32(c["bias"] and c["bias"][0]), bias_values=f32(c["bias"] and c["bias"][1]), mask=None if c["mask"] is None else _bits(c["mask"]),
                mask_index=flat(i32(c["index"])), tree_tokens=flat(i32(c["tokens"])), tree_parents=flat(i32(c["parents"])), status_ws=ws)


def _logits_check(c, got, left=None):
    """`left`: what rows without a sequence hold."""
    x = c["x"]
    want, mag, touched = lref.logits64(x.double().numpy(), c["history"], c["lens"], c["starts"], c["rep"], c["pres"], c["freq"], c["bias"], c["mask"], c["index"], c["tokens"],
                                       c["parents"])
    got = got.cpu()
    live = torch.from_numpy(np.array([c["lens"] is None or n >= 0 for n in (c["lens"] if c["lens"] is not None else [0] * len(x))]))
    same = torch.from_numpy(~touched) & live[:, None, None]
    raw = {4: torch.int32, 2: torch.int16}[x.element_size()]
    assert torch.equal(got.view(raw)[same], x.view(raw)[same])  # untouched entries keep their bits
    y, lost = got.double().numpy(), np.isneginf(want)
    assert np.array_equal(np.isneginf(y)[live.numpy()], lost[live.numpy()])
    fine = touched & ~lost & live.numpy()[:, None, None]
    # the rounding at the end and four in 32 bits before it
    tol = ref.HALF_STEP[x.dtype] * np.abs(want) + 4 * 2.0 ** -24 * mag + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    bad = np.abs(y - np.where(lost, 0, want)) > tol
    assert not bad[fine].any(), np.argwhere(bad & fine)[:4]
    if left is not None:
        assert torch.equal(got[~live], left.cpu()[~live])


LOGITS = [  # B, T, V, history, bias, masks, tree
    (1, 1, 1, 3, 0, 0, None), (1, 1, 33, 10, 5, 2, None), (3, 1, 1000, 100, 0, 0, None), (2, 5, 4097, 700, 30, 3, "tree"), (1, 64, 1003, 50, 9, 0, "tree"),
    (2, 64, 32000, 2000, 0, 9, "tree"), (4, 3, 8192, 0, 0, 4, "chain"), (5, 1, 32001, 3000, 50, 0, "chain"), (2, 100, 500, 20, 4, 3, None), (1, 1, 200000, 5000, 300, 1, None),
    (300, 1, 70, 9, 3, 8, None), (2, 7, 12345, 40, 0, 2, "chain"),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(LOGITS)))
def test_logits(dtype, in_place, case):
    b, t, v, history, bias, masks, tree = LOGITS[case]
    c = _logits_case(np.random.default_rng(4000 + case), b, t, v, dtype, history, bias, masks, tree)
    x, ws = c["x"].cuda(), _status()
    out = x if in_place else torch.full_like(x, 7.0)
    assert mt.process_logits(x, out, **_logits_kw(c, ws)) is out and mt.read_status(ws) == 0
    _logits_check(c, out)
    if not in_place:
        assert torch.equal(x.cpu(), c["x"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_each_part_alone_and_nothing(dtype):
    rng = np.random.default_rng(60)
    full = _logits_case(rng, 3, 4, 999, dtype, 60, 10, 3, "tree")
    keep = {"x": full["x"]}
    for names in ((), ("rep", "history", "lens"), ("pres", "history", "lens"), ("freq", "history", "lens", "starts"), ("bias",), ("mask", "index"), ("tokens", "parents", "freq"),
                  ("tokens", "rep"), ("history", "lens")):
        c = {k: None for k in full} | keep | {n: full[n] for n in names}
        for in_place in (False, True):
            x, ws = c["x"].cuda(), _status()
            out = x if in_place else torch.full_like(x, 7.0)
            mt.process_logits(x, out, **_logits_kw(c, ws))
            assert mt.read_status(ws) == 0
            _logits_check(c, out)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("shift, out_shift", [(0, 0), (1, 1), (3, 0), (0, 5), (2, 3)])
def test_logits_strides_and_alignment(dtype, shift, out_shift):
    rng = np.random.default_rng(61)
    c = _logits_case(rng, 3, 2, 501, dtype, 60, 10, 3, "chain", per_row=True)
    wide, to = torch.full((3, 5, 600), 9.0, dtype=DT[dtype], device="cuda"), torch.full((3, 3, 611), 9.0, dtype=DT[dtype], device="cuda")
    x, out = wide[:, 1::2, shift:shift + 501], to[:, :2, out_shift:out_shift + 501]
    x.copy_(c["x"])
    ws, kw = _status(), None
    kw = _logits_kw(c, ws)
    mt.process_logits(x, out, **kw)
    _logits_check(c, out)
    rest = to.clone()
    rest[:, :2, out_shift:out_shift + 501] = 9.0
    assert bool((rest == 9.0).all())  # nothing beside the rows
    mt.process_logits(x, x, **kw)
    _logits_check(c, x)
    both = torch.empty(2, 3, 501, dtype=DT[dtype], device="cuda").transpose(0, 1)  # rows of a sequence far apart
    mt.process_logits(both.copy_(c["x"]), both, **kw)
    _logits_check(c, both)
    one = torch.empty(3, 2, 501, dtype=DT[dtype], device="cuda")
    mt.process_logits(c["x"][:1, :1].cuda().expand(3, 2, 501), one, status_ws=ws)  # one row read by all
    assert torch.equal(one.cpu(), c["x"][:1, :1].expand(3, 2, 501)) and mt.read_status(ws) == 0


def test_logits_two_dims_and_places_without_a_sequence():
    rng = np.random.default_rng(62)
    c = _logits_case(rng, 5, 1, 777, "bf16", 40, 4, 3, None)
    c["lens"] = np.array([30, -1, 0, 45, -7])
    x, ws = c["x"].cuda(), _status()
    out = torch.full((5, 777), 7.0, dtype=torch.bfloat16, device="cuda")
    mt.process_logits(x[:, 0], out, **_logits_kw(c, ws, two=True))
    _logits_check(c, out[:, None], left=torch.full_like(x, 7.0))
    y = x.clone()
    mt.process_logits(y, y, **_logits_kw(c, ws))
    _logits_check(c, y, left=x)
    assert mt.read_status(ws) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_logits_infinities_and_nan(dtype):
    x = torch.tensor([[float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 65504.0 if dtype == "f16" else 3e38, 1.0, -1.0] * 2], dtype=DT[dtype])
    history, ws = _i32([[0, 1, 2, 3, 4, 5, 6, 7]]).cuda(), _status()
    f = lambda a: torch.tensor([a], device="cuda")  # noqa: E731
    out = torch.empty_like(x).cuda()
    mt.process_logits(x.cuda(), out, history=history, history_lens=_i32([8]).cuda(), repetition=f(2.0), presence=f(0.5), frequency=f(0.25), status_ws=ws)
    y = x.float()[0, :8]
    want = torch.where(y > 0, y / 2, y * 2) - 0.25 - 0.5
    assert torch.equal(out[0, :8].cpu().isnan(), want.isnan()) and torch.equal(out[0, 1:8].cpu(), want[1:].to(x.dtype))
    assert torch.equal(out[0, 8:].cpu().nan_to_num(9), x[0, 8:].nan_to_num(9))
    none = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    mt.process_logits(x.cuda(), out, mask=none, mask_index=_i32([0]).cuda(), status_ws=ws)  # a NaN is masked like the rest
    assert bool((out == float("-inf")).all())
    mt.process_logits(x.cuda(), out, history=torch.empty(1, 0, dtype=torch.int32, device="cuda"), history_lens=_i32([3]).cuda(), status_ws=ws)
    assert torch.equal(out.cpu().nan_to_num(9), x.nan_to_num(9)) and mt.read_status(ws) == 0


def test_logits_of_a_bad_tree():
    c = _logits_case(np.random.default_rng(63), 2, 4, 300, "f32", 10, 0, 0, "tree")
    c["parents"][1] = [-1, 0, 2, 9]
    x, ws = c["x"].cuda(), _status()
    out = torch.empty_like(x)
    mt.process_logits(x, out, **_logits_kw(c, ws))
    assert mt.read_status(ws) == -3
    c["parents"][1] = [-1, 0, -1, -1]
    _logits_check(c, out)


def test_logits_in_a_graph_on_another_stream_and_the_same_twice():
    c = _logits_case(np.random.default_rng(64), 2, 6, 32000, "bf16", 500, 20, 3, "tree")
    x, ws = c["x"].cuda(), _status()
    kw, out = _logits_kw(c, ws), torch.empty_like(x)
    mt.process_logits(x, out, **kw)
    want = out.clone()
    g = _graph(lambda: mt.process_logits(x, out, **kw))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    other, s = torch.empty_like(x), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mt.process_logits(x, other, stream=s, **kw)
    s.synchronize()
    assert torch.equal(other, want)


def test_logits_far_rows():
    v, rows = 500000, 4500  # elements past 2^31
    x = torch.empty(rows, v, dtype=torch.float16, device="cuda")
    x[-1] = torch.arange(v, device="cuda") % 1000
    lens, ws = torch.full((rows,), -1, dtype=torch.int32, device="cuda"), _status()
    lens[-1] = 2
    history = torch.zeros(rows, 2, dtype=torch.int32, device="cuda")
    history[-1] = _i32([499999, 5]).cuda()
    before = x[-1].clone()
    mt.process_logits(x, x, history=history, history_lens=lens, presence=torch.ones(rows, device="cuda"), status_ws=ws)
    before[499999] -= 1
    before[5] -= 1
    assert torch.equal(x[-1], before) and mt.read_status(ws) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv, d, lens", [(64, 8, 2, 128, [3000, 1, 700, -1, 130]), (25, 2, 1, 64, [1027]), (64, 12, 2, 128, [260, 900]), (49, 4, 4, 64, [128, 127, 129]),
                                                  (64, 40, 4, 128, [500, 77])])
@pytest.mark.parametrize("which", ["all", "path"])
def test_slot_weights_of_chunks(dtype, t, hq, hkv, d, lens, which):
    # more rows a head than a few tiles of eight: the tensor-core path, in one pass and in more
    rng = np.random.default_rng(47)
    c = _attn_case(rng, len(lens), t, hq, hkv, d, lens, dtype, "tree")
    path = None
    if which == "path":
        rows = np.stack([np.sort(rng.permutation(t)) for _ in lens])
        path = rows, rng.integers(t - 25, t, len(lens))
        path[1][0] = 0  # one row
    prev = [max(n - 150, 0) for n in lens]
    _weights_check(c, prev, path, 0.9, in_place=True, seed=t)


def test_slot_weights_of_many_sequences_in_chunks():
    rng = np.random.default_rng(48)
    lens = [int(n) for n in rng.integers(-1, 300, 200)]
    c = _attn_case(rng, 200, 20, 8, 2, 64, lens, "bf16", "chain")
    _weights_check(c, None, None, 1.0, False)


def test_slot_weights_of_chunks_bad_paths_and_pages():
    rng = np.random.default_rng(49)
    c = _attn_case(rng, 3, 64, 4, 2, 64, [300, 200, 40], "bf16", "chain")
    lse, ws = torch.zeros(3, 64, 4, device="cuda"), _status()
    w = torch.ones(c["k"].shape[0], 2, P, device="cuda")
    path = np.tile(np.arange(64), (3, 1))
    path[1, 5] = 64
    c["table"][0, 3] = -5
    mt.kv_attn_weights(c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w,
                       accept_path=_i32(path).cuda(), accept_len=_i32([40, 40, 40]).cuda(), status_ws=ws)
    assert mt.read_status(ws) == -4
    touched = {p for p in c["table"][0][:19] if p >= 0} | set(c["table"][2][:3])
    left = torch.tensor([p not in touched for p in range(len(w))])
    assert bool((w.cpu()[left] == 1).all()) and not bool((w.cpu()[~left][:, :, 0] == 1).any())


def test_slot_weights_nan_among_chunks():
    c = _attn_case(np.random.default_rng(57), 2, 40, 8, 2, 128, [250, 130], "bf16", "chain")
    c["k"][c["table"][0][1], 1, 4, 9] = 0x7F
    c["k"][c["table"][1][8], 0, 5, 9] = 0x7F  # behind the second sequence's end
    c["q"][1, 2, 0, 5] = float("inf")
    lse = torch.zeros(2, 40, 8, device="cuda")
    w, ws = torch.zeros(c["k"].shape[0], 2, P, device="cuda"), _status()
    mt.kv_attn_weights(c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w, status_ws=ws)
    want = np.zeros(w.shape, bool)
    want[c["table"][0][1], 1, 4] = True
    for s in range(130):
        want[c["table"][1][s // P], 0, s % P] = True
    assert np.array_equal(w.isnan().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("span", [3, 5, 7, 12])
def test_slot_weights_rows_of_unlike_size(dtype, d, span):
    # rows' largest values 2^0 to 2^-span, some rows of zeros; the second pass has like ones, or the other way round
    rng = np.random.default_rng(61)
    c = _attn_case(rng, 2, 40, 16, 2, d, [300, 129], dtype, "chain")
    size = torch.from_numpy(2.0 ** -rng.integers(0, span + 1, (2, 40, 16)))
    size[torch.from_numpy(rng.random((2, 40, 16)) < 0.02)] = 0
    size[0, 33:], size[1, :31] = 0.5, 0.25
    c["q"] = (c["q"].double() * size[..., None]).to(c["q"].dtype)
    _weights_check(c, None, None, 1.0, False)


def test_slot_weights_of_zero_keys_behind_large_scales():
    c = _attn_case(np.random.default_rng(62), 1, 64, 4, 1, 128, [100], "bf16", "chain")
    c["q"] = (c["q"].float() * 2.0 ** 100).to(torch.bfloat16)
    lse = torch.zeros(1, 64, 4, device="cuda")
    w, ws = torch.zeros(c["k"].shape[0], 1, P, device="cuda"), _status()
    ks = torch.full((c["k"].shape[0], 1), 2.0 ** 100, device="cuda")
    mt.kv_attn_weights(c["q"].cuda(), torch.zeros_like(_f8(c["k"])), ks, _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w, status_ws=ws)
    pages, at = c["table"][0][np.arange(100) // P], np.arange(100) % P
    assert (w.cpu().numpy()[pages, 0, at] == 256).all() and float(w.sum()) == 25600


def test_slot_weights_wait_bound():
    """A pipeline wait that only its bound ends: the status says so, and the next call is right."""
    c = _attn_case(np.random.default_rng(58), 2, 32, 8, 2, 128, [100, 400], "bf16", "chain")
    lse = _lse_of(c)
    w, ws = torch.zeros(c["k"].shape[0], 2, P, device="cuda"), _status()
    args = (c["q"].cuda(), _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w)
    try:
        mt.debug_set_wait(20_000_000, stall=True)
        mt.kv_attn_weights(*args, status_ws=ws)
        assert mt.read_status(ws) == -6
    finally:
        mt.debug_set_wait()
    _weights_check(c, None, None, 1.0, True)


# ---- the operators together ---------------------------------------------------------

def test_a_long_conversation_in_a_bounded_cache():
    """Two layers, three turns: a tree step over the cache with its log-sum-exp, acceptance, the accepted path's weights,
    the path appended, the cache brought back to its budget, the next token drawn from processed logits; each result
    against the plain implementations, and the next turn on what this one left."""
    rng = np.random.default_rng(70)
    b, t, hq, hkv, d, v, dt = 2, 8, 8, 2, 128, 500, torch.bfloat16
    budget, sinks, recent = 48, 2, 12
    lens, blocks, pages = [61, 40], 6, 60
    free = [int(p) for p in rng.permutation(pages)]
    table = np.full((b, blocks), -1, np.int32)
    for i, n in enumerate(lens):
        for j in range(-(-(n + t) // P)):
            table[i, j] = free.pop()
    parents = np.array([[-1, 0, 0, 1, 1, 2, 3, 3]] * b)
    history = np.full((b, 40), -1, np.int32)
    history[:, :10] = rng.integers(0, v, (b, 10))
    said = [10, 10]  # tokens of each history; the first ten are the prompt's
    ws = _status()

    def cache():
        c = dict(k=np.zeros((pages, hkv, P, d), np.uint8), v=np.zeros((pages, hkv, P, d), np.uint8), ks=np.ones((pages, hkv)), vs=np.ones((pages, hkv)))
        for x, s in (("k", "ks"), ("v", "vs")):
            for i, n in enumerate(lens):
                for p in range(-(-n // P)):
                    for h in range(hkv):
                        m = min(P, n - p * P)
                        c[x][table[i, p], h, :m], c[s][table[i, p], h] = ref.block_codes(rng.standard_normal((m, d)))
        c |= dict(K=_f8(c["k"]), V=_f8(c["v"]), KS=torch.from_numpy(c["ks"]).float().cuda(), VS=torch.from_numpy(c["vs"]).float().cuda(),
                  W=torch.rand(pages, hkv, P, device="cuda"), prev=list(lens))
        return c

    def back(c):
        """The layer's state on the host, as the last call left it."""
        c["k"], c["v"] = _codes(c["K"]).copy(), _codes(c["V"]).copy()
        c["ks"], c["vs"] = c["KS"].cpu().double().numpy(), c["VS"].cpu().double().numpy()

    layers = [cache() for _ in range(2)]
    for turn in range(3):
        tokens = rng.integers(0, v, (b, t))
        logits = _rand(rng, b, t, v, scale=2.0)
        end = [5, 3]
        for i, e in enumerate(end):  # the path to node e is accepted
            n = e
            while parents[i, n] >= 0:
                logits[i, parents[i, n], tokens[i, n]] = 30.0
                n = parents[i, n]
            for c in range(t):
                if parents[i, c] == e:
                    logits[i, e, tokens[i, c]] = -30.0
        alen, path = torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros(b, 4, dtype=torch.int32, device="cuda")
        mt.tree_accept_greedy(_i32(tokens).cuda(), logits.cuda(), _i32(parents).cuda(), alen, path, argmax_out=torch.zeros(b, t, dtype=torch.int32, device="cuda"),
                              next_token=torch.zeros(b, dtype=torch.int32, device="cuda"), workspace=mt.alloc_accept_workspace(b, t))
        hpath, hlen = path.cpu().numpy(), alen.cpu().numpy()
        assert hlen.tolist() == [2, 2] and [hpath[i, 2] for i in range(b)] == end
        dlens, dtab = _i32(lens).cuda(), _i32(table).cuda()
        grown = [n + int(m) + 1 for n, m in zip(lens, hlen)]
        new_table = np.full((b, blocks), -1, np.int32)
        for i, n in enumerate(grown):
            for j in range(-(-min(n, budget) // P)):
                new_table[i, j] = free.pop()
        for c in layers:
            q, kn, vn = (_rand(rng, b, t, h, d, dtype=dt, scale=s) for h, s in ((hq, 2.0), (hkv, 1.0), (hkv, 1.0)))
            step = dict(c, q=q, kn=kn, vn=vn, table=table, lens=lens, parents=parents)
            out, lse = torch.empty(b, t, hq, d, dtype=dt, device="cuda"), torch.empty(b, t, hq, device="cuda")
            aws = mt.alloc_block8_workspace(out, c["K"], dtab)
            attn = (q.cuda(), c["K"], c["V"], c["KS"], c["VS"], dtab, dlens, _i32(parents).cuda(), out)
            mt.tree_attn_paged_block8(*attn, k_new=kn.cuda(), v_new=vn.cuda(), workspace=aws, window=20, sinks=sinks)  # a windowed layer's view of it
            _window_check(step, out, None, 20, sinks)
            mt.tree_attn_paged_block8(*attn, k_new=kn.cuda(), v_new=vn.cuda(), workspace=aws, lse=lse)
            assert mt.read_status(aws) == 0
            _window_check(step, out, lse, 0, 0)
            old = c["W"].cpu().numpy()
            mt.kv_attn_weights(q.cuda(), c["K"], c["KS"], dtab, dlens, lse, c["W"], prev_lens=_i32(c["prev"]).cuda(), accept_path=path, accept_len=alen, decay=0.9, status_ws=ws)
            want, tol = lref.weights64(step, old, lse.cpu().double().numpy(), lens, c["prev"], lambda i: hpath[i][:hlen[i] + 1], 0.9, d ** -0.5)
            assert (np.abs(c["W"].cpu().double().numpy() - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
            mt.kv_append_accepted(kn.cuda(), vn.cuda(), path, alen, c["K"], c["V"], dtab, dlens, status_ws=ws, k_scales=c["KS"], v_scales=c["VS"])
            back(c)
            weights, kept = c["W"].cpu().numpy(), torch.empty(b, hkv, budget, dtype=torch.int32, device="cuda")
            mt.kv_evict(c["K"], c["V"], c["W"], dtab, _i32(grown).cuda(), _i32(new_table).cuda(), kept, sinks=sinks, recent=recent, k_scales=c["KS"], v_scales=c["VS"], status_ws=ws)
            want = lref.evict("block8", [c["k"], c["v"]], [c["ks"], c["vs"]], weights, table, grown, new_table, budget, sinks, recent)
            assert np.array_equal(kept.cpu().numpy(), want)
            assert np.array_equal(_codes(c["K"]), c["k"]) and np.array_equal(_codes(c["V"]), c["v"]) and np.array_equal(c["W"].cpu().numpy(), weights)
            assert np.array_equal(c["KS"].cpu().double().numpy(), c["ks"]) and np.array_equal(c["VS"].cpu().double().numpy(), c["vs"])
            c["prev"] = [min(n, budget) for n in grown]
        free += [int(p) for p in table.ravel() if p >= 0]
        table, lens = new_table, [min(n, budget) for n in grown]
        for i, n in enumerate(lens):  # room for the next tree
            for j in range(-(-n // P), -(-(n + t) // P)):
                table[i, j] = free.pop()
        # the next token: from the end nodes' logits, the path's tokens penalised, a grammar over one of them
        x = logits.cuda().clone()
        case = dict(x=logits, history=history, lens=np.array(said), starts=np.array([10, 10]), rep=np.float32([1.2, 1.0]), pres=np.float32([0.5, 0.0]), freq=np.float32([0.0, 0.3]),
                    bias=(np.array([[7], [8]]), np.float32([[2.0], [-1.0]])), mask=rng.random((1, v)) < 0.5, index=np.where(np.arange(t) == end[0], 0, -1)[None].repeat(b, 0),
                    tokens=tokens, parents=parents)
        mt.process_logits(x, x, **_logits_kw(case, ws))
        _logits_check(case, x)
        rows, u = [int(end[i]) + i * t for i in range(b)], rng.random(b)
        got = torch.empty(b, dtype=torch.int32, device="cuda")
        f32 = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
        mt.sample_tokens(x.view(b * t, v), f32(u), got, temperature=f32([0.8] * b), top_k=_i32([40] * b).cuda(), row_index=_i32(rows).cuda())
        f = lambda a: np.float64(np.float32(a))  # noqa: E731
        y = x.view(b * t, v).cpu().double().numpy()
        assert got.tolist() == [ref.sample64(y[rows[i]], f(u[i]), f(0.8), 40, 1.0, 0.0) for i in range(b)]
        for i in range(b):
            new = [int(tokens[i, n]) for n in hpath[i][:hlen[i] + 1]]
            history[i, said[i]:said[i] + len(new)] = new
            said[i] += len(new)
    assert mt.read_status(ws) == 0


@pytest.mark.parametrize("b, hkv, longest", [(100, 4, 300), (200, 2, 2500), (50, 8, 30000)])
def test_evict_many_rows(b, hkv, longest):
    # more rows than SMs: fewer threads for short tables, less shared memory for long ones
    rng = np.random.default_rng(59)
    lens = [int(n) for n in rng.integers(-1, 90, b)]
    lens[3], lens[b - 1] = longest, longest - 7
    e = Evict(rng, "e4m3", torch.bfloat16, hkv, 64, lens, 40)
    e.run(3, 9)
    e.check(3, 9)


@pytest.mark.parametrize("t, hq, hkv", [(41, 4, 2), (33, 2, 1), (16, 16, 2)])  # 82, 66 and 128 rows a head: a unit a pair of tiles
def test_slot_weights_of_one_unit_a_pair_of_tiles(t, hq, hkv):
    c = _attn_case(np.random.default_rng(68), 1, t, hq, hkv, 64, [9000], "bf16", "chain")
    lse = torch.zeros(1, t, hq, device="cuda")
    args = (c["q"].cuda() * 0.1, _f8(c["k"]), torch.from_numpy(c["ks"]).float().cuda(), _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse)
    ws, w = _status(), torch.zeros(c["k"].shape[0], hkv, P, device="cuda")
    mt.kv_attn_weights(*args, w, status_ws=ws)
    for _ in range(50):  # the CTAs' roles meet in another order every time
        again = torch.zeros_like(w)
        mt.kv_attn_weights(*args, again, status_ws=ws)
        assert torch.equal(again, w)
    assert mt.read_status(ws) == 0
    c["q"] = (c["q"].cuda() * 0.1).cpu()
    want, tol = lref.weights64(c, np.zeros(w.shape, np.float32), lse.cpu().double().numpy(), c["lens"], [0], lambda i: range(t), 1.0, 64 ** -0.5)
    assert (np.abs(w.cpu().double().numpy() - want) <= tol).all()
