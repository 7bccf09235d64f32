"""Places of the operators for long sequences where a result could go wrong without a size or a mask being odd: what one
lane leaves for another, extreme scales, queries with a dominant channel, scales that are not powers of two.  Against the
plain implementations in 64 bits (long_reference)."""
import bisect
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import long_reference as lref
import medusa_tree_speculative_attn_gb300 as mt
import serve_reference as ref
from test_gpu_long import Evict, _f8, _hide, _lse_of, _weights_check, _window_check, _window_run
from test_gpu_serve import P, _attn_case, _codes, _i32, _status

pytestmark = pytest.mark.gpu


# ---- attention under a window ------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t, hq, hkv", [(1, 4, 2), (3, 4, 2), (8, 8, 4), (6, 6, 2)])  # the register-fragment kernel's instances
def test_window_values_that_one_lane_changes_for_another(d, t, hq, hkv):
    # every value of every slot out of sight is a NaN code, in pages that are in sight in part: at the window's edge,
    # behind the sinks and behind the sequence's end.  A lane that read a value before another lane took it out of the
    # products would make its column NaN.
    window, sinks = 37, 5
    lens = [90, 301, 16 * 40 + 3, 52]
    c = _attn_case(np.random.default_rng(70), len(lens), t, hq, hkv, d, lens, "bf16", "chain")
    for i, n in enumerate(lens):
        for s in [*range(sinks, n - window + 1), *range(n, -(-n // P) * P)]:
            c["v"][c["table"][i, s // P], :, s % P] = 0x7F
    _hide(c, window, sinks)
    out, lse, ws, args, kw = _window_run(c, window, sinks)
    _window_check(c, out, lse, window, sinks)
    for _ in range(30):
        again = torch.full_like(out, 5.0)
        mt.tree_attn_paged_block8(*args[:8], again, **kw)
        assert torch.equal(again, out)
    assert mt.read_status(ws) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t, hq, hkv, n, window", [(3, 4, 2, 300, 30), (6, 6, 2, 2007, 700), (20, 4, 1, 300, 36), (40, 8, 2, 150, 40), (64, 7, 1, 2000, 1000)])
def test_window_attention_of_a_key_scale_that_some_rows_do_not_see(dtype, bad, t, hq, hkv, n, window):
    # the page at the window's edge has a key scale that is no number: rows that see one of its slots are none either (under
    # an infinity a score may be -inf, and its weight 0), and the deeper nodes, which see none, have what they would have
    c = _attn_case(np.random.default_rng(73), 1, t, hq, hkv, 128, [n], dtype, "chain")
    far = n - window + 1
    edge = [d for d in range(t) if (far + d) // P == far // P]  # depths that see a slot of that page
    assert edge and len(edge) < t
    want, mag, wlse = lref.window_attn64(c, window, 0, 128 ** -0.5)
    c["ks"][c["table"][0, far // P], 0] = bad
    _hide(c, window, 0)
    out, lse, ws, _, _ = _window_run(c, window, 0)
    got, glse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    g = hq // hkv
    assert np.isnan(got[:, edge, :g]).all() or bad == float("inf")
    calm = np.ones(got.shape[:3], bool)
    calm[:, edge, :g] = False
    tol = ref.HALF_STEP[c["q"].dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -8) * mag + 1e-7  # as test_gpu_long's
    assert (np.abs(got - want) <= tol)[calm].all()
    assert (np.abs(glse - wlse) <= 2.0 ** -9 + 2.0 ** -20 * (1 + np.abs(wlse)))[calm].all()
    assert mt.read_status(ws) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv, d, lens", [(1, 8, 2, 128, [0, 40, 700]), (4, 4, 2, 64, [2000, 1]), (6, 6, 2, 128, [333]), (24, 8, 2, 128, [90, 1500]), (64, 4, 1, 64, [500])])
@pytest.mark.parametrize("window, sinks, spread", [(0, 0, 2.0), (50, 4, 0.5), (300, 0, 6.0)])
def test_log_sum_exp_in_32_bits(dtype, t, hq, hkv, d, lens, window, sinks, spread):
    # Off by what a score is off by: 2 D 2^-24 sum |q k| for products and sums in 32 bits, and for each channel 2^-17 of the
    # row's largest |q| for what the parts of a query leave; and by 2^-20 of itself, the largest score and 1 for the units,
    # the exponentials, their sum and its logarithm.  The largest sum |q k| is at most the log-sum-exp of the magnitudes,
    # sum |k| that of queries of ones.
    c = _attn_case(np.random.default_rng(77), len(lens), t, hq, hkv, d, lens, dtype, "tree", spread=spread)
    sm = d ** -0.5
    for i, n in enumerate(lens):  # no NaN codes in sight of a row, or of its page
        c["k"][c["table"][i][:-(-n // P)]] &= 0xF7
    _, _, want = lref.window_attn64(c, window, sinks, sm)
    mags = dict(c, q=c["q"].abs(), kn=c["kn"].abs(), k=c["k"] & 0x7F)
    _, _, products = lref.window_attn64(mags, window, sinks, sm)
    _, _, keys = lref.window_attn64(dict(mags, q=torch.ones_like(c["q"])), window, sinks, sm)
    top = c["q"].double().abs().amax(-1).numpy()
    tol = 2 * d * 2.0 ** -24 * products + 2.0 ** -17 * top * keys + 2.0 ** -20 * (1 + np.abs(want) + products)
    _, lse, ws, _, _ = _window_run(c, window, sinks)
    off = np.abs(lse.cpu().double().numpy() - want)
    assert (off <= tol).all(), (np.argwhere(off > tol)[:4], (off / tol).max())
    assert mt.read_status(ws) == 0

@pytest.mark.parametrize("t, hq, hkv", [(24, 8, 2), (64, 32, 8)])
def test_a_workspace_without_room_for_depths_serves_the_call_that_has_none(t, hq, hkv):
    # what the call without a window asked for before there was one: all but the last part, the nodes' depths
    c = _attn_case(np.random.default_rng(76), 3, t, hq, hkv, 128, [300, 20, 64], "bf16", "tree")
    want, _, ws, args, kw = _window_run(c, 0, 0)
    room = ws.numel() * ws.element_size() - -(-3 * t * 4 // 256) * 256
    less = torch.zeros(room, dtype=torch.uint8, device="cuda")
    out, kw = torch.full_like(want, 5.0), {k: kw[k] for k in ("k_new", "v_new")}
    mt.tree_attn_paged_block8(*args[:8], out, workspace=less, **kw)
    assert torch.equal(out, want) and mt.read_status(less) == 0
    for more in (dict(workspace=less, window=9), dict(workspace=less, lse=torch.zeros(3, t, hq, device="cuda")), dict(workspace=less[:-256])):
        with pytest.raises(mt.MedusaTreeError):
            mt.tree_attn_paged_block8(*args[:8], out, **kw, **more)


# ---- weights of cached slots ---------------------------------------------------

KERNELS = [(1, 4, 1), (4, 8, 2), (64, 4, 1)]  # T, Hq, Hkv: a few rows a head, and many


@pytest.mark.parametrize("dtype, exponent", [("bf16", 100), ("bf16", 118), ("f16", 15)])
@pytest.mark.parametrize("t, hq, hkv", KERNELS)
def test_slot_weights_of_zero_keys_behind_the_largest_scales(dtype, exponent, t, hq, hkv):
    # queries and page scales whose product is no 32-bit number: a key of zeros has the score 0 all the same
    c = _attn_case(np.random.default_rng(71), 1, t, hq, hkv, 128, [100], dtype, "chain")
    c["q"] = (torch.sign(c["q"].float()) * 2.0 ** exponent).to(c["q"].dtype)
    lse = torch.zeros(1, t, hq, device="cuda")
    w, ws = torch.zeros(c["k"].shape[0], hkv, P, device="cuda"), _status()
    ks = torch.full((c["k"].shape[0], hkv), 2.0 ** 119, device="cuda")
    mt.kv_attn_weights(c["q"].cuda(), torch.zeros_like(_f8(c["k"])), ks, _i32(c["table"]).cuda(), _i32(c["lens"]).cuda(), lse, w, status_ws=ws)
    pages, at = c["table"][0][np.arange(100) // P], np.arange(100) % P
    rows = t * hq // hkv
    assert (w.cpu().numpy()[pages, :, at] == rows).all() and float(w.sum()) == 100 * hkv * rows


@pytest.mark.parametrize("t, hq, hkv", KERNELS)
def test_slot_weights_of_small_queries_behind_large_scales(t, hq, hkv):
    # the other way round: codes and a page's scale whose product is no 32-bit number, and queries so small that the scores
    # are of ordinary size.  Some rows are of ordinary size themselves, with a log-sum-exp beyond all their scores.
    c = _attn_case(np.random.default_rng(72), 2, t, hq, hkv, 128, [100, 37], "bf16", "chain")
    lse = torch.zeros(2, t, hq, device="cuda")
    small = torch.ones(2, t, hq, dtype=torch.bool)
    small[:, ::3, 1::2] = False
    c["q"] = torch.where(small[..., None], c["q"].double() * 2.0 ** -121, c["q"].double()).to(torch.bfloat16)
    lse[~small.cuda()] = 2.0 ** 126
    c["ks"][:] = 2.0 ** 119
    got = _weights_check(c, None, None, 1.0, False, lse=lse)
    assert np.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, hq, hkv", KERNELS + [(40, 16, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dominant, apart", [(8, 0), (8, 6), (12, 3), (12, 6)])
def test_slot_weights_of_queries_with_a_dominant_channel(dtype, t, hq, hkv, d, dominant, apart):
    # one channel of a query is 2^dominant times the others, and the keys have nothing there, so that the scores come from
    # the small ones alone; rows are up to 2^apart apart.  (The tolerance counts 32 bits of what enters a score.)  The new
    # tokens' keys have nothing there either: with them a log-sum-exp of 577 leaves weights of 10^-63, which no 32 bits hold.
    rng = np.random.default_rng(74)
    c = _attn_case(rng, 2, t, hq, hkv, d, [200, 37], dtype, "chain")
    q = c["q"].double()
    q[..., 11] = 2.0 ** dominant * torch.sign(q[..., 11])
    q *= torch.from_numpy(2.0 ** -rng.integers(0, apart + 1, (2, t, hq, 1)))
    c["q"] = q.to(c["q"].dtype)
    c["k"][..., 11] = 0
    c["kn"][..., 11] = 0
    _weights_check(c, [150, 20], None, 0.9, False)


# ---- eviction -------------------------------------------------------------------

def _reencoded(old, new):
    """The code of (value * old / new) for each of the 256 codes, by exact arithmetic: nearest, ties to the even code."""
    out = np.zeros(256, np.uint8)
    f = Fraction(float(old)) / Fraction(float(new))
    values = [Fraction(float(v)) for v in ref.VALUES]
    for code, v in enumerate(values):
        x = v * f
        at = min(bisect.bisect_left(values, x), 126)  # the first value >= x
        if values[at] != x and at > 0:
            lo, hi = x - values[at - 1], values[at] - x
            at -= lo < hi or (lo == hi and at % 2 == 1)
        out[code] = at
    out[0x7F] = 0x7F
    out[128:] = out[:128] | 0x80
    return out


def test_reencoding_of_powers_of_two():
    for k in range(12):
        want = ref.encode(ref.decode(np.arange(256)) * 2.0 ** -k)
        got = _reencoded(1.0, 2.0 ** k)
        nan = np.arange(256) & 0x7F == 0x7F
        assert np.array_equal(got[~nan], want[~nan])


def _borders(rng, shape):
    """Scales of which one in three is the largest, and the others put some code's value on the border of two codes under
    it, or just beside: old / new = m / c with c a code's four bits and m a border's five, up to a power of two."""
    new = 45045 * 16  # every c divides it
    out = np.full(shape, new, np.float32)
    for at in np.ndindex(*shape):
        if at[0] % 3:
            c, m = 8 + int(rng.integers(0, 8)), 17 + 2 * int(rng.integers(0, 8))
            out[at] = new // c * m / 2.0 ** rng.integers(2, 6)
            if at[0] % 3 == 2:
                out[at] = np.nextafter(out[at], np.float32(rng.choice([0, 2e9])))
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["any", "borders", "near 1", "far apart"])
def test_evict_scales_that_are_not_powers_of_two(d, what):
    rng = np.random.default_rng(75)
    e = Evict(rng, "block8", torch.bfloat16, 2, d, [500, 64, 201], 100)
    for x in range(2):
        s = e.cache.host_scales[x]
        if what == "any":
            s[...] = np.exp(2 * rng.standard_normal(s.shape)).astype(np.float32)
        elif what == "near 1":
            s[...] = (np.float32(1) + rng.integers(0, 4, s.shape).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
        elif what == "far apart":
            s[...] = np.float32(1.7) * 2.0 ** rng.integers(-64, 119, s.shape).astype(np.float32)
        else:
            s[...] = _borders(rng, s.shape)
        e.cache.scales[x].copy_(torch.from_numpy(s).float())
        s[...] = e.cache.scales[x].cpu().numpy()
        assert s.max() <= 2.0 ** 119
    e.run(3, 10)
    kept = e.kept.cpu().numpy()
    tables = {}
    for x, cache in enumerate((e.cache.k, e.cache.v)):
        got, src, new_scales = _codes(cache), e.cache.host[x].view(torch.uint8).numpy(), e.cache.scales[x].cpu().numpy()
        for b in range(len(e.lens)):
            for h in range(2):
                stay = kept[b, h][kept[b, h] >= 0]
                for j in range(0, len(stay), P):
                    slots = stay[j:j + P]
                    pages = e.table[b][slots // P]
                    old, to = e.cache.host_scales[x][pages, h].astype(np.float32), e.new[b][j // P]
                    assert new_scales[to, h] == old.max()
                    for r, (slot, page) in enumerate(zip(slots, pages)):
                        key = (float(old[r]), float(old.max()))
                        if key not in tables:
                            tables[key] = _reencoded(*key)
                        row = src[page, h, slot % P]
                        want = row if key[0] == key[1] else tables[key][row]
                        nan = row & 0x7F == 0x7F
                        assert np.array_equal(got[to, h, r][~nan], want[~nan]) and (got[to, h, r][nan] & 0x7F == 0x7F).all()
    assert len(tables) > 20 or what == "near 1"


def test_evict_again_and_again():
    # a scale stays when the row that made it goes: over three evictions a value loses no more than what falls below the
    # smallest code under the largest scale on its way, half of 2^-9 of it each time
    rng = np.random.default_rng(78)
    e = Evict(rng, "block8", torch.bfloat16, 2, 64, [700, 333], 256)
    for x in range(2):
        e.cache.host[x].view(torch.uint8).numpy()[...] &= 0xF7  # no NaN codes
        (e.cache.k, e.cache.v)[x].view(torch.uint8).copy_(e.cache.host[x].view(torch.uint8).cuda())
    value = lambda x, page, h, at: ref.decode(e.cache.host[x].view(torch.uint8).numpy()[page, h, at]) * e.cache.host_scales[x][page, h][..., None]  # noqa: E731
    first, first_lens = e.table.copy(), list(e.lens)
    start = [[[value(x, first[b][np.arange(n) // P], h, np.arange(n) % P) for h in range(2)] for b, n in enumerate(first_lens)] for x in range(2)]
    slots = [[np.arange(n)] * 2 for n in first_lens]  # what is left, by its first slot
    for budget in (256, 100, 33):
        e.budget = budget
        e.run(2, 9)
        e.check(2, 9)
        kept = e.kept.cpu().numpy()
        e.lens = [min(n, budget) for n in e.lens]
        slots = [[slots[b][h][kept[b, h][:n]] for h in range(2)] for b, n in enumerate(e.lens)]
        e.table, e.new = e.new, e.table  # the pages that are free again
    for x in range(2):
        for b, n in enumerate(e.lens):
            for h in range(2):
                at = np.arange(n)
                pages = e.table[b][at // P]
                now, then = value(x, pages, h, at % P), start[x][b][h][slots[b][h]]
                assert (np.abs(now - then) <= 3 * 2.0 ** -10 * e.cache.host_scales[x][pages, h][:, None]).all()
                assert (np.abs(now - then) > 0).any() or x  # (some did fall below)
