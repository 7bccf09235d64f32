"""The plain implementations that the operators for long sequences are held to, pinned on the CPU by other ways to the
same numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import long_reference as lref
import serve_reference as ref

P = 16


@pytest.mark.parametrize("n, window, sinks", [(0, 3, 0), (5, 1, 0), (5, 3, 1), (9, 4, 20), (9, 100, 2), (7, 0, 3)])
def test_a_chain_sees_a_band_and_the_first_columns(n, window, sinks):
    t = 6
    got = lref.sees(n, t, None, window, sinks)
    place = np.arange(n + t)
    row = n + np.arange(t)[:, None]
    want = (place <= row) & ((place > row - window) | (place < sinks) | (window == 0))
    assert np.array_equal(got, want)


def test_siblings_do_not_see_one_another_and_share_a_position():
    got = lref.sees(4, 4, [-1, 0, 0, 2], 2, 1)  # nodes 1 and 2 at position 5, node 3 at 6
    assert got[:, 0].all()  # the sink
    assert got[0, 3] and not got[1:, 1:4].any()  # position 3 is in the root's window alone
    assert got[:, 4:].astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [0, 0, 1, 1]]


def test_attention_without_a_window_is_the_attention_and_weights_are_shares_of_one():
    rng = np.random.default_rng(0)
    n, t, hq, hkv, d = 21, 3, 4, 2, 64
    c = dict(q=torch.from_numpy(rng.standard_normal((1, t, hq, d))), kn=torch.from_numpy(rng.standard_normal((1, t, hkv, d))), vn=torch.from_numpy(rng.standard_normal((1, t, hkv, d))),
             k=rng.integers(0, 120, (3, hkv, P, d)).astype(np.uint8), v=rng.integers(0, 120, (3, hkv, P, d)).astype(np.uint8), ks=np.full((3, hkv), 2.0 ** -6),
             vs=np.full((3, hkv), 0.5), table=np.array([[2, 0]]), lens=[n], parents=None)
    out, mag, lse = lref.window_attn64(c, 0, 0, 0.1)
    want, wmag = ref.attn64(*(c[x].numpy() if x == "q" else c[x] for x in ("q", "k", "v", "ks", "vs", "table", "lens", "parents")), c["kn"].numpy(), c["vn"].numpy(), 0.1)
    assert np.allclose(out, want, rtol=1e-12) and np.allclose(mag, wmag, rtol=1e-12)
    w, tol = lref.weights64(c, np.zeros((3, hkv, P), np.float32), lse, [n], [0], lambda b: range(t), 1.0, 0.1)
    slots = np.concatenate([w[2].T, w[0].T])[:n]  # [n][Hkv]
    for h in range(hkv):  # what is left of each row's share is its own tokens'
        rest = 0.0
        for j in range(2 * h, 2 * h + 2):
            for i in range(t):
                codes, s = ref.block_codes(c["kn"].numpy()[0, :, h])
                z = (ref.decode(codes) * s)[:i + 1] @ c["q"].numpy()[0, i, j] * 0.1
                rest += np.exp(z - lse[0, i, j]).sum()
        assert abs(slots[:, h].sum() + rest - 2 * t) < 1e-9
    assert (w[1] == 0).all() and (w[0][:, n - P:] == 0).all() and (tol >= 0).all()


def test_kept_slots_by_counting():
    rng = np.random.default_rng(1)
    for _ in range(200):
        n, budget = int(rng.integers(1, 40)), int(rng.integers(1, 30))
        sinks = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - sinks + 1))
        w = rng.choice(np.array([np.nan, -np.inf, -1, 0, -0.0, 1, 2, np.inf], np.float32), n)
        kept = lref.kept_slots(w, budget, sinks, recent)
        assert len(kept) == min(n, budget) and (np.diff(kept) > 0).all()
        if n <= budget:
            continue
        protected = set(range(sinks)) | set(range(n - recent, n))
        assert protected <= set(kept)
        key = lambda s: -2e308 if np.isnan(w[s]) else max(float(w[s]), -1e300)  # noqa: E731
        for a in set(range(n)) - set(kept):  # nothing left out beats what stayed
            for b in set(kept) - protected:
                assert key(b) > key(a) or (key(b) == key(a) and b < a), (w, a, b)


def test_logits_of_one_row_by_hand():
    x = np.array([[[2.0, -2.0, 1.0, 0.0, 5.0]]])
    out, _, touched = lref.logits64(x, np.array([[0, 1, 0, 9]]), [3], [1], [2.0], [0.5], [0.25], (np.array([[3, 3, -1]]), np.array([[1.0, 4.0, 9.0]])), np.array([[1, 1, 1, 1, 0]], bool),
                                    np.array([[0]]), [[2]], None)
    # token 0: seen, generated once; 1: seen, generated once; 2: the node's own; 3: the last bias; 4: masked
    assert out[0, 0].tolist() == [2 / 2 - 0.25 - 0.5, -4 - 0.25 - 0.5, 0.5 - 0.25 - 0.5, 4.0, -np.inf] and touched.all()
