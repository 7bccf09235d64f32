"""The plain implementations that the serving operators are held to, pinned on the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serve_reference as ref


def test_codes_are_the_e4m3_values():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = ref.decode(codes)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.array_equal(got[fine], want[fine])
    assert np.array_equal(ref.encode(got[fine]), codes[fine])


def test_encoding_rounds_to_the_nearest_even_code_and_saturates():
    x = np.random.default_rng(0).normal(size=20000) * np.exp2(np.random.default_rng(1).uniform(-14, 9, 20000))
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(np.float64(np.float32(x))), want)
    v = ref.VALUES
    mid = (v[:-1] + v[1:]) / 2
    assert np.array_equal(ref.encode(mid) % 2, np.zeros(len(mid), np.uint8))
    assert list(ref.encode([1e9, -np.inf, 448.0, 0.0])) == [126, 254, 126, 0]


@pytest.mark.parametrize("amax, k", [(0.0, -64), (448.0, 0), (448.1, 1), (447.0, 0), (224.0, -1), (1e-30, -64),
                                     (3e38, 119), (np.inf, 119), (7.0, -6)])
def test_block_scales(amax, k):
    assert ref.scale_of(amax) == 2.0 ** k


def test_sampling_reference_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))   # masses 1, 4, 2, 1 of 8
    pick = lambda u, **kw: ref.sample64(x, u, **{**dict(t=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw})  # noqa: E731
    assert [pick(u) for u in (0.0, 0.12, 0.13, 0.62, 0.63, 0.87, 0.88, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [pick(u, top_k=2) for u in (0.0, 0.66, 0.67)] == [1, 1, 2]
    assert [pick(u, top_k=3) for u in (0.1, 0.2)] == [0, 1]     # ties: the lower index stays
    assert [pick(u, top_p=0.5) for u in (0.0, 0.99)] == [1, 1]  # 4 of 8 reach it
    assert [pick(u, top_p=0.51) for u in (0.66, 0.67)] == [1, 2]
    assert [pick(u, min_p=0.3) for u in (0.66, 0.67)] == [1, 2]
    assert pick(0.9, t=0.0) == 1


def test_ancestors_of_a_small_tree():
    m = ref.ancestors([-1, 0, 0, 1], 4)
    assert m.astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert np.array_equal(ref.ancestors(None, 3), np.tril(np.ones((3, 3), bool)))
