"""Places of the operators for long sequences where a result could go wrong without a size or a mask being odd: what one
lane leaves for another, extreme scales, queries with a dominant channel, scales that are not powers of two.  Against the
plain implementations in 64 bits (long_reference)."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import long_reference as lref
import medusa_tree_speculative_attn_gb300 as mt
import serve_reference as ref
from test_gpu_long import _f8, _hide, _lse_of, _weights_check, _window_check, _window_run
from test_gpu_serve import P, _attn_case, _i32, _status

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
