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
