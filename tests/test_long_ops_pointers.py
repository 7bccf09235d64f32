"""Host-side checks, without a GPU: a misaligned pointer to a 32-bit array is refused by the call (on the device it would be a
fault), and a count that is no whole number by the binding."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import medusa_tree_speculative_attn_gb300 as mt
from test_long_ops import _logits_desc
from test_serve_ops import INVALID, _append_desc, _attn_desc, _norm_desc, lib  # noqa: F401 (lib: the fixture)


def _at(n):
    return [(i + 1) << 32 for i in range(n)]  # far apart


def _odd(call, n, which):
    for i in which:
        for shift in (1, 2):
            args = _at(n)
            args[i] += shift
            assert call(*args) == INVALID, (i, shift)


def test_window_attention(lib):  # noqa: F811
    # q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, tables, lens, parents, out, lse, workspace
    _odd(lambda *a: lib.mt_tree_attn_paged_block8_window(_attn_desc(), 8, 4, *a, 1 << 40, None), 13, (5, 6, 7, 8, 9, 11))
    _odd(lambda *a: lib.mt_tree_attn_paged_block8(_attn_desc(), *a, 1 << 40, None), 12, (5, 6, 7, 8, 9))


def test_weights(lib):  # noqa: F811
    # q, lse, k_cache, k_scales, tables, lens, prev, path, path lengths, weights, out, status
    _odd(lambda *a: lib.mt_kv_attn_weights(_attn_desc(), 3, 1.0, *a, None), 12, (1, 3, 4, 5, 6, 7, 8))


def test_evict(lib):  # noqa: F811
    # k_cache, v_cache, k_scales, v_scales, weights, tables, lens, new tables, kept, status
    _odd(lambda *a: lib.mt_kv_evict(_attn_desc(), 2, 20, 2, 4, *a, None), 10, (2, 3, 5, 6, 7, 8))


def test_logits(lib):  # noqa: F811
    # logits, out, history, lens, starts, rep, pres, freq, bias tokens, bias values, mask, index, tokens, parents, status
    _odd(lambda *a: lib.mt_process_logits(_logits_desc(), *a, None), 15, range(2, 14))


def test_append(lib):  # noqa: F811
    # k, v, row offsets, (rope), k_cache, v_cache, k_scales, v_scales, tables, lens, status
    _odd(lambda k, v, o, *a: lib.mt_kv_append_paged(_append_desc(), k, v, o, None, *a, None), 10, (2, 5, 6, 7, 8))
    # k, v, path, path lengths, (rope), ...
    d = _append_desc(batch=2, num_rows=10)
    _odd(lambda k, v, p, n, *a: lib.mt_kv_append_accepted(d, 5, 2, k, v, p, n, None, *a, None), 11, (2, 3, 6, 7, 8, 9))


def test_norm_positions(lib):  # noqa: F811
    # q, k, positions, weights, (rope), q_out, k_out, status
    _odd(lambda q, k, p, qw, kw, *a: lib.mt_qk_norm_rope(_norm_desc(), q, k, p, qw, kw, None, *a, None), 8, (2,))


def test_sampling(lib):  # noqa: F811
    # logits, row index, uniforms, temperature, top_k, top_p, min_p, tokens
    _odd(lambda x, i, *a: lib.mt_sample_tokens(4, 10, 2, x, 4, 10, i, *a, None), 8, range(1, 8))


def test_counts_of_the_binding():
    for good in (0, 7, 2 ** 31 - 1, np.int32(5), True):
        assert mt._int32(good, "n") == int(good) and type(mt._int32(good, "n")) is int
    for bad in (2.5, 2.0, "3", None, np.float32(1)):
        with pytest.raises(TypeError, match="window must be an integer"):
            mt._int32(bad, "window")
    for bad in (-1, 2 ** 31, 2 ** 40):
        with pytest.raises(ValueError, match="window must be in"):
            mt._int32(bad, "window")


@pytest.mark.gpu
def test_counts_of_the_calls():
    cu = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, n, cache, table = cu(3, 4, 8, 128), cu(3, 4, 2, 128), cu(6, 2, 16, 128, dtype=torch.float8_e4m3fn), cu(3, 2, dtype=torch.int32)
    scales, ws, lens, out = cu(6, 2, dtype=torch.float32) + 1, mt.alloc_block8_workspace(q, cache, table), cu(3, dtype=torch.int32), torch.empty_like(q)
    for kw in (dict(window=2.5), dict(window=5, sinks=1.5), dict(window=5.0), dict(sinks=-1), dict(window="5")):
        with pytest.raises((TypeError, ValueError)):
            mt.tree_attn_paged_block8(q, cache, cache, scales, scales, table, lens, None, out, k_new=n, v_new=n, workspace=ws, **kw)
    kept, weights = cu(3, 2, 20, dtype=torch.int32), cu(6, 2, 16, dtype=torch.float32)
    for kw in (dict(sinks=1.5), dict(recent=2.0)):
        with pytest.raises(TypeError):
            mt.kv_evict(cache, cache, weights, table, lens, table, kept, status_ws=ws, **kw)
