"""Host-side checks, without a GPU: a misaligned pointer to a 32-bit array is refused by the call (on the device it would be a
fault)."""
import pytest

pytest.importorskip("torch")

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
