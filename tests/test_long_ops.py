"""Host-side checks of the operators for long sequences and shaped answers, without a GPU: the C ABI refuses bad
descriptors and pointers before it touches the device, and the binding refuses arguments that do not fit."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import medusa_tree_speculative_attn_gb300 as mt
from test_serve_ops import INVALID, ODD, OK, PTR, UNSUPPORTED, _attn_desc, lib  # noqa: F401 (lib: the fixture)


# ---- attention under a window ----

@pytest.mark.parametrize("window, sinks, desc, want", [
    (-1, 0, {}, INVALID), (8, -1, {}, INVALID), (8, 4, dict(tree_size=65), UNSUPPORTED), (8, 4, dict(dtype=0), UNSUPPORTED), (0, 0, dict(batch=0), INVALID),
])
def test_window_sizes(lib, window, sinks, desc, want):  # noqa: F811
    assert lib.mt_tree_attn_paged_block8_window(_attn_desc(**desc), window, sinks, *[PTR] * 13, 1 << 40, None) == want


def test_window_pointers(lib):  # noqa: F811
    at = [(i + 1) << 32 for i in range(13)]  # q, k_new, v_new, ... far apart; tree_parents 9, out 10, lse 11, workspace 12
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 12):
        args = list(at)
        args[i] = None
        assert lib.mt_tree_attn_paged_block8_window(_attn_desc(), 8, 4, *args, 1 << 40, None) == INVALID, i
    for i in (0, 1, 2, 3, 4, 10, 11, 12):
        args = list(at)
        args[i] += 2
        assert lib.mt_tree_attn_paged_block8_window(_attn_desc(), 8, 4, *args, 1 << 40, None) == INVALID, i
    size = 4 * 2 * 4 * 8  # lse, just before and just behind what it must not overlap
    for i, n in ((0, 2 * 2 * 4 * 8 * 128), (1, 2 * 2 * 4 * 2 * 128), (2, 2 * 2 * 4 * 2 * 128), (10, 2 * 2 * 4 * 8 * 128)):
        for shift in (0, 4 - size, n - 4):
            args = list(at)
            args[11] = args[i] + shift
            assert lib.mt_tree_attn_paged_block8_window(_attn_desc(), 8, 4, *args, 1 << 40, None) == INVALID, (i, shift)
    assert lib.mt_tree_attn_paged_block8_window(None, 8, 4, *at, 1 << 40, None) == INVALID


@pytest.mark.gpu
def test_the_binding_refuses_windows_that_do_not_fit():
    cu = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, n, cache, table = cu(3, 4, 8, 128), cu(3, 4, 2, 128), cu(6, 2, 16, 128, dtype=torch.float8_e4m3fn), cu(3, 2, dtype=torch.int32)
    scales, ws, lse = cu(6, 2, dtype=torch.float32) + 1, mt.alloc_block8_workspace(q, cache, table), cu(3, 4, 8, dtype=torch.float32)
    call = lambda **kw: mt.tree_attn_paged_block8(**{**dict(q=q, k_cache=cache, v_cache=cache, k_scales=scales, v_scales=scales, block_tables=table,  # noqa: E731
                                                            seq_lens=cu(3, dtype=torch.int32), tree_parents=None, out=torch.empty_like(q), k_new=n, v_new=n, workspace=ws,
                                                            window=5, sinks=2, lse=lse), **kw})
    call()
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=2 ** 31), dict(sinks=2 ** 32 + 1), dict(lse=lse[:2]), dict(lse=lse.half()), dict(lse=lse.cpu()),
               dict(lse=lse.transpose(0, 1)), dict(window=0, sinks=-1)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(mt.MedusaTreeError):
        call(workspace=ws[:512])
    torch.cuda.synchronize()


# ---- weights of cached slots ----

@pytest.mark.parametrize("depth, decay, desc, want", [
    (-1, 1.0, {}, INVALID), (64, 1.0, {}, INVALID), (3, -0.5, {}, INVALID), (3, float("inf"), {}, INVALID), (3, float("nan"), {}, INVALID),
    (3, 1.0, dict(head_dim=96), UNSUPPORTED), (3, 1.0, dict(dtype=0), UNSUPPORTED), (3, 1.0, dict(cache_dtype=0), UNSUPPORTED), (3, 1.0, dict(batch=0), INVALID),
    (3, 1.0, dict(num_q_heads=7), INVALID), (3, 1.0, dict(sm_scale=-1.0), INVALID),
])
def test_weights_sizes(lib, depth, decay, desc, want):  # noqa: F811
    assert lib.mt_kv_attn_weights(_attn_desc(**desc), depth, decay, *[PTR] * 12, None) == want


def test_weights_pointers(lib):  # noqa: F811
    # q, lse, k_cache, k_scales, tables, lens, prev (may be null), path, path lengths (both or none), weights, out, status
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10, 11):
        args = [PTR] * 12
        args[i] = None
        assert lib.mt_kv_attn_weights(_attn_desc(), 3, 1.0, *args, None) == INVALID, i
    for i in (0, 1, 2, 9, 10, 11):
        args = [PTR] * 12
        args[i] = ODD
        assert lib.mt_kv_attn_weights(_attn_desc(), 3, 1.0, *args, None) == INVALID, i
    args = [PTR] * 12
    args[10] = PTR + 16  # out over a part of weights
    assert lib.mt_kv_attn_weights(_attn_desc(), 3, 1.0, *args, None) == INVALID
    assert lib.mt_kv_attn_weights(None, 3, 1.0, *[PTR] * 12, None) == INVALID


@pytest.mark.gpu
def test_the_binding_refuses_weights_that_do_not_fit():
    cu = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, cache, table = cu(3, 4, 8, 128, dtype=torch.bfloat16), cu(6, 2, 16, 128, dtype=torch.float8_e4m3fn), cu(3, 2, dtype=torch.int32)
    i32 = lambda *s: cu(*s, dtype=torch.int32)  # noqa: E731
    call = lambda **kw: mt.kv_attn_weights(**{**dict(q=q, k_cache=cache, k_scales=cu(6, 2), block_tables=table, seq_lens=i32(3), lse=cu(3, 4, 8), weights=cu(6, 2, 16),  # noqa: E731
                                                     status_ws=cu(64)), **kw})
    call()
    call(accept_path=i32(3, 2), accept_len=i32(3), prev_lens=i32(3), out=cu(6, 2, 16))
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()), dict(k_cache=q), dict(k_scales=cu(6, 3)), dict(block_tables=i32(3)), dict(seq_lens=i32(2)), dict(lse=cu(3, 4, 7)),
               dict(weights=cu(6, 2, 8)), dict(weights=cu(6, 16, 2).transpose(1, 2)), dict(out=cu(5, 2, 16)), dict(prev_lens=i32(4)), dict(accept_path=i32(3, 2)),
               dict(accept_path=i32(2, 2), accept_len=i32(3)), dict(accept_path=i32(3), accept_len=i32(3)), dict(status_ws=cu(8)), dict(weights=None)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(decay=-1.0), dict(sm_scale=-1.0), dict(accept_path=i32(3, 65), accept_len=i32(3))):
        with pytest.raises(mt.MedusaTreeError):
            call(**kw)
    torch.cuda.synchronize()


# ---- eviction ----

def _evict(lib, args, blocks=2, budget=20, sinks=2, recent=4, **desc):  # noqa: F811
    return lib.mt_kv_evict(_attn_desc(**desc), blocks, budget, sinks, recent, *args, None)


@pytest.mark.parametrize("kw, want", [
    (dict(budget=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(sinks=10, recent=11), INVALID), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID),
    (dict(blocks=1), INVALID), (dict(blocks=0), INVALID), (dict(batch=0), INVALID), (dict(batch=8193), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(page_size=32), UNSUPPORTED), (dict(max_blocks_per_seq=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 27), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(cache_dtype=2), UNSUPPORTED), (dict(cache_dtype=0), INVALID), (dict(max_blocks_per_seq=1 << 27), UNSUPPORTED),
])
def test_evict_sizes(lib, kw, want):  # noqa: F811
    assert _evict(lib, [PTR] * 10, **kw) == want


def test_evict_pointers(lib):  # noqa: F811
    # k_cache, v_cache, k_scales, v_scales (both or none), weights, tables, lens, new tables, kept, status
    for i in range(10):
        args = [PTR] * 10
        args[i] = None
        assert _evict(lib, args) == INVALID, i
    for i in (0, 1, 4, 8, 9):
        args = [PTR] * 10
        args[i] = ODD
        assert _evict(lib, args) == INVALID, i
    assert lib.mt_kv_evict(None, 2, 20, 2, 4, *[PTR] * 10, None) == INVALID


@pytest.mark.gpu
def test_the_binding_refuses_evictions_that_do_not_fit():
    cu = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: cu(*s, dtype=torch.int32)  # noqa: E731
    f8 = lambda *s: cu(*s, dtype=torch.float8_e4m3fn)  # noqa: E731
    call = lambda **kw: mt.kv_evict(**{**dict(k_cache=f8(6, 2, 16, 64), v_cache=f8(6, 2, 16, 64), weights=cu(6, 2, 16), block_tables=i32(3, 2), seq_lens=i32(3) - 1,  # noqa: E731
                                              new_tables=i32(3, 2), kept=i32(3, 2, 20), sinks=2, recent=4, k_scales=cu(6, 2), v_scales=cu(6, 2), status_ws=cu(64)), **kw})
    call()
    call(k_scales=None, v_scales=None)
    for kw in (dict(k_scales=None), dict(k_cache=cu(6, 2, 16, 64), v_cache=cu(6, 2, 16, 64)), dict(v_cache=f8(6, 2, 16, 128)), dict(weights=cu(6, 2, 17)), dict(weights=cu(6, 2, 16).half()),
               dict(block_tables=i32(2, 2)), dict(new_tables=i32(6)), dict(seq_lens=i32(3, 1)), dict(kept=i32(3, 3, 20)), dict(kept=i32(3, 2, 20).long()), dict(sinks=-1), dict(recent=2 ** 31),
               dict(k_cache=torch.zeros(6, 2, 16, 64)), dict(status_ws=cu(8)), dict(k_cache=f8(6, 16, 2, 64).transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(sinks=17), dict(kept=i32(3, 2, 33)), dict(kept=i32(3, 2, 0))):
        with pytest.raises(mt.MedusaTreeError):
            call(**kw)
    torch.cuda.synchronize()


# ---- logits ----

def _logits_desc(**kw):
    base = dict(batch=2, tree_size=4, vocab=100, dtype=2, history_width=8, num_bias=3, num_masks=2, stride=(400, 100), out_stride=(400, 100))
    return ctypes.byref(mt.LogitsDesc(**{**base, **kw}))


@pytest.mark.parametrize("desc, want", [
    (dict(batch=-1), INVALID), (dict(tree_size=-1), INVALID), (dict(vocab=0), INVALID), (dict(vocab=(1 << 30) + 1), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(history_width=-1), INVALID), (dict(history_width=1 << 30), INVALID), (dict(num_bias=-1), INVALID), (dict(num_masks=-1), INVALID), (dict(stride=(-400, 100)), INVALID),
    (dict(out_stride=(400, 99)), INVALID), (dict(out_stride=(399, 100)), INVALID), (dict(out_stride=(0, 100)), INVALID), (dict(out_stride=(150, 200)), INVALID),
    (dict(tree_size=65, stride=(6500, 100), out_stride=(6500, 100)), UNSUPPORTED), (dict(batch=1 << 24), INVALID), (dict(batch=0), OK), (dict(tree_size=0), OK),
    (dict(stride=(1 << 39, 100)), INVALID), (dict(out_stride=(400, 1 << 40)), INVALID), (dict(stride=(800, 100)), INVALID),  # the same place under other strides
])
def test_logits_sizes(lib, desc, want):  # noqa: F811
    assert lib.mt_process_logits(_logits_desc(**desc), *[PTR] * 15, None) == want


def test_logits_pointers(lib):  # noqa: F811
    names = "logits out history lens starts rep pres freq bias_tokens bias_values mask index tokens parents status".split()
    at = {n: (i + 1) << 32 for i, n in enumerate(names)}
    call = lambda **kw: lib.mt_process_logits(_logits_desc(), *{**at, **kw}.values(), None)  # noqa: E731
    for kw in (dict(logits=None), dict(out=None), dict(status=None), dict(logits=PTR + 1), dict(out=PTR + 1), dict(status=ODD), dict(history=None), dict(lens=None, starts=None),
               dict(history=None, lens=None), dict(bias_tokens=None), dict(bias_values=None), dict(mask=None), dict(index=None), dict(tokens=None)):
        assert call(**kw) == INVALID, kw
    for shift in (2, 1598, -2, -1598):  # out over a part of the logits
        assert call(out=at["logits"] + shift) == INVALID
    assert lib.mt_process_logits(None, *at.values(), None) == INVALID


@pytest.mark.gpu
def test_the_binding_refuses_logits_that_do_not_fit():
    cu = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: cu(*s, dtype=torch.int32)  # noqa: E731
    x = cu(2, 3, 50)
    call = lambda **kw: mt.process_logits(**{**dict(logits=x, out=cu(2, 3, 50), history=i32(2, 9), history_lens=i32(2), output_starts=i32(2), repetition=cu(2) + 1,  # noqa: E731
                                                    presence=cu(2), frequency=cu(2), bias_tokens=i32(2, 4), bias_values=cu(2, 4), mask=i32(5, 2), mask_index=i32(2, 3),
                                                    tree_tokens=i32(2, 3), tree_parents=i32(2, 3) - 1, status_ws=cu(64)), **kw})
    call()
    for kw in (dict(logits=x.double()), dict(logits=x[0, 0]), dict(logits=x.cpu()), dict(out=x[:1]), dict(out=x.half()), dict(out=None), dict(out=cu(2, 50, 3).transpose(1, 2)),
               dict(history=i32(2)), dict(history=None), dict(history_lens=None), dict(history_lens=i32(3)), dict(output_starts=cu(2)), dict(repetition=cu(3)), dict(presence=cu(2).double()),
               dict(frequency=[0.0, 0.0]), dict(bias_tokens=i32(2, 3)), dict(bias_values=None), dict(mask=i32(5, 1)), dict(mask=i32(10)), dict(mask_index=i32(6)), dict(tree_tokens=i32(2, 4)),
               dict(tree_parents=i32(2, 2)), dict(status_ws=cu(8))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(out=cu(1, 3, 50).expand(2, 3, 50)), dict(mask=None), dict(mask_index=None), dict(tree_tokens=None), dict(history=None, history_lens=None)):
        with pytest.raises(mt.MedusaTreeError):
            call(**kw)
    torch.cuda.synchronize()
