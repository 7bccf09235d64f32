"""Host-side checks of the serving operators, without a GPU: the C ABI refuses bad descriptors and pointers before
it touches the device, and the binding refuses arguments that do not fit one another."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import medusa_tree_speculative_attn_gb300 as mt

OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def lib():
    from medusa_tree_speculative_attn_gb300 import build
    build.build()
    return mt.library()


BUF = (ctypes.c_char * 4096)()
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256  # an aligned host address: refused calls never look at it
ODD = PTR + 2


def _norm_desc(**kw):
    base = dict(num_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=2, eps=1e-6, q_stride=(1024, 128),
                k_stride=(256, 128), q_out_stride=(1024, 128), k_out_stride=(256, 128))
    return ctypes.byref(mt.NormRopeDesc(**{**base, **kw}))


@pytest.mark.parametrize("desc, want", [
    (dict(num_tokens=-1), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(eps=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(q_stride=(1024, 132)), INVALID), (dict(k_stride=(-256, 128)), INVALID), (dict(q_out_stride=(1028, 128)), INVALID),
    (dict(k_out_stride=(256, 4)), INVALID), (dict(num_tokens=0), OK),
])
def test_norm_rope_descriptors(lib, desc, want):
    assert lib.mt_qk_norm_rope(_norm_desc(**desc), PTR, PTR, PTR, PTR, PTR, None, PTR, PTR, PTR, None) == want


@pytest.mark.parametrize("args", [
    (None, PTR, PTR, PTR, PTR, None, PTR, PTR, PTR), (PTR, None, PTR, PTR, PTR, None, PTR, PTR, PTR), (PTR, PTR, PTR, PTR, None, None, PTR, PTR, PTR),
    (PTR, PTR, PTR, None, None, None, PTR, PTR, PTR), (PTR, PTR, PTR, PTR, PTR, None, None, PTR, PTR), (PTR, PTR, PTR, PTR, PTR, None, PTR, PTR, None),
    (ODD, PTR, PTR, PTR, PTR, None, PTR, PTR, PTR), (PTR, PTR, PTR, ODD, PTR, None, PTR, PTR, PTR), (PTR, PTR, PTR, PTR, PTR, None, PTR, ODD, PTR),
])
def test_norm_rope_pointers(lib, args):
    assert lib.mt_qk_norm_rope(_norm_desc(), *args, None) == INVALID
    assert lib.mt_qk_norm_rope(None, *args, None) == INVALID


def _append_desc(**kw):
    base = dict(batch=2, num_rows=10, num_kv_heads=2, head_dim=64, page_size=16, max_blocks_per_seq=4, num_pages=9, dtype=2, cache_dtype=3,
                k_scale=1.0, v_scale=1.0, k_stride=(128, 64), v_stride=(128, 64))
    return ctypes.byref(mt.AppendDesc(**{**base, **kw}))


@pytest.mark.parametrize("desc, want", [
    (dict(batch=0), INVALID), (dict(batch=8193), INVALID), (dict(num_rows=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=80), UNSUPPORTED),
    (dict(page_size=32), UNSUPPORTED), (dict(max_blocks_per_seq=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 27), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(cache_dtype=2), UNSUPPORTED), (dict(cache_dtype=0), INVALID),
    (dict(k_stride=(128, 60)), INVALID), (dict(v_stride=(-128, 64)), INVALID), (dict(num_rows=0), OK),
])
def test_append_descriptors(lib, desc, want):
    d = _append_desc(**desc)
    assert lib.mt_kv_append_paged(d, PTR, PTR, PTR, None, PTR, PTR, PTR, PTR, PTR, PTR, PTR, None) == want


def test_append_scales_and_pointers(lib):
    good = [PTR, PTR, PTR, None, PTR, PTR, PTR, PTR, PTR, PTR, PTR]
    for i in (0, 1, 2, 4, 5, 6, 7, 8, 9, 10):
        bad = list(good)
        bad[i] = None
        assert lib.mt_kv_append_paged(_append_desc(), *bad, None) == INVALID, i
    for i in (0, 1, 4, 5, 10):
        bad = list(good)
        bad[i] = ODD
        assert lib.mt_kv_append_paged(_append_desc(), *bad, None) == INVALID, i
    one = good[:6] + [None, None] + good[8:]
    for scales in (dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("inf")), dict(v_scale=float("nan"))):
        assert lib.mt_kv_append_paged(_append_desc(**scales), *one, None) == INVALID
    assert lib.mt_kv_append_paged(None, *good, None) == INVALID


@pytest.mark.parametrize("t, depth, rows, want", [(0, 1, 0, UNSUPPORTED), (65, 1, 130, UNSUPPORTED), (5, -1, 10, INVALID), (5, 64, 10, INVALID), (5, 2, 9, INVALID)])
def test_append_accepted_sizes(lib, t, depth, rows, want):
    d = _append_desc(num_rows=rows)
    assert lib.mt_kv_append_accepted(d, t, depth, PTR, PTR, PTR, PTR, None, PTR, PTR, PTR, PTR, PTR, PTR, PTR, None) == want


def _attn_desc(**kw):
    base = dict(batch=2, tree_size=4, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, max_blocks_per_seq=8, num_pages=32, num_splits=0, dtype=2,
                sm_scale=0.0, kernel=0, cache_dtype=3, k_scale=1.0, v_scale=1.0)
    return ctypes.byref(mt.AttnDesc(**{**base, **kw}))


@pytest.mark.parametrize("desc, want", [
    (dict(batch=0), INVALID), (dict(batch=8193), INVALID), (dict(tree_size=0), UNSUPPORTED), (dict(tree_size=65), UNSUPPORTED), (dict(num_q_heads=7), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=64), UNSUPPORTED), (dict(max_blocks_per_seq=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 26), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(cache_dtype=0), UNSUPPORTED),
    (dict(sm_scale=-1.0), INVALID), (dict(sm_scale=float("inf")), INVALID), (dict(sm_scale=float("nan")), INVALID),
])
def test_attention_descriptors(lib, desc, want):
    d = _attn_desc(**desc)
    assert lib.mt_tree_attn_paged_block8(d, *[PTR] * 12, 1 << 40, None) == want
    assert lib.mt_tree_attn_block8_workspace_size(d) == 0


def test_attention_pointers(lib):
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11):  # tree_parents (9) may be null
        args = [PTR] * 12
        args[i] = None
        assert lib.mt_tree_attn_paged_block8(_attn_desc(), *args, 1 << 40, None) == INVALID, i
    for i in (0, 1, 2, 3, 4, 10, 11):
        args = [PTR] * 12
        args[i] = ODD
        assert lib.mt_tree_attn_paged_block8(_attn_desc(), *args, 1 << 40, None) == INVALID, i
    assert lib.mt_tree_attn_paged_block8(None, *[PTR] * 12, 1 << 40, None) == INVALID


def test_attention_output_over_its_inputs(lib):
    at = [(i + 1) << 32 for i in range(12)]  # q, k_new, v_new, ... far apart
    d = _attn_desc()
    size = 2 * 2 * 4 * 8 * 128
    for i in (0, 1, 2):
        for shift in (0, 16, 16 - size):  # the same, just behind, just before
            args = list(at)
            args[10] = args[i] + shift
            assert lib.mt_tree_attn_paged_block8(d, *args, 1 << 40, None) == INVALID, (i, shift)


@pytest.mark.parametrize("n, v, dt, rows, index, stride, want", [
    (-1, 10, 2, 4, PTR, 10, INVALID), (4, 0, 2, 4, PTR, 10, INVALID), (4, 500001, 2, 4, PTR, 10, UNSUPPORTED), (4, 10, 3, 4, PTR, 10, UNSUPPORTED),
    (4, 10, 2, 5, None, 10, INVALID), (4, 10, 2, -1, PTR, 10, INVALID), (4, 10, 2, 4, None, -10, INVALID), (0, 10, 2, 0, None, 10, OK), (0, 10, 2, 7, PTR, 10, OK),
])
def test_sampling_sizes(lib, n, v, dt, rows, index, stride, want):
    assert lib.mt_sample_tokens(n, v, dt, PTR, rows, stride, index, PTR, PTR, PTR, PTR, PTR, PTR, None) == want


def test_sampling_pointers(lib):
    good = [PTR, 4, 10, None, PTR, None, None, None, None, PTR]
    for i in (0, 4, 9):
        bad = list(good)
        bad[i] = None
        assert lib.mt_sample_tokens(4, 10, 2, *bad, None) == INVALID
    assert lib.mt_sample_tokens(4, 10, 2, PTR + 1, *good[1:], None) == INVALID


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    ws, i32 = torch.zeros(256, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(4, 4, 16, 64, dtype=torch.float8_e4m3fn)
    scales = torch.ones(4, 4)
    table = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mt.qk_norm_rope(x, x, None, x, x, q_weight=x[0, 0], k_weight=x[0, 0], status_ws=ws)
    with pytest.raises(ValueError, match="CUDA"):
        mt.kv_append_paged(x, x, cache, cache, table, i32[:2], i32, status_ws=ws, k_scales=scales, v_scales=scales)
    y = x.view(2, 1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mt.kv_append_accepted(y, y, table, i32[:2], cache, cache, table, i32[:2], status_ws=ws)
    with pytest.raises(ValueError, match="CUDA"):
        mt.tree_attn_paged_block8(y, cache, cache, scales, scales, table, i32[:2], None, y, k_new=y, v_new=y, workspace=ws)
    with pytest.raises(ValueError, match="CUDA"):
        mt.alloc_block8_workspace(y, cache, table)
    with pytest.raises(ValueError, match="CUDA"):
        mt.sample_tokens(torch.zeros(2, 5), torch.zeros(2), i32[:2])


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_fit():
    cu = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: cu(*s, dtype=torch.int32)  # noqa: E731
    q, k, ws = cu(5, 8, 128), cu(5, 2, 128), cu(256, dtype=torch.uint8)
    w = cu(128)
    bad = pytest.raises((ValueError, TypeError))
    norm = lambda **kw: mt.qk_norm_rope(**{**dict(q=q, k=k, positions=i32(5), q_out=q, k_out=k, q_weight=w, k_weight=w, status_ws=ws), **kw})  # noqa: E731
    norm()
    for kw in (dict(k=cu(4, 2, 128)), dict(k=cu(5, 2, 64)), dict(k=cu(5, 2, 128, dtype=torch.float16)), dict(q_out=cu(5, 8, 64)), dict(k_out=cu(1, 2, 128).expand(5, 2, 128)),
               dict(positions=cu(5)), dict(positions=i32(4)), dict(q_weight=None), dict(q_weight=cu(64)), dict(q_weight=None, k_weight=None),
               dict(status_ws=cu(255, dtype=torch.uint8)), dict(q=q.transpose(0, 1)), dict(q=cu(5, 8, 129)[..., 1:]), dict(q=q.float()), dict(q=q.cpu()),
               dict(rope=mt.Rope(1e4, 128, 8), positions=None), dict(status_ws=None)):
        with bad:
            norm(**kw)
    with pytest.raises(mt.MedusaTreeError):
        norm(rope=mt.Rope(1e4, 64, 8))
    with pytest.raises(mt.MedusaTreeError):
        mt.qk_norm_rope(cu(5, 8, 96), cu(5, 2, 96), None, cu(5, 8, 96), cu(5, 2, 96), q_weight=cu(96), k_weight=cu(96), status_ws=ws)

    cache, scales, table = cu(6, 2, 16, 128, dtype=torch.float8_e4m3fn), cu(6, 2, dtype=torch.float32), i32(3, 2)
    app = lambda **kw: mt.kv_append_paged(**{**dict(k=k, v=k, k_cache=cache, v_cache=cache.clone(), block_tables=table, seq_lens=i32(3), row_offsets=i32(4),  # noqa: E731
                                                    status_ws=ws, k_scales=scales, v_scales=scales.clone()), **kw})
    app()
    for kw in (dict(k=cu(5, 3, 128)), dict(v=cu(4, 2, 128)), dict(v=k.float()), dict(k_cache=cu(6, 2, 16, 128, dtype=torch.float16)), dict(v_cache=cache[:5]), dict(k_scales=None),
               dict(k_scales=cu(6, 3, dtype=torch.float32)), dict(v_scales=scales.double()), dict(seq_lens=i32(2)), dict(row_offsets=i32(3)), dict(block_tables=i32(6)),
               dict(k_cache=cu(6, 2, 16, 128), v_cache=cu(6, 2, 16, 128)), dict(status_ws=ws[:100])):
        with bad:
            app(**kw)
    with pytest.raises(mt.MedusaTreeError):
        app(k_cache=cu(6, 2, 32, 128, dtype=torch.float8_e4m3fn), v_cache=cu(6, 2, 32, 128, dtype=torch.float8_e4m3fn))

    q4, n4 = cu(3, 4, 8, 128), cu(3, 4, 2, 128)
    aws = mt.alloc_block8_workspace(q4, cache, table)
    attn = lambda **kw: mt.tree_attn_paged_block8(**{**dict(q=q4, k_cache=cache, v_cache=cache, k_scales=scales + 1, v_scales=scales + 1, block_tables=table,  # noqa: E731
                                                            seq_lens=i32(3), tree_parents=None, out=torch.empty_like(q4), k_new=n4, v_new=n4, workspace=aws), **kw})
    attn()
    for kw in (dict(q=q4.float()), dict(q=cu(3, 4, 8, 64)), dict(k_new=cu(3, 4, 3, 128)), dict(v_new=cu(3, 5, 2, 128)), dict(out=cu(3, 4, 8, 64)), dict(k_cache=cu(6, 2, 16, 128)),
               dict(v_cache=cache[:3]), dict(k_scales=scales[:3]), dict(seq_lens=i32(4)), dict(tree_parents=i32(3, 3)), dict(block_tables=i32(2, 2)), dict(workspace=None),
               dict(workspace=aws.cpu()), dict(v_new=cu(3, 4, 4, 128)[:, :, ::2])):
        with bad:
            attn(**kw)
    with pytest.raises(mt.MedusaTreeError):
        attn(workspace=aws[:512])
    with pytest.raises(mt.MedusaTreeError):
        attn(sm_scale=-1.0)

    x, u, tok = cu(4, 33), cu(4, dtype=torch.float32), i32(4)
    draw = lambda **kw: mt.sample_tokens(**{**dict(logits=x, uniforms=u, tokens=tok), **kw})  # noqa: E731
    draw()
    for kw in (dict(logits=x.t()), dict(logits=x.double()), dict(logits=x[0]), dict(uniforms=u[:3]), dict(uniforms=u.double()), dict(tokens=tok.long()), dict(tokens=i32(5)),
               dict(temperature=u[:1]), dict(top_k=u), dict(top_p=tok), dict(min_p=u.cpu()), dict(row_index=i32(4, 1)), dict(row_index=i32(3))):
        with bad:
            draw(**kw)
    with pytest.raises(mt.MedusaTreeError):
        draw(logits=cu(4, 500001))
    torch.cuda.synchronize()
