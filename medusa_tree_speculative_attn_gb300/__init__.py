"""Medusa tree-verification step for NVIDIA GB300 (sm_103a).

A thin ctypes binding over ``lib/libmedusa_tree.so`` (C ABI in
``include/medusa_tree.h``).  Python only marshals arguments: every step of the
path (RoPE, tree mask, attention, combine, argmax, acceptance, commit) runs in
the library's CUDA kernels.  PyTorch supplies device memory and the stream.
There is no CPU fallback: if the library is missing this module raises.

Calls (same names as the C ABI without the ``mt_`` prefix):
  tree_attn_paged    tree tokens attend to the paged prefix + their ancestors
  tree_accept_greedy per-node argmax and the longest matching root path
  kv_commit          move accepted K/V into place, grow lengths, release pages
  tree_accept_commit the last two in one launch
  tree_candidates    the tree's tokens from the base and Medusa-head logits
  qk_norm_rope       norms of query and key heads, with the rotation in the same pass
  kv_append_paged    new keys and values into the paged cache (prompts, decoding steps)
  kv_append_accepted an accepted path's keys and values into the paged cache
  tree_attn_paged_block8  tree attention over an 8-bit cache with a scale per page and head
  sample_tokens      temperature, top-k, top-p and min-p from given uniform numbers
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmedusa_tree.so")

MT_OK = 0
KERNELS = {"auto": 0, "simt": 1, "tc": 2}
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MT_E4M3 = 3  # cache element type: OCP FP8 E4M3 codes (torch.float8_e4m3fn)


class MedusaTreeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status} ({status_string(status)})")


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("tree_size", ctypes.c_int),
                ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("num_splits", ctypes.c_int), ("dtype", ctypes.c_int),
                ("sm_scale", ctypes.c_float), ("kernel", ctypes.c_int),
                ("cache_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class NormRopeDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int), ("num_q_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_stride", ctypes.c_longlong * 2),
                ("k_stride", ctypes.c_longlong * 2), ("q_out_stride", ctypes.c_longlong * 2),
                ("k_out_stride", ctypes.c_longlong * 2)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("num_rows", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_blocks_per_seq", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("dtype", ctypes.c_int), ("cache_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("k_stride", ctypes.c_longlong * 2),
                ("v_stride", ctypes.c_longlong * 2)]


# The descriptors as the binding passes them: the same bytes, packed in one go
# (filling a ctypes structure costs several times as much).
_NORM_ROPE_DESC = struct.Struct("@5if8q")
_APPEND_DESC = struct.Struct("@9i2f4q")
_ATTN_DESC = struct.Struct("@10ifi" "i2f")
assert (_NORM_ROPE_DESC.size == ctypes.sizeof(NormRopeDesc) and _APPEND_DESC.size == ctypes.sizeof(AppendDesc)
        and _ATTN_DESC.size == ctypes.sizeof(AttnDesc))

_lib = None


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "(there is no fallback path)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        D = ctypes.POINTER(AttnDesc)
        lib.mt_version.restype = I
        lib.mt_status_string.argtypes = [I]
        lib.mt_status_string.restype = ctypes.c_char_p
        lib.mt_rope_create.argtypes = [ctypes.c_double, I, I, ctypes.POINTER(P)]
        lib.mt_rope_destroy.argtypes = [P]
        lib.mt_tree_attn_workspace_size.argtypes = [D]
        lib.mt_tree_attn_workspace_size.restype = Z
        lib.mt_tree_attn_paged.argtypes = [D] + [P] * 12 + [Z, P]
        lib.mt_tree_accept_workspace_size.argtypes = [I, I]
        lib.mt_tree_accept_workspace_size.restype = Z
        lib.mt_tree_accept_greedy.argtypes = [I, I, I, I, I] + [P] * 8 + [Z, P]
        lib.mt_tree_accept_typical.argtypes = ([I, I, I, I, I] + [P] * 3 + [ctypes.c_float] * 3 +
                                               [P] * 5 + [Z, P])
        lib.mt_kv_commit.argtypes = [D, I] + [P] * 8 + [P]
        lib.mt_tree_accept_commit.argtypes = [D, I, I, I] + [P] * 12 + [P, Z, P]
        lib.mt_tree_candidates.argtypes = [I, I, I, I, I] + [P] * 5 + [P]
        L = ctypes.c_longlong
        lib.mt_qk_norm_rope.argtypes = [P] + [P] * 10
        lib.mt_kv_append_paged.argtypes = [P] + [P] * 12
        lib.mt_kv_append_accepted.argtypes = [P, I, I] + [P] * 13
        lib.mt_tree_attn_block8_workspace_size.argtypes = [P]
        lib.mt_tree_attn_block8_workspace_size.restype = Z
        lib.mt_tree_attn_paged_block8.argtypes = [P] + [P] * 12 + [Z, P]
        lib.mt_sample_tokens.argtypes = [I, I, I, P, I, L] + [P] * 7 + [P]
        lib.mt_read_status.argtypes = [P, P, ctypes.POINTER(I)]
        lib.mt_profile_enable.argtypes = [I]
        lib.mt_profile_read.argtypes = [ctypes.POINTER(ctypes.c_float), I, ctypes.POINTER(I)]
        lib.mt_debug_set_wait.argtypes = [ctypes.c_ulonglong, I]
        _lib = lib
    return _lib


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _load()


def status_string(status: int) -> str:
    return _load().mt_status_string(int(status)).decode()


def _check(st: int, what: str):
    if st != MT_OK:
        raise MedusaTreeError(st, what)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _shape(t: torch.Tensor, name: str, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _min_bytes(t: torch.Tensor, name: str, n: int):
    if t.numel() * t.element_size() < n:
        raise ValueError(f"{name} must hold at least {n} bytes")


def _on_device(**tensors):
    """Every tensor on the first one's CUDA device: the kernels dereference the
    pointers as device memory, so a host tensor must never reach them."""
    dev = None
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")


class Rope:
    """Library-owned fp32 cos/sin table on the current device."""

    def __init__(self, base: float, head_dim: int, max_pos: int):
        self._lib = _load()
        self.handle = ctypes.c_void_p()
        _check(self._lib.mt_rope_create(float(base), int(head_dim), int(max_pos),
                                        ctypes.byref(self.handle)), "mt_rope_create")
        self.base, self.head_dim, self.max_pos = base, head_dim, max_pos

    def __del__(self):
        if getattr(self, "handle", None) and self.handle.value:
            self._lib.mt_rope_destroy(self.handle)
            self.handle = ctypes.c_void_p()


def _fp8(cache: torch.Tensor) -> bool:
    return cache.dtype == torch.float8_e4m3fn


def make_desc(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
              num_splits: int = 0, kernel: str = "auto", sm_scale: float = 0.0,
              k_scale: float = 1.0, v_scale: float = 1.0) -> AttnDesc:
    """The call's descriptor; an FP8 E4M3 cache (torch.float8_e4m3fn) holds the
    codes of value / k_scale (keys) and value / v_scale (values)."""
    B, T, Hq, D = q.shape
    num_pages, Hkv, P, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache head_dim differ")
    return AttnDesc(B, T, Hq, Hkv, D, P, block_tables.shape[1], num_pages, int(num_splits),
                    _DTYPES[q.dtype], float(sm_scale), KERNELS[kernel],
                    MT_E4M3 if _fp8(k_cache) else 0, float(k_scale), float(v_scale))


def _commit_desc(B: int, T: int, k_cache: torch.Tensor, max_blocks: int) -> AttnDesc:
    num_pages, Hkv, P, D = k_cache.shape
    if _fp8(k_cache):   # the act dtype does not matter to a commit: bytes move as they are
        return AttnDesc(B, T, Hkv, Hkv, D, P, max_blocks, num_pages, 0, _DTYPES[torch.bfloat16],
                        0.0, 0, MT_E4M3, 1.0, 1.0)
    return AttnDesc(B, T, Hkv, Hkv, D, P, max_blocks, num_pages, 0, _DTYPES[k_cache.dtype], 0.0, 0,
                    0, 1.0, 1.0)


def attn_workspace_size(desc: AttnDesc) -> int:
    return int(_load().mt_tree_attn_workspace_size(ctypes.byref(desc)))


def alloc_attn_workspace(desc: AttnDesc, device="cuda") -> torch.Tensor:
    n = attn_workspace_size(desc)
    if n == 0:
        raise MedusaTreeError(-1, "mt_tree_attn_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def accept_workspace_size(batch: int, tree_size: int) -> int:
    return int(_load().mt_tree_accept_workspace_size(int(batch), int(tree_size)))


def alloc_accept_workspace(batch: int, tree_size: int, device="cuda") -> torch.Tensor:
    return torch.zeros(accept_workspace_size(batch, tree_size), dtype=torch.uint8, device=device)


def tree_attn_paged(q, k_cache, v_cache, block_tables, seq_lens, tree_parents, tree_depths, out, *,
                    k_new, v_new, rope: Rope, workspace: torch.Tensor, num_splits: int = 0,
                    kernel: str = "auto", sm_scale: float = 0.0, k_scale: float = 1.0,
                    v_scale: float = 1.0, stream=None):
    """out[b,i,h] = attention of tree node i (head h) over the prefix + its ancestors.

    The caches hold q's dtype, or FP8 E4M3 codes (torch.float8_e4m3fn) of
    value / k_scale and value / v_scale (read on either kernel; the tensor-core
    kernel converts the codes to q's dtype in shared memory)."""
    for name, t in (("q", q), ("k_new", k_new), ("v_new", v_new), ("out", out)):
        _need(t, name, q.dtype, 4)
    cache_dtype = torch.float8_e4m3fn if _fp8(k_cache) else q.dtype
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, cache_dtype, 4)
    for name, t in (("block_tables", block_tables), ("tree_parents", tree_parents),
                    ("tree_depths", tree_depths)):
        _need(t, name, torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(workspace, "workspace")
    B, T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _shape(t, name, (B, T, Hkv, D))
    _shape(out, "out", q.shape)
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(seq_lens, "seq_lens", (B,))
    if block_tables.shape[0] != B:
        raise ValueError("block_tables must have one row per sequence")
    for name, t in (("tree_parents", tree_parents), ("tree_depths", tree_depths)):
        _shape(t, name, (B, T))
    desc = make_desc(q, k_cache, block_tables, num_splits, kernel, sm_scale, k_scale, v_scale)
    _on_device(q=q, k_new=k_new, v_new=v_new, out=out, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, seq_lens=seq_lens, tree_parents=tree_parents,
               tree_depths=tree_depths, workspace=workspace)
    st = _load().mt_tree_attn_paged(ctypes.byref(desc), _ptr(q), _ptr(k_new), _ptr(v_new),
                                    _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                    _ptr(seq_lens), _ptr(tree_parents), _ptr(tree_depths),
                                    rope.handle, _ptr(out), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "mt_tree_attn_paged")
    return out


def tree_accept_greedy(tree_tokens, target_logits, tree_parents, accept_len, accept_path, *,
                       argmax_out, next_token, workspace: torch.Tensor, max_depth: Optional[int] = None,
                       stream=None):
    """Greedy acceptance; fills argmax_out, accept_len, accept_path, next_token."""
    _need(tree_tokens, "tree_tokens", torch.int32, 2)
    _need(tree_parents, "tree_parents", torch.int32, 2)
    _need(target_logits, "target_logits", None, 3)
    for name, t in (("accept_len", accept_len), ("next_token", next_token)):
        _need(t, name, torch.int32, 1)
    _need(accept_path, "accept_path", torch.int32, 2)
    _need(argmax_out, "argmax_out", torch.int32, 2)
    _need(workspace, "workspace")
    B, T = tree_tokens.shape
    V = target_logits.shape[2]
    if max_depth is None:
        max_depth = accept_path.shape[1] - 1
    if accept_path.shape[1] != max_depth + 1:
        raise ValueError("accept_path must have max_depth + 1 columns")
    _accept_shapes(B, T, V, target_logits, tree_parents, accept_len, accept_path, next_token,
                   argmax_out=argmax_out)
    _on_device(tree_tokens=tree_tokens, target_logits=target_logits, tree_parents=tree_parents,
               argmax_out=argmax_out, accept_len=accept_len, accept_path=accept_path,
               next_token=next_token, workspace=workspace)
    st = _load().mt_tree_accept_greedy(B, T, V, int(max_depth), _DTYPES[target_logits.dtype],
                                       _ptr(tree_tokens), _ptr(target_logits), _ptr(tree_parents),
                                       _ptr(argmax_out), _ptr(accept_len), _ptr(accept_path),
                                       _ptr(next_token), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "mt_tree_accept_greedy")
    return accept_len, accept_path


def _accept_shapes(B, T, V, target_logits, tree_parents, accept_len, accept_path, next_token, **per_node):
    _shape(target_logits, "target_logits", (B, T, V))
    _shape(tree_parents, "tree_parents", (B, T))
    _shape(accept_len, "accept_len", (B,))
    _shape(next_token, "next_token", (B,))
    if accept_path.shape[0] != B:
        raise ValueError("accept_path must have one row per sequence")
    for name, t in per_node.items():
        _shape(t, name, (B, T))


def tree_accept_typical(tree_tokens, target_logits, tree_parents, accept_len, accept_path, *,
                        node_accept, next_token, workspace: torch.Tensor, temperature: float,
                        epsilon: float, delta: float, max_depth: Optional[int] = None, stream=None):
    """Typical acceptance: node i passes when its token's probability under its
    parent's tempered row exceeds min(epsilon, delta * exp(-entropy)); fills
    node_accept, accept_len, accept_path, next_token (the end row's argmax)."""
    _need(tree_tokens, "tree_tokens", torch.int32, 2)
    _need(tree_parents, "tree_parents", torch.int32, 2)
    _need(target_logits, "target_logits", None, 3)
    for name, t in (("accept_len", accept_len), ("next_token", next_token)):
        _need(t, name, torch.int32, 1)
    _need(accept_path, "accept_path", torch.int32, 2)
    _need(node_accept, "node_accept", torch.int32, 2)
    _need(workspace, "workspace")
    B, T = tree_tokens.shape
    V = target_logits.shape[2]
    if max_depth is None:
        max_depth = accept_path.shape[1] - 1
    if accept_path.shape[1] != max_depth + 1:
        raise ValueError("accept_path must have max_depth + 1 columns")
    _accept_shapes(B, T, V, target_logits, tree_parents, accept_len, accept_path, next_token,
                   node_accept=node_accept)
    _on_device(tree_tokens=tree_tokens, target_logits=target_logits, tree_parents=tree_parents,
               node_accept=node_accept, accept_len=accept_len, accept_path=accept_path,
               next_token=next_token, workspace=workspace)
    st = _load().mt_tree_accept_typical(B, T, V, int(max_depth), _DTYPES[target_logits.dtype],
                                        _ptr(tree_tokens), _ptr(target_logits), _ptr(tree_parents),
                                        float(temperature), float(epsilon), float(delta),
                                        _ptr(node_accept), _ptr(accept_len), _ptr(accept_path),
                                        _ptr(next_token), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "mt_tree_accept_typical")
    return accept_len, accept_path


def released_width(tree_size: int, page_size: int) -> int:
    return (tree_size + 2 * page_size - 2) // page_size


def kv_commit(accept_path, accept_len, k_cache, v_cache, block_tables, seq_lens, released_pages, *,
              tree_size: int, status_ws: torch.Tensor, stream=None):
    """Commit accepted K/V, grow seq_lens, release scratch pages (in place)."""
    _need(accept_path, "accept_path", torch.int32, 2)
    _need(accept_len, "accept_len", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(released_pages, "released_pages", torch.int32, 2)
    _need(k_cache, "k_cache", None, 4)
    _need(v_cache, "v_cache", k_cache.dtype, 4)
    _need(status_ws, "status_ws")
    P = k_cache.shape[2]
    B = block_tables.shape[0]
    if released_pages.shape != (B, released_width(tree_size, P)):
        raise ValueError("released_pages must be [B, (T + 2P - 2) // P]")
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(accept_len, "accept_len", (B,))
    _shape(seq_lens, "seq_lens", (B,))
    if accept_path.shape[0] != B:
        raise ValueError("accept_path must have one row per sequence")
    _min_bytes(status_ws, "status_ws", 256)
    desc = _commit_desc(B, int(tree_size), k_cache, block_tables.shape[1])
    _on_device(accept_path=accept_path, accept_len=accept_len, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, seq_lens=seq_lens, released_pages=released_pages,
               status_ws=status_ws)
    st = _load().mt_kv_commit(ctypes.byref(desc), accept_path.shape[1] - 1, _ptr(accept_path),
                              _ptr(accept_len), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                              _ptr(seq_lens), _ptr(released_pages), _ptr(status_ws), _stream(stream))
    _check(st, "mt_kv_commit")


def tree_accept_commit(tree_tokens, target_logits, tree_parents, accept_len, accept_path, k_cache,
                       v_cache, block_tables, seq_lens, released_pages, *, argmax_out, next_token,
                       workspace: torch.Tensor, max_depth: Optional[int] = None, stream=None):
    """tree_accept_greedy followed by kv_commit, in one launch (same results)."""
    _need(tree_tokens, "tree_tokens", torch.int32, 2)
    _need(tree_parents, "tree_parents", torch.int32, 2)
    _need(target_logits, "target_logits", None, 3)
    for name, t in (("accept_len", accept_len), ("next_token", next_token), ("seq_lens", seq_lens)):
        _need(t, name, torch.int32, 1)
    for name, t in (("accept_path", accept_path), ("argmax_out", argmax_out),
                    ("block_tables", block_tables), ("released_pages", released_pages)):
        _need(t, name, torch.int32, 2)
    _need(k_cache, "k_cache", None, 4)
    _need(v_cache, "v_cache", k_cache.dtype, 4)
    _need(workspace, "workspace")
    B, T = tree_tokens.shape
    V = target_logits.shape[2]
    if max_depth is None:
        max_depth = accept_path.shape[1] - 1
    if accept_path.shape[1] != max_depth + 1:
        raise ValueError("accept_path must have max_depth + 1 columns")
    P = k_cache.shape[2]
    if released_pages.shape != (B, released_width(T, P)):
        raise ValueError("released_pages must be [B, (T + 2P - 2) // P]")
    _accept_shapes(B, T, V, target_logits, tree_parents, accept_len, accept_path, next_token,
                   argmax_out=argmax_out)
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(seq_lens, "seq_lens", (B,))
    if block_tables.shape[0] != B:
        raise ValueError("block_tables must have one row per sequence")
    desc = _commit_desc(B, int(T), k_cache, block_tables.shape[1])
    _on_device(tree_tokens=tree_tokens, target_logits=target_logits, tree_parents=tree_parents,
               argmax_out=argmax_out, accept_len=accept_len, accept_path=accept_path,
               next_token=next_token, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               seq_lens=seq_lens, released_pages=released_pages, workspace=workspace)
    st = _load().mt_tree_accept_commit(ctypes.byref(desc), V, int(max_depth),
                                       _DTYPES[target_logits.dtype], _ptr(tree_tokens),
                                       _ptr(target_logits), _ptr(tree_parents), _ptr(argmax_out),
                                       _ptr(accept_len), _ptr(accept_path), _ptr(next_token),
                                       _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                       _ptr(seq_lens), _ptr(released_pages), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "mt_tree_accept_commit")
    return accept_len, accept_path


def tree_candidates(root_logits, head_logits, tree_parents, tree_tokens, *, status_ws: torch.Tensor,
                    stream=None):
    """Tree tokens from the base logits [B,V] and the Medusa heads' logits [B,heads,V]:
    node 0 takes the argmax of the base logits, the r-th child (r earlier siblings)
    of a depth-(d-1) node the rank-r token of head d-1."""
    _need(root_logits, "root_logits", None, 2)
    _need(head_logits, "head_logits", root_logits.dtype, 3)
    _need(tree_parents, "tree_parents", torch.int32, 2)
    _need(tree_tokens, "tree_tokens", torch.int32, 2)
    B, V = root_logits.shape
    heads = head_logits.shape[1]
    if head_logits.shape != (B, heads, V):
        raise ValueError("head_logits must be [B, heads, V]")
    T = tree_parents.shape[1]
    if tree_parents.shape != (B, T) or tree_tokens.shape != (B, T):
        raise ValueError("tree_parents and tree_tokens must be [B, T]")
    _need(status_ws, "status_ws")
    _min_bytes(status_ws, "status_ws", 256)
    _on_device(root_logits=root_logits, head_logits=head_logits, tree_parents=tree_parents,
               tree_tokens=tree_tokens, status_ws=status_ws)
    st = _load().mt_tree_candidates(B, T, heads, V, _DTYPES[root_logits.dtype], _ptr(root_logits),
                                    _ptr(head_logits), _ptr(tree_parents), _ptr(tree_tokens),
                                    _ptr(status_ws), _stream(stream))
    _check(st, "mt_tree_candidates")
    return tree_tokens


# ---- the serving operators around the step ----------------------------------
#
# One check per argument (dtype, shape, device, layout), then the call on the
# arguments' device.  A decoding step makes several of these calls per layer, so
# an argument that fits costs one pass over its attributes; the reason is worked
# out for one that does not.

_E4M3 = torch.float8_e4m3fn


def _refuse(t, name, dtype, shape, dev, layout):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    raise ValueError(f"{name} must {layout}, got strides {t.stride()}")


def _arg(t, name, dtype, shape, dev):
    """A dense CUDA tensor of this dtype, shape and device; its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev, "be contiguous")


def _rows_arg(t, name, dtype, shape, dev):
    """A CUDA tensor [rows, heads, D] whose head rows are dense and 16-byte
    aligned (a view of a projection's output, say); its address and strides."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev:
            s0, s1, s2 = t.stride()
            if shape[0] <= 1:
                s0 = 0
            if shape[1] <= 1:
                s1 = 0
            p = t.data_ptr()
            if s2 == 1 and not (p | (s0 | s1) * t.element_size()) & 15:
                return p, s0, s1
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev, "have dense, 16-byte aligned head rows")


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    return t.device


def _act(t, name, kinds=_DTYPES):
    if t.dtype not in kinds:
        raise ValueError(f"{name} must be one of {sorted(str(k) for k in kinds)}, got {t.dtype}")
    return _DTYPES[t.dtype]


def _status_arg(t, name, dev, nbytes=256):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} must be a dense tensor of at least {nbytes} bytes on {dev}")
    return t.data_ptr()


def _invoke(fn, what, dev, stream, *args):
    """The call on its tensors' device: on `stream`, or that device's current one."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev.index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != MT_OK:
        raise MedusaTreeError(st, what)


def qk_norm_rope(q, k, positions, q_out, k_out, *, rope: Optional[Rope] = None, q_weight=None,
                 k_weight=None, eps: float = 1e-6, status_ws: torch.Tensor, stream=None):
    """Norms every head row of q [N,Hq,D] and k [N,Hkv,D] (with weights [D]) and
    rotates it at positions[i] (with rope), into q_out and k_out (which may be q
    and k).  A negative position leaves its rows as they were.  q, k and the
    outputs may be views with dense head rows."""
    dev = _cuda_device(q, "q")
    dt = _act(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q and k must have 3 dims (tokens, heads, head_dim)")
    n, hq, d = q.shape
    hkv = k.shape[1]
    ty, qshape, kshape = q.dtype, (n, hq, d), (n, hkv, d)
    qp, q0, q1 = _rows_arg(q, "q", ty, qshape, dev)
    kp, k0, k1 = _rows_arg(k, "k", ty, kshape, dev)
    qop, qo0, qo1 = _rows_arg(q_out, "q_out", ty, qshape, dev)
    kop, ko0, ko1 = _rows_arg(k_out, "k_out", ty, kshape, dev)
    if (n > 1 and not (qo0 and ko0)) or (hq > 1 and not qo1) or (hkv > 1 and not ko1):
        raise ValueError("q_out and k_out must not be expanded views")
    pos = None if positions is None else _arg(positions, "positions", torch.int32, (n,), dev)
    if rope is not None and positions is None:
        raise ValueError("a rotation needs positions")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if q_weight is None and rope is None:
        raise ValueError("nothing to do: neither weights nor rope")
    qw = None if q_weight is None else _arg(q_weight, "q_weight", ty, (d,), dev)
    kw = None if k_weight is None else _arg(k_weight, "k_weight", ty, (d,), dev)
    desc = _NORM_ROPE_DESC.pack(n, hq, hkv, d, dt, eps, q0, q1, k0, k1, qo0, qo1, ko0, ko1)
    _invoke(_load().mt_qk_norm_rope, "mt_qk_norm_rope", dev, stream, desc, qp, kp, pos, qw, kw,
            None if rope is None else rope.handle, qop, kop, _status_arg(status_ws, "status_ws", dev))
    return q_out, k_out


def _append_args(k, v, k_cache, v_cache, block_tables, seq_lens, k_scales, v_scales, k_scale, v_scale):
    """Checks shared by the appends: the batch, the descriptor and the addresses."""
    dev = _cuda_device(k, "k")
    dt = _act(k, "k")
    n, hkv, d = k.shape
    kp, k0, k1 = _rows_arg(k, "k", k.dtype, (n, hkv, d), dev)
    vp, v0, v1 = _rows_arg(v, "v", k.dtype, (n, hkv, d), dev)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must have 4 dims (pages, heads, slots, head_dim)")
    cdt = k_cache.dtype
    if cdt is not k.dtype and cdt is not _E4M3:
        raise ValueError(f"k_cache must be {k.dtype} or {_E4M3}, got {cdt}")
    pages, page = k_cache.shape[0], k_cache.shape[2]
    kcp = _arg(k_cache, "k_cache", cdt, (pages, hkv, page, d), dev)
    vcp = _arg(v_cache, "v_cache", cdt, (pages, hkv, page, d), dev)
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise ValueError("block_tables must have 2 dims")
    b, blocks = block_tables.shape
    btp = _arg(block_tables, "block_tables", torch.int32, (b, blocks), dev)
    slp = _arg(seq_lens, "seq_lens", torch.int32, (b,), dev)
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales go together")
    ksp = vsp = None
    if k_scales is not None:
        if cdt is not _E4M3:
            raise ValueError(f"block scales need a cache of {_E4M3}")
        ksp = _arg(k_scales, "k_scales", torch.float32, (pages, hkv), dev)
        vsp = _arg(v_scales, "v_scales", torch.float32, (pages, hkv), dev)
    desc = _APPEND_DESC.pack(b, n, hkv, d, page, blocks, pages, dt, MT_E4M3 if cdt is _E4M3 else 0,
                             k_scale, v_scale, k0, k1, v0, v1)
    return dev, b, desc, (kp, vp), (kcp, vcp, ksp, vsp, btp, slp)


def kv_append_paged(k, v, k_cache, v_cache, block_tables, seq_lens, row_offsets, *,
                    status_ws: torch.Tensor, rope: Optional[Rope] = None, k_scales=None, v_scales=None,
                    k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """New keys and values k, v [N,Hkv,D] into the paged cache: rows
    row_offsets[b] .. row_offsets[b+1]-1 go to sequence b's slots from
    seq_lens[b] on, the keys rotated at their slots (with rope).  The cache holds
    k's dtype, E4M3 codes under k_scale / v_scale, or E4M3 codes under
    k_scales / v_scales [pages,Hkv] (updated).  seq_lens is not changed."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must have 3 dims (rows, heads, head_dim)")
    dev, b, desc, kv, rest = _append_args(k, v, k_cache, v_cache, block_tables, seq_lens, k_scales,
                                          v_scales, k_scale, v_scale)
    off = _arg(row_offsets, "row_offsets", torch.int32, (b + 1,), dev)
    _invoke(_load().mt_kv_append_paged, "mt_kv_append_paged", dev, stream, desc, *kv, off,
            None if rope is None else rope.handle, *rest, _status_arg(status_ws, "status_ws", dev))


def kv_append_accepted(k_new, v_new, accept_path, accept_len, k_cache, v_cache, block_tables, seq_lens,
                       *, status_ws: torch.Tensor, rope: Optional[Rope] = None, k_scales=None,
                       v_scales=None, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """The accepted path's keys and values into the paged cache: row i of
    sequence b is node accept_path[b,i] of k_new, v_new [B,T,Hkv,D], i up to
    accept_len[b].  Otherwise as kv_append_paged; seq_lens is not changed (it
    grows by accept_len + 1 once every layer has appended)."""
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must have 4 dims (batch, tree, heads, head_dim)")
    if not isinstance(v_new, torch.Tensor) or v_new.shape != k_new.shape:
        raise ValueError("v_new must have k_new's shape")
    if not k_new.is_contiguous() or not v_new.is_contiguous():
        raise ValueError("k_new and v_new must be contiguous")
    b, t, hkv, d = k_new.shape
    dev, nb, desc, kv, rest = _append_args(k_new.view(b * t, hkv, d), v_new.view(b * t, hkv, d),
                                           k_cache, v_cache, block_tables, seq_lens, k_scales, v_scales,
                                           k_scale, v_scale)
    if nb != b:
        raise ValueError("block_tables must have one row per sequence")
    if not isinstance(accept_path, torch.Tensor) or accept_path.dim() != 2:
        raise ValueError("accept_path must have 2 dims")
    path = _arg(accept_path, "accept_path", torch.int32, (b, accept_path.shape[1]), dev)
    length = _arg(accept_len, "accept_len", torch.int32, (b,), dev)
    _invoke(_load().mt_kv_append_accepted, "mt_kv_append_accepted", dev, stream, desc, t,
            accept_path.shape[1] - 1, *kv, path, length, None if rope is None else rope.handle, *rest,
            _status_arg(status_ws, "status_ws", dev))


def _block8_desc(q, k_cache, block_tables, sm_scale=0.0):
    b, t, hq, d = q.shape
    pages, hkv, page = k_cache.shape[:3]
    return _ATTN_DESC.pack(b, t, hq, hkv, d, page, block_tables.shape[1], pages, 0, _DTYPES[q.dtype],
                           sm_scale, 0, MT_E4M3, 1.0, 1.0)


def alloc_block8_workspace(q, k_cache, block_tables) -> torch.Tensor:
    """The workspace of tree_attn_paged_block8 for these sizes, on q's device."""
    dev = _cuda_device(q, "q")
    _act(q, "q", (torch.float16, torch.bfloat16))
    with torch.cuda.device(dev):
        n = int(_load().mt_tree_attn_block8_workspace_size(_block8_desc(q, k_cache, block_tables)))
    if n == 0:
        raise MedusaTreeError(-1, "mt_tree_attn_block8_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=dev)


def tree_attn_paged_block8(q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens,
                           tree_parents, out, *, k_new, v_new, workspace: torch.Tensor,
                           sm_scale: float = 0.0, stream=None):
    """out[b,i,h] = attention of new token i (head h) over the cached slots
    0 .. seq_lens[b]-1 and its tree ancestors, itself included (tree_parents
    None: the tokens are a chain; T = 1: a decoding step).

    The cache holds E4M3 codes under k_scales / v_scales [pages,Hkv] and is only
    read; q and k_new are rotated already (qk_norm_rope); the new keys and values
    are seen as kv_append_paged would store them, in blocks of 16 tokens.  A
    sequence with seq_lens[b] < 0 leaves its rows of out as they were.  out must
    not overlap q, k_new or v_new; the workspace serves any call that it is large
    enough for, one at a time."""
    dev = _cuda_device(q, "q")
    dt = q.dtype
    _act(q, "q", (torch.float16, torch.bfloat16))
    if q.dim() != 4 or not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("q and k_cache must have 4 dims")
    b, t, hq, d = q.shape
    pages, hkv, page = k_cache.shape[:3]
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise ValueError("block_tables must have 2 dims")
    cache, scales, new, rows = (pages, hkv, page, d), (pages, hkv), (b, t, hkv, d), (b, t, hq, d)
    f32, i32 = torch.float32, torch.int32
    _invoke(_load().mt_tree_attn_paged_block8, "mt_tree_attn_paged_block8", dev, stream,
            _block8_desc(q, k_cache, block_tables, sm_scale), _arg(q, "q", dt, rows, dev),
            _arg(k_new, "k_new", dt, new, dev), _arg(v_new, "v_new", dt, new, dev),
            _arg(k_cache, "k_cache", _E4M3, cache, dev), _arg(v_cache, "v_cache", _E4M3, cache, dev),
            _arg(k_scales, "k_scales", f32, scales, dev), _arg(v_scales, "v_scales", f32, scales, dev),
            _arg(block_tables, "block_tables", i32, (b, block_tables.shape[1]), dev),
            _arg(seq_lens, "seq_lens", i32, (b,), dev),
            None if tree_parents is None else _arg(tree_parents, "tree_parents", i32, (b, t), dev),
            _arg(out, "out", dt, rows, dev), _status_arg(workspace, "workspace", dev),
            workspace.numel() * workspace.element_size())
    return out


def sample_tokens(logits, uniforms, tokens, *, temperature=None, top_k=None, top_p=None, min_p=None,
                  row_index=None, stream=None):
    """Draws tokens[i] from row row_index[i] (row i without it) of logits [R,V]
    with the given uniforms [N]: temperature (<= 0: the argmax), top_k, top_p and
    min_p are tensors [N] or None.  Rows of logits may be strided; a negative
    row_index leaves its token as it was."""
    dev = _cuda_device(logits, "logits")
    dt = _act(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must have 2 dims")
    r, v = logits.shape
    st = logits.stride()
    if v > 1 and st[1] != 1:
        raise ValueError("logits must have dense rows")
    n = r
    if row_index is not None:
        if not isinstance(row_index, torch.Tensor) or row_index.dim() != 1:
            raise ValueError("row_index must have 1 dim")
        n = row_index.shape[0]
    f32, i32, one = torch.float32, torch.int32, (n,)
    opt = lambda t, name, ty: None if t is None else _arg(t, name, ty, one, dev)  # noqa: E731
    _invoke(_load().mt_sample_tokens, "mt_sample_tokens", dev, stream, n, v, dt, logits.data_ptr(), r,
            st[0] if r > 1 else 0, opt(row_index, "row_index", i32), _arg(uniforms, "uniforms", f32, one, dev),
            opt(temperature, "temperature", f32), opt(top_k, "top_k", i32), opt(top_p, "top_p", f32),
            opt(min_p, "min_p", f32), _arg(tokens, "tokens", i32, one, dev))
    return tokens


def read_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronises the stream, returns and clears the device status word."""
    _need(workspace, "workspace")
    _min_bytes(workspace, "workspace", 4)
    _on_device(workspace=workspace)
    v = ctypes.c_int(0)
    _check(_load().mt_read_status(_ptr(workspace), _stream(stream), ctypes.byref(v)), "mt_read_status")
    return v.value


def profile_enable(max_records: int):
    """Record CUDA events around the main attention kernel of the next calls."""
    _check(_load().mt_profile_enable(int(max_records)), "mt_profile_enable")


def profile_read(max_records: int = 65536):
    """Elapsed milliseconds of the main attention kernel, one per recorded call."""
    buf = (ctypes.c_float * max_records)()
    n = ctypes.c_int(0)
    _check(_load().mt_profile_read(buf, max_records, ctypes.byref(n)), "mt_profile_read")
    return [buf[i] for i in range(n.value)]


def debug_set_wait(limit_ns: int = 0, stall: bool = False):
    """Bound of the tensor-core kernel's pipeline waits for later attention
    calls (0: the default, 2 s); stall=True makes its first wait one that only
    a timeout ends (tests of the timeout path)."""
    _check(_load().mt_debug_set_wait(int(limit_ns), 1 if stall else 0), "mt_debug_set_wait")


def version() -> int:
    return int(_load().mt_version())
