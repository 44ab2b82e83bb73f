"""Python binding of libkvq (rotated INT2 KV-cache attention for GB300).

Argument marshalling only: every computation runs in the CUDA kernels of
``libkvq.so`` behind the C ABI declared in ``include/kvq.h``.  PyTorch supplies
device memory and streams.  There is no CPU path: if the library has not been
built, importing the binding functions raises.

Functions carry the C names (``kvq_quantize_append``, ``kvq_decode_attention``,
``kvq_out_proj``, ``kvq_calib_nmse`` and helpers) and take torch tensors.
Around the cache: ``kvq_norm_rope`` makes q, k and v of a layer's projections
(``Rope``), ``kvq_read_cache`` gives cached tokens back, and
``kvq_decode_attention_score`` and ``kvq_chunk_attention_score`` attend with capped
scores, a distance bias, a sliding window and a prefix (``Score``).

A decode step, end to end (shapes as in ``include/kvq.h``)::

    import torch, int2_kv_cache_gb300 as kvq
    from int2_kv_cache_gb300 import _build
    _build.build()                                   # nvcc, sm_103a, in-tree libkvq.so
    lay = kvq.make_layout(page_tokens=16, n_kv_heads=8, n_q_heads=32, num_blocks=nb, max_blocks_per_seq=mb)
    pool = torch.zeros(kvq.kvq_pool_bytes(lay), dtype=torch.uint8, device="cuda")
    rk = kvq.DeviceRot("dense", dense=r_k)           # [H_kv, 128, 128] fp32; or "signed_hadamard" / "identity"
    rv = kvq.DeviceRot("dense", dense=r_v)
    kvq.kvq_key_mean(k_calib, mu)                    # Eq. 19; then mu R_K (Eq. 20):
    kvq.kvq_rotate_heads(mu[None], rk, mu_rot[None])
    kvq.kvq_quantize_append(lay, k, v, cu_new, start_pos, table, rk, rv, mu_rot, 0.96, 0.92, pool)
    ws = torch.empty(kvq.kvq_decode_workspace_size(lay, n_seqs, max_len), dtype=torch.uint8, device="cuda")
    kvq.kvq_decode_attention(lay, q, seq_lens, max_len, table, rk, pool, ws, o_rot)
    kvq.kvq_fold_wo(w_o, 32, 8, rv, w_fold)          # once: W_O R_V (Eqs. 29-31)
    kvq.kvq_out_proj(o_rot.reshape(n_seqs, -1), w_fold, y)

With BF16 sink / recent windows, add ``win = kvq.Window(64, 256, buf)`` (``buf`` of
``kvq.Window.buffer_bytes(n_seqs, 8, 64, 256)`` bytes), call ``kvq_window_append(lay,
k, v, cu_new, start_pos, mu, win)`` beside the append, and decode with
``kvq_decode_attention_win(lay, q, seq_lens, max_len, table, rk, rv, pool, win, ws, o_rot)``
(workspace from ``kvq_decode_workspace_size_win``).

Speculative decoding on the same pool: ``kvq_plan_pages`` (old -> new lengths: pages, ``cu_new``, slots),
``kvq_quantize_append`` (the drafts), ``kvq_tree_attention(lay, q, cu_new, max_drafts, parents, lens, max_len, table,
rk, pool, ws, o_rot)`` (workspace from ``kvq_query_block_workspace_size``), ``kvq_tree_commit`` (the accepted path) and
``kvq_plan_pages`` again for the pages of the rejected drafts.  ``kvq_cross_attention``: query blocks over an encoder's
cached states.  Candidate selection:
``kvq_calib_nmse``; per-head error report: ``kvq_head_error_report``.
"""
from __future__ import annotations

import ctypes
import math
import os

from ._build import LIB as LIB_PATH

KVQ_OK, KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_ECUDA, KVQ_EDEVICE_FLAG = 0, -1, -2, -3, -4
ROT_KIND = {"identity": 0, "signed_hadamard": 1, "dense": 2}
KVQ_F32, KVQ_BF16 = 0, 1
HEAD_DIM = 128


class KvqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"kvq status {status}: {message}")
        self.status = status


class KvqLayout(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int)]


class KvqRot(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("signs", ctypes.c_void_p), ("dense", ctypes.c_void_p)]


class KvqOptrTrace(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_tok", ctypes.c_int),
                ("n_qpos", ctypes.c_int)]


class KvqWindow(ctypes.Structure):
    _fields_ = [("sink_tokens", ctypes.c_int), ("recent_tokens", ctypes.c_int), ("buf", ctypes.c_void_p)]


class KvqRope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("inv_freq", ctypes.c_void_p), ("axis", ctypes.c_void_p)]


class KvqScore(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("window", ctypes.c_int),
                ("prefix_lens", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libkvq.so (built in-tree by ``_build.build()``); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkvq.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, st, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
        lp = ctypes.POINTER(KvqLayout)
        wp = ctypes.POINTER(KvqWindow)
        tp = ctypes.POINTER(KvqOptrTrace)
        sigs = {
            "kvq_last_error": ([], ctypes.c_char_p),
            "kvq_pool_bytes": ([lp], sz),
            "kvq_device_check": ([vp], st),
            "kvq_key_mean": ([i, i, vp, i, vp, vp], st),
            "kvq_rotate_heads": ([i, i, i, vp, KvqRot, vp, vp], st),
            "kvq_quantize_append": ([lp, i, i, vp, vp, i, vp, vp, vp, KvqRot, KvqRot, vp, f, f, vp, vp], st),
            "kvq_decode_workspace_size": ([lp, i, i, i, ctypes.POINTER(sz)], st),
            "kvq_decode_attention": ([lp, i, vp, i, vp, i, vp, KvqRot, vp, i, vp, sz, vp, vp], st),
            "kvq_decode_attention_noalloc": ([lp, i, vp, i, vp, i, vp, KvqRot, vp, i, vp, vp], st),
            "kvq_decode_step": ([lp, i, vp, vp, vp, i, vp, i, vp, KvqRot, KvqRot, vp, f, f, vp, i, vp, sz, vp, vp],
                                st),
            "kvq_window_append": ([lp, i, i, vp, vp, i, vp, vp, vp, wp, vp], st),
            "kvq_decode_step_win": ([lp, i, vp, vp, vp, i, vp, i, vp, KvqRot, KvqRot, vp, vp, f, f, vp, wp, i, vp, sz,
                                     vp, vp], st),
            "kvq_decode_workspace_size_win": ([lp, i, i, i, wp, ctypes.POINTER(sz)], st),
            "kvq_decode_attention_win": ([lp, i, vp, i, vp, i, vp, KvqRot, KvqRot, vp, wp, i, vp, sz, vp, vp], st),
            "kvq_plan_workspace_size": ([i, ctypes.POINTER(sz)], st),
            "kvq_plan_pages": ([lp, i, vp, vp, vp, vp, vp, vp, i, vp, vp, vp, sz, vp], st),
            "kvq_query_block_workspace_size": ([lp, i, i, i, i, ctypes.POINTER(sz)], st),
            "kvq_tree_attention": ([lp, i, i, vp, i, vp, i, vp, vp, i, vp, KvqRot, vp, vp, sz, vp, vp], st),
            "kvq_cross_attention": ([lp, i, i, vp, i, vp, i, vp, i, vp, KvqRot, vp, vp, sz, vp, vp], st),
            "kvq_tree_commit": ([lp, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp], st),
            "kvq_norm_rope": ([i, i, i, vp, i, ctypes.c_int64, vp, ctypes.POINTER(KvqRope), vp, vp, f, vp, vp, vp, vp],
                              st),
            "kvq_read_cache": ([lp, i, i, vp, vp, vp, KvqRot, KvqRot, vp, vp, vp, vp, i, vp], st),
            "kvq_decode_attention_score": ([lp, i, vp, i, vp, i, vp, KvqRot, vp, ctypes.POINTER(KvqScore), vp, sz, vp, vp],
                                           st),
            "kvq_chunk_attention_score": ([lp, i, i, vp, i, vp, i, vp, i, vp, KvqRot, vp, ctypes.POINTER(KvqScore), vp, sz,
                                           vp, vp], st),
            "kvq_fold_wo": ([i, i, i, vp, i, KvqRot, vp, i, vp], st),
            "kvq_out_proj": ([i, i, i, vp, vp, i, vp, vp], st),
            "kvq_wo_packed_bytes": ([i, i, ctypes.POINTER(sz)], st),
            "kvq_pack_wo": ([i, i, vp, vp, vp], st),
            "kvq_out_proj_packed": ([i, i, i, vp, vp, vp, vp], st),
            "kvq_calib_workspace_size": ([i, i, i, i, i, ctypes.POINTER(sz)], st),
            "kvq_report_workspace_size": ([i, i, i, i, ctypes.POINTER(sz)], st),
            "kvq_head_error_report": ([i, i, i, i, i, vp, vp, vp, i, vp, i, KvqRot, KvqRot, vp, f, f, vp, vp, sz,
                                       vp], st),
            "kvq_calib_nmse": ([i, i, i, i, i, vp, vp, vp, i, vp, i, i, ctypes.POINTER(KvqRot), i,
                                ctypes.POINTER(ctypes.c_float), vp, i, vp, vp, vp, sz, vp], st),
            "kvq_optr_workspace_size": ([i, i, i, i, i, ctypes.POINTER(sz)], st),
            "kvq_optr_loss_grad": ([i, tp, i, i, vp, vp, vp, vp, vp, f, f, f, vp, vp, vp, sz, vp], st),
            "kvq_optr_calibrate_head": ([tp, tp, i, i, vp, vp, vp, vp, f, f, f, i, f, i, vp, vp, vp, vp, vp, sz,
                                         vp], st),
        }
        for name, (argtypes, restype) in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = L
    return _lib


EXPORTED = ("kvq_last_error", "kvq_pool_bytes", "kvq_device_check", "kvq_key_mean", "kvq_rotate_heads",
            "kvq_quantize_append", "kvq_decode_workspace_size", "kvq_decode_attention",
            "kvq_decode_attention_noalloc", "kvq_decode_step", "kvq_decode_step_win", "kvq_window_append", "kvq_decode_workspace_size_win",
            "kvq_decode_attention_win", "kvq_plan_workspace_size", "kvq_plan_pages", "kvq_query_block_workspace_size",
            "kvq_tree_attention", "kvq_cross_attention", "kvq_tree_commit", "kvq_norm_rope", "kvq_read_cache",
            "kvq_decode_attention_score",
            "kvq_chunk_attention_score", "kvq_fold_wo",
            "kvq_out_proj", "kvq_wo_packed_bytes", "kvq_pack_wo", "kvq_out_proj_packed", "kvq_calib_workspace_size", "kvq_calib_nmse", "kvq_report_workspace_size",
            "kvq_head_error_report", "kvq_optr_workspace_size", "kvq_optr_loss_grad", "kvq_optr_calibrate_head")


def _check(status: int) -> None:
    if status != KVQ_OK:
        raise KvqError(status, lib().kvq_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return KVQ_F32
    if t.dtype == torch.bfloat16:
        return KVQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _contig(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class DeviceRot:
    """A rotation spec with its device tensors kept alive."""

    def __init__(self, kind: str, signs=None, dense=None):
        self.kind = kind
        self.signs = signs
        self.dense = dense

    @classmethod
    def from_spec(cls, rot, device="cuda"):
        import torch
        s = torch.as_tensor(rot.signs, dtype=torch.float32, device=device).contiguous() if rot.signs is not None else None
        d = torch.as_tensor(rot.dense, dtype=torch.float32, device=device).contiguous() if rot.dense is not None else None
        return cls(rot.kind, s, d)

    @property
    def c(self) -> KvqRot:
        return KvqRot(ROT_KIND[self.kind], _ptr(self.signs), _ptr(self.dense))


def make_layout(page_tokens: int, n_kv_heads: int, n_q_heads: int, num_blocks: int,
                max_blocks_per_seq: int) -> KvqLayout:
    return KvqLayout(HEAD_DIM, page_tokens, n_kv_heads, n_q_heads, num_blocks, max_blocks_per_seq)


def kvq_pool_bytes(layout: KvqLayout) -> int:
    return int(lib().kvq_pool_bytes(ctypes.byref(layout)))


def kvq_device_check(stream=None) -> None:
    _check(lib().kvq_device_check(_stream(stream)))


def kvq_key_mean(k, mu, stream=None) -> None:
    n_tok, h, d = k.shape
    _check(lib().kvq_key_mean(n_tok, h, _ptr(_contig(k, "k")), _dtype_code(k), _ptr(mu), _stream(stream)))


def kvq_rotate_heads(x, rot: DeviceRot, y, heads_per_rot: int = 1, stream=None) -> None:
    n_rows, n_heads, _ = x.shape
    _check(lib().kvq_rotate_heads(n_rows, n_heads, heads_per_rot, _ptr(_contig(x, "x")), rot.c, _ptr(y),
                                  _stream(stream)))


def kvq_quantize_append(layout: KvqLayout, k, v, cu_new, start_pos, block_table, rot_k: DeviceRot,
                        rot_v: DeviceRot, mu_rot_k, clip_k: float, clip_v: float, pool, stream=None) -> None:
    n_new = k.shape[0]
    n_seqs = start_pos.shape[0]
    _check(lib().kvq_quantize_append(ctypes.byref(layout), n_seqs, n_new, _ptr(_contig(k, "k")),
                                     _ptr(_contig(v, "v")), _dtype_code(k), _ptr(cu_new), _ptr(start_pos),
                                     _ptr(block_table), rot_k.c, rot_v.c, _ptr(mu_rot_k), clip_k, clip_v,
                                     _ptr(pool), _stream(stream)))


def kvq_decode_workspace_size(layout: KvqLayout, n_seqs: int, max_seq_len: int, n_splits: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_decode_workspace_size(ctypes.byref(layout), n_seqs, max_seq_len, n_splits, ctypes.byref(out)))
    return int(out.value)


def kvq_decode_attention(layout: KvqLayout, q, seq_lens, max_seq_len: int, block_table, rot_k: DeviceRot,
                         pool, workspace, o_rot, n_splits: int = 0, stream=None) -> None:
    n_seqs = q.shape[0]
    _check(lib().kvq_decode_attention(ctypes.byref(layout), n_seqs, _ptr(_contig(q, "q")), _dtype_code(q),
                                      _ptr(seq_lens), max_seq_len, _ptr(block_table), rot_k.c, _ptr(pool),
                                      n_splits, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _ptr(o_rot), _stream(stream)))


def kvq_decode_attention_noalloc(layout: KvqLayout, q, seq_lens, max_seq_len: int, block_table,
                                 rot_k: DeviceRot, pool, o_rot, n_splits: int = 0, stream=None) -> None:
    """Decode attention without a caller-provided workspace (for callers that may
    not allocate device memory); the split partials live in a fixed library buffer."""
    n_seqs = q.shape[0]
    _check(lib().kvq_decode_attention_noalloc(ctypes.byref(layout), n_seqs, _ptr(_contig(q, "q")), _dtype_code(q),
                                              _ptr(seq_lens), max_seq_len, _ptr(block_table), rot_k.c, _ptr(pool),
                                              n_splits, _ptr(o_rot), _stream(stream)))


def kvq_decode_step(layout: KvqLayout, q, k_new, v_new, seq_lens, max_seq_len: int, block_table,
                    rot_k: DeviceRot, rot_v: DeviceRot, mu_rot_k, clip_k: float, clip_v: float, pool, workspace,
                    o_rot, n_splits: int = 0, stream=None) -> None:
    """One decode step: each sequence's new token (k_new[b], v_new[b]) is appended at
    position seq_lens[b] - 1 and the decode attention reads it, in one call."""
    n_seqs = q.shape[0]
    if k_new.dtype != q.dtype or v_new.dtype != q.dtype:
        raise TypeError("q, k_new and v_new must share a dtype")
    _check(lib().kvq_decode_step(ctypes.byref(layout), n_seqs, _ptr(_contig(q, "q")), _ptr(_contig(k_new, "k_new")),
                                 _ptr(_contig(v_new, "v_new")), _dtype_code(q), _ptr(seq_lens), max_seq_len,
                                 _ptr(block_table), rot_k.c, rot_v.c, _ptr(mu_rot_k), clip_k, clip_v, _ptr(pool),
                                 n_splits, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(o_rot), _stream(stream)))


class Window:
    """BF16 sink / recent window sizes and the caller's record buffer (see kvq_window)."""

    def __init__(self, sink_tokens: int, recent_tokens: int, buf=None):
        self.sink_tokens = sink_tokens
        self.recent_tokens = recent_tokens
        self.buf = buf

    @staticmethod
    def buffer_bytes(n_seqs: int, n_kv_heads: int, sink_tokens: int, recent_tokens: int) -> int:
        return n_seqs * n_kv_heads * (sink_tokens + recent_tokens) * 512

    @property
    def c(self) -> KvqWindow:
        return KvqWindow(self.sink_tokens, self.recent_tokens, _ptr(self.buf))


def _win_ref(win):
    return None if win is None else ctypes.byref(win.c)


def kvq_window_append(layout: KvqLayout, k, v, cu_new, start_pos, mu_k, win: Window, stream=None) -> None:
    _check(lib().kvq_window_append(ctypes.byref(layout), start_pos.shape[0], k.shape[0], _ptr(_contig(k, "k")),
                                   _ptr(_contig(v, "v")), _dtype_code(k), _ptr(cu_new), _ptr(start_pos),
                                   _ptr(mu_k), _win_ref(win), _stream(stream)))


def kvq_decode_workspace_size_win(layout: KvqLayout, n_seqs: int, max_seq_len: int, win: Window | None,
                                  n_splits: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_decode_workspace_size_win(ctypes.byref(layout), n_seqs, max_seq_len, n_splits, _win_ref(win),
                                               ctypes.byref(out)))
    return int(out.value)


def kvq_decode_step_win(layout: KvqLayout, q, k_new, v_new, seq_lens, max_seq_len: int, block_table,
                        rot_k: DeviceRot, rot_v: DeviceRot, mu_rot_k, mu_k, clip_k: float, clip_v: float, pool,
                        win: Window | None, workspace, o_rot, n_splits: int = 0, stream=None) -> None:
    """kvq_decode_step with BF16 windows: the new token is also copied into its window
    slot (key centred by the unrotated mean mu_k) before the windowed decode reads it."""
    n_seqs = q.shape[0]
    if k_new.dtype != q.dtype or v_new.dtype != q.dtype:
        raise TypeError("q, k_new and v_new must share a dtype")
    _check(lib().kvq_decode_step_win(ctypes.byref(layout), n_seqs, _ptr(_contig(q, "q")), _ptr(_contig(k_new, "k_new")),
                                     _ptr(_contig(v_new, "v_new")), _dtype_code(q), _ptr(seq_lens), max_seq_len,
                                     _ptr(block_table), rot_k.c, rot_v.c, _ptr(mu_rot_k), _ptr(mu_k), clip_k, clip_v,
                                     _ptr(pool), _win_ref(win), n_splits, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(o_rot), _stream(stream)))


def kvq_decode_attention_win(layout: KvqLayout, q, seq_lens, max_seq_len: int, block_table, rot_k: DeviceRot,
                             rot_v: DeviceRot, pool, win: Window | None, workspace, o_rot, n_splits: int = 0,
                             stream=None) -> None:
    n_seqs = q.shape[0]
    _check(lib().kvq_decode_attention_win(ctypes.byref(layout), n_seqs, _ptr(_contig(q, "q")), _dtype_code(q),
                                          _ptr(seq_lens), max_seq_len, _ptr(block_table), rot_k.c, rot_v.c,
                                          _ptr(pool),
                                          _win_ref(win), n_splits, _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(o_rot),
                                          _stream(stream)))


# ---- speculative decoding and cross attention over the cache ----
def _device_and_stream(stream):
    """The current CUDA device (-2 without one: every tensor is then refused) and the raw stream of a call on it."""
    import torch
    try:
        dev = torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2, None
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, getattr(stream, "cuda_stream", stream)


def _dense(t, name: str, dtype, shape, dev: int):
    """The address of a dense tensor of this type and shape (None: any) on the current device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _pool(layout: KvqLayout, pool, dev: int):
    """The cache pool: uint8 of any shape, no smaller than the layout's."""
    import torch
    need = layout.num_blocks * layout.n_kv_heads * layout.page_tokens * 72
    if pool.numel() < need:
        raise ValueError(f"pool has {pool.numel()} bytes, the layout needs {need}")
    return _dense(pool, "pool", torch.uint8, None, dev)


def _rot(layout: KvqLayout, rot: DeviceRot, dev: int, of: str = "rot_k") -> KvqRot:
    """A rotation of (at least) every KV head, which the kernels index as dense fp32."""
    import torch

    def of_heads(t, name, *each):
        if t is None:
            raise ValueError(f"{name} is missing")
        if t.numel() < layout.n_kv_heads * math.prod(each):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, the layout needs {(layout.n_kv_heads, *each)}")
        return _dense(t, name, torch.float32, None, dev)

    signs = of_heads(rot.signs, f"{of}.signs", HEAD_DIM) if rot.kind == "signed_hadamard" else None
    dense = of_heads(rot.dense, f"{of}.dense", HEAD_DIM, HEAD_DIM) if rot.kind == "dense" else None
    return KvqRot(ROT_KIND[rot.kind], signs, dense)


def kvq_plan_workspace_size(n_seqs: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_plan_workspace_size(n_seqs, ctypes.byref(out)))
    return int(out.value)


def kvq_plan_pages(layout: KvqLayout, old_lens, new_lens, block_table, free_ring, ring_in, ring_out, cu_new, slot_map,
                   workspace, stream=None) -> None:
    """Takes and gives back pages for requests going from old_lens to new_lens tokens: block_table and the ring of
    free pages in place (counters (head, tail): ring_in -> ring_out, int64 [2]); cu_new int32 [n + 1] and slot_map
    int64 [capacity for new tokens] are written.  See include/kvq.h."""
    import torch
    i32, i64 = torch.int32, torch.int64
    dev, raw = _device_and_stream(stream)
    n, room = old_lens.shape[0], slot_map.shape[0]
    _check(lib().kvq_plan_pages(
        ctypes.byref(layout), n, _dense(old_lens, "old_lens", i32, (n,), dev),
        _dense(new_lens, "new_lens", i32, (n,), dev),
        _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev),
        _dense(free_ring, "free_ring", i32, (layout.num_blocks,), dev), _dense(ring_in, "ring_in", i64, (2,), dev),
        _dense(ring_out, "ring_out", i64, (2,), dev), room, _dense(cu_new, "cu_new", i32, (n + 1,), dev),
        _dense(slot_map, "slot_map", i64, (room,), dev), _dense(workspace, "workspace", torch.uint8, None, dev),
        workspace.numel(), raw))


def kvq_query_block_workspace_size(layout: KvqLayout, n_seqs: int, n_q_total: int, max_q: int, max_seq_len: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_query_block_workspace_size(ctypes.byref(layout), n_seqs, n_q_total, max_q, max_seq_len,
                                                ctypes.byref(out)))
    return int(out.value)


def kvq_tree_attention(layout: KvqLayout, q, cu_q, max_q: int, parents, seq_lens, max_seq_len: int, block_table,
                       rot_k: DeviceRot, pool, workspace, o_rot, stream=None) -> None:
    """Attention of every sequence's drafts (q [n_q_total, H_q, 128], rows cu_q[b] .. cu_q[b + 1]) over the cache and
    over their own ancestors; the drafts are the last of the seq_lens[b] cached tokens.  parents: int32 [n_q_total]
    (index within the sequence, -1: follows the cache), or None for a chain (a causal chunk).  o_rot: fp32 like q."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    n, total = seq_lens.shape[0], q.shape[0]
    rows, rot = (total, layout.n_q_heads, HEAD_DIM), _rot(layout, rot_k, dev)
    _check(lib().kvq_tree_attention(
        ctypes.byref(layout), n, total, _dense(q, "q", q.dtype, rows, dev), _dtype_code(q),
        _dense(cu_q, "cu_q", i32, (n + 1,), dev), max_q,
        None if parents is None else _dense(parents, "parents", i32, (total,), dev),
        _dense(seq_lens, "seq_lens", i32, (n,), dev), max_seq_len,
        _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev), rot,
        _pool(layout, pool, dev), _dense(workspace, "workspace", torch.uint8, None, dev), workspace.numel(),
        _dense(o_rot, "o_rot", torch.float32, rows, dev), raw))


def kvq_cross_attention(layout: KvqLayout, q, cu_q, max_q: int, state_lens, max_state_len: int, block_table,
                        rot_k: DeviceRot, pool, workspace, o_rot, stream=None) -> None:
    """Attention of query blocks over all cached states of their sequence (an encoder's), without a mask."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    n, total = state_lens.shape[0], q.shape[0]
    rows, rot = (total, layout.n_q_heads, HEAD_DIM), _rot(layout, rot_k, dev)
    _check(lib().kvq_cross_attention(
        ctypes.byref(layout), n, total, _dense(q, "q", q.dtype, rows, dev), _dtype_code(q),
        _dense(cu_q, "cu_q", i32, (n + 1,), dev), max_q, _dense(state_lens, "state_lens", i32, (n,), dev),
        max_state_len, _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev), rot,
        _pool(layout, pool, dev), _dense(workspace, "workspace", torch.uint8, None, dev), workspace.numel(),
        _dense(o_rot, "o_rot", torch.float32, rows, dev), raw))


def kvq_tree_commit(layout: KvqLayout, cu_q, accepted, n_accepted, slot_map, seq_lens, new_lens, pool,
                    stream=None) -> None:
    """Moves the accepted drafts' records (accepted int32 [n, max_accept], increasing; n_accepted int32 [n]) to the
    places of the first drafts and writes new_lens = seq_lens - drafts + accepted."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    n, total = seq_lens.shape[0], slot_map.shape[0]
    depth = accepted.shape[1]
    _check(lib().kvq_tree_commit(
        ctypes.byref(layout), n, total, depth, _dense(cu_q, "cu_q", i32, (n + 1,), dev),
        _dense(accepted, "accepted", i32, (n, depth), dev), _dense(n_accepted, "n_accepted", i32, (n,), dev),
        _dense(slot_map, "slot_map", torch.int64, (total,), dev), _dense(seq_lens, "seq_lens", i32, (n,), dev),
        _dense(new_lens, "new_lens", i32, (n,), dev), _pool(layout, pool, dev), raw))


# ---- around the cache ----
class Rope:
    """A position rotation (see kvq_rope): inv_freq, radians a position for each pair of the first 2 len(inv_freq)
    channels; axis, the axis of each pair's position (None: axis 0); interleaved: pairs (2i, 2i + 1)."""

    def __init__(self, inv_freq, axis=None, n_axes: int = 1, interleaved: bool = False):
        n = len(inv_freq)
        if axis is not None and len(axis) != n:
            raise ValueError(f"axis has {len(axis)} entries, inv_freq {n}")
        self.n_axes = n_axes
        self.rotary_dim = 2 * n
        self._inv_freq = (ctypes.c_double * n)(*[float(x) for x in inv_freq])
        self._axis = None if axis is None else (ctypes.c_int32 * n)(*[int(x) for x in axis])
        self.c = KvqRope(2 * n, int(interleaved), n_axes, ctypes.addressof(self._inv_freq),
                         None if axis is None else ctypes.addressof(self._axis))


def kvq_norm_rope(qkv, positions, rope: Rope, w_q, w_k, eps: float, q, k, v, stream=None) -> None:
    """qkv [n_tok, (H_q + 2 H_kv) * 128] (rows may be strided) into q [n_tok, H_q, 128], k and v [n_tok, H_kv, 128]:
    heads normed by w_q, w_k (fp32 [128], None: not normed) and turned by positions (int32 [n_axes, n_tok]; None without
    a rotation); v is copied (None: not).  See include/kvq.h."""
    import torch
    dev, raw = _device_and_stream(stream)
    n, h_q, h_kv = qkv.shape[0], q.shape[1], k.shape[1]
    width = (h_q + 2 * h_kv) * HEAD_DIM
    if qkv.dim() != 2 or qkv.shape[1] != width:
        raise ValueError(f"qkv has shape {tuple(qkv.shape)}, expected {(n, width)}")
    if qkv.get_device() != dev:
        raise ValueError(f"qkv is on {qkv.device}, not on the current CUDA device")
    if qkv.stride(1) != 1 and n * width > 0:
        raise ValueError("the rows of qkv must be contiguous")
    stride = qkv.stride(0) if n > 1 else width  # a single row's is not used
    if stride < width:
        raise ValueError(f"the rows of qkv overlap (stride {stride}, {width} elements)")
    f32 = torch.float32
    pos = None
    if rope.rotary_dim:
        if positions is None:
            raise ValueError("positions are missing")
        pos = _dense(positions, "positions", torch.int32, (rope.n_axes, n), dev)
    _check(lib().kvq_norm_rope(
        n, h_q, h_kv, qkv.data_ptr(), _dtype_code(qkv), stride, pos, ctypes.byref(rope.c),
        None if w_q is None else _dense(w_q, "w_q", f32, (HEAD_DIM,), dev),
        None if w_k is None else _dense(w_k, "w_k", f32, (HEAD_DIM,), dev), eps,
        _dense(q, "q", qkv.dtype, (n, h_q, HEAD_DIM), dev), _dense(k, "k", qkv.dtype, (n, h_kv, HEAD_DIM), dev),
        None if v is None else _dense(v, "v", qkv.dtype, (n, h_kv, HEAD_DIM), dev), raw))


def kvq_read_cache(layout: KvqLayout, cu_tok, start_pos, block_table, rot_k: DeviceRot, rot_v: DeviceRot, mu_k, pool, k,
                   v, stream=None) -> None:
    """Cached tokens back as keys and values: row t of sequence b (cu_tok[b] <= t < cu_tok[b + 1]) is position
    start_pos[b] + t - cu_tok[b].  k, v: [n, H_kv, 128] bf16 or fp32, either may be None; mu_k fp32 [H_kv, 128] or None."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    one = k if k is not None else v
    if one is None:
        raise ValueError("k and v are both None")
    n, total = start_pos.shape[0], one.shape[0]
    rows = (total, layout.n_kv_heads, HEAD_DIM)
    rk = KvqRot(0, None, None) if k is None else _rot(layout, rot_k, dev)
    rv = KvqRot(0, None, None) if v is None else _rot(layout, rot_v, dev, "rot_v")
    _check(lib().kvq_read_cache(
        ctypes.byref(layout), n, total, _dense(cu_tok, "cu_tok", i32, (n + 1,), dev),
        _dense(start_pos, "start_pos", i32, (n,), dev),
        _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev),
        rk, rv, None if mu_k is None else _dense(mu_k, "mu_k", torch.float32, (layout.n_kv_heads, HEAD_DIM), dev),
        _pool(layout, pool, dev), None if k is None else _dense(k, "k", one.dtype, rows, dev),
        None if v is None else _dense(v, "v", one.dtype, rows, dev), _dtype_code(one), raw))


class Score:
    """What a layer does to its scores (see kvq_score): cap (0: none), slopes (fp32 [H_q] on the device, or None), window
    (tokens, 0: no limit), prefix_lens (int32 [n_seqs] on the device, or None)."""

    def __init__(self, cap: float = 0.0, slopes=None, window: int = 0, prefix_lens=None):
        if cap and not ctypes.c_float(cap).value:
            raise ValueError(f"score cap {cap} is 0 in fp32, which means none")
        if not -2 ** 31 <= window < 2 ** 31:  # negative ones are refused by the call
            raise ValueError(f"score window {window} is no int32")
        self.cap, self.slopes, self.window, self.prefix_lens = cap, slopes, window, prefix_lens

    def c(self, layout: KvqLayout, n_seqs: int, dev: int) -> KvqScore:
        import torch
        slopes = None if self.slopes is None else _dense(self.slopes, "score slopes", torch.float32, (layout.n_q_heads,), dev)
        prefix = None if self.prefix_lens is None else _dense(self.prefix_lens, "score prefix_lens", torch.int32, (n_seqs,),
                                                              dev)
        return KvqScore(self.cap, slopes, self.window, prefix)


def kvq_decode_attention_score(layout: KvqLayout, q, seq_lens, max_seq_len: int, block_table, rot_k: DeviceRot, pool,
                               score: Score, workspace, o_rot, stream=None) -> None:
    """kvq_decode_attention with capped scores, distance bias, window and prefix (workspace of
    kvq_decode_workspace_size)."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    n = seq_lens.shape[0]
    rows, rot = (n, layout.n_q_heads, HEAD_DIM), _rot(layout, rot_k, dev)
    _check(lib().kvq_decode_attention_score(
        ctypes.byref(layout), n, _dense(q, "q", q.dtype, rows, dev), _dtype_code(q),
        _dense(seq_lens, "seq_lens", i32, (n,), dev), max_seq_len,
        _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev), rot, _pool(layout, pool, dev),
        ctypes.byref(score.c(layout, n, dev)), _dense(workspace, "workspace", torch.uint8, None, dev),
        workspace.numel(), _dense(o_rot, "o_rot", torch.float32, rows, dev), raw))


def kvq_chunk_attention_score(layout: KvqLayout, q, cu_q, max_q: int, seq_lens, max_seq_len: int, block_table,
                              rot_k: DeviceRot, pool, score: Score, workspace, o_rot, stream=None) -> None:
    """kvq_tree_attention of causal chunks (the last cu_q[b + 1] - cu_q[b] of seq_lens[b] cached tokens) with capped
    scores, distance bias, window and prefix (workspace of kvq_query_block_workspace_size)."""
    import torch
    i32 = torch.int32
    dev, raw = _device_and_stream(stream)
    n, total = seq_lens.shape[0], q.shape[0]
    rows, rot = (total, layout.n_q_heads, HEAD_DIM), _rot(layout, rot_k, dev)
    _check(lib().kvq_chunk_attention_score(
        ctypes.byref(layout), n, total, _dense(q, "q", q.dtype, rows, dev), _dtype_code(q),
        _dense(cu_q, "cu_q", i32, (n + 1,), dev), max_q, _dense(seq_lens, "seq_lens", i32, (n,), dev), max_seq_len,
        _dense(block_table, "block_table", i32, (n, layout.max_blocks_per_seq), dev), rot, _pool(layout, pool, dev),
        ctypes.byref(score.c(layout, n, dev)), _dense(workspace, "workspace", torch.uint8, None, dev),
        workspace.numel(), _dense(o_rot, "o_rot", torch.float32, rows, dev), raw))


def kvq_fold_wo(w_o, n_q_heads: int, n_kv_heads: int, rot_v: DeviceRot, w_folded, stream=None) -> None:
    d_model = w_o.shape[0]
    _check(lib().kvq_fold_wo(d_model, n_q_heads, n_kv_heads, _ptr(_contig(w_o, "w_o")), _dtype_code(w_o),
                             rot_v.c, _ptr(w_folded), _dtype_code(w_folded), _stream(stream)))


def kvq_out_proj(x, w, y, stream=None) -> None:
    n_rows, k_dim = x.shape[0], x.numel() // max(1, x.shape[0])
    d_model = w.shape[0]
    _check(lib().kvq_out_proj(n_rows, d_model, k_dim, _ptr(_contig(x, "x")), _ptr(_contig(w, "w")),
                              _dtype_code(w), _ptr(y), _stream(stream)))


def kvq_calib_workspace_size(n_tok: int, n_qpos: int, n_kv_heads: int, gqa: int, joint: bool) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_calib_workspace_size(n_tok, n_qpos, n_kv_heads, gqa, int(joint), ctypes.byref(out)))
    return int(out.value)


def kvq_calib_nmse(q, k, v, w_o, cands, clips, mu, joint: bool, nmse, ref, workspace, stream=None) -> None:
    n_qpos, hq, _ = q.shape
    n_tok, hkv, _ = k.shape
    gqa = hq // hkv
    d_model = w_o.shape[0]
    rot_arr = (KvqRot * len(cands))(*[c.c for c in cands])
    clip_arr = (ctypes.c_float * len(clips))(*[float(c) for c in clips])
    _check(lib().kvq_calib_nmse(n_tok, n_qpos, hkv, gqa, d_model, _ptr(_contig(q, "q")), _ptr(_contig(k, "k")),
                                _ptr(_contig(v, "v")), _dtype_code(k), _ptr(_contig(w_o, "w_o")), _dtype_code(w_o),
                                len(cands), rot_arr, len(clips), clip_arr, _ptr(mu), int(joint), _ptr(nmse),
                                _ptr(ref), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)))


def kvq_report_workspace_size(n_tok: int, n_qpos: int, n_kv_heads: int, gqa: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_report_workspace_size(n_tok, n_qpos, n_kv_heads, gqa, ctypes.byref(out)))
    return int(out.value)


def kvq_head_error_report(q, k, v, w_o, rot_k: DeviceRot, rot_v: DeviceRot, mu, clip_k: float, clip_v: float, out,
                          workspace, stream=None) -> None:
    """out: float64 [5, H_kv] (E, E_key, E_val, E_naive, Y per KV head; see include/kvq.h)."""
    n_qpos, hq, _ = q.shape
    n_tok, hkv, _ = k.shape
    _check(lib().kvq_head_error_report(n_tok, n_qpos, hkv, hq // hkv, w_o.shape[0], _ptr(_contig(q, "q")),
                                       _ptr(_contig(k, "k")), _ptr(_contig(v, "v")), _dtype_code(k),
                                       _ptr(_contig(w_o, "w_o")), _dtype_code(w_o), rot_k.c, rot_v.c, _ptr(mu),
                                       float(clip_k), float(clip_v), _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


# ---- OptR gradient calibration of one KV head ----
KVQ_OPTR_KEYS = 0
KVQ_OPTR_VALUES = 1


def _trace(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        _contig(t, name)
    return KvqOptrTrace(_ptr(q), _ptr(k), _ptr(v), k.shape[0], q.shape[0])


def kvq_optr_workspace_size(n_tok: int, n_qpos: int, gqa: int, n_tok_heldout: int = 0, n_qpos_heldout: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_optr_workspace_size(n_tok, n_qpos, n_tok_heldout, n_qpos_heldout, gqa, ctypes.byref(out)))
    return int(out.value)


def kvq_optr_loss_grad(phase: int, q, k, v, w_o, mu, r0, a, r_k_sel, clip_k: float, clip_v: float, lambda_k: float,
                       loss, grad, workspace, stream=None) -> None:
    """One OptR objective (keys: Eq. 14; values: Eq. 16) and dL/dA at R = r0 exp(a - a^T).
    q [n_qpos][gqa][128], k, v [n_tok][128], w_o [d_model][gqa*128], mu [128] (fp32);
    r0, a, r_k_sel, grad: fp64 [128][128]; loss: fp64 [1]."""
    tr = _trace(q, k, v)
    _check(lib().kvq_optr_loss_grad(phase, ctypes.byref(tr), q.shape[1], w_o.shape[0], _ptr(_contig(w_o, "w_o")),
                                    _ptr(mu), _ptr(r0), _ptr(a), _ptr(r_k_sel), clip_k, clip_v, lambda_k, _ptr(loss),
                                    _ptr(grad), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)))


def kvq_optr_calibrate_head(train, heldout, w_o, mu, r_k0, r_v0, clip_k: float, clip_v: float, lambda_k: float,
                            steps: int, lr: float, every: int, r_k, r_v, loss_k, loss_v, workspace,
                            stream=None) -> None:
    """Algorithm 1 for one KV head.  train / heldout: (q, k, v) tuples of fp32 tensors (heldout may be None)."""
    tr = _trace(*train)
    ho = _trace(*heldout) if heldout is not None else None
    q = train[0]
    _check(lib().kvq_optr_calibrate_head(ctypes.byref(tr), ctypes.byref(ho) if ho is not None else None, q.shape[1],
                                         w_o.shape[0], _ptr(_contig(w_o, "w_o")), _ptr(mu), _ptr(r_k0), _ptr(r_v0),
                                         clip_k, clip_v, lambda_k, steps, lr, every, _ptr(r_k), _ptr(r_v),
                                         _ptr(loss_k), _ptr(loss_v), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))


# ---- the folded W_O in the projection's box order ----
def kvq_wo_packed_bytes(d_model: int, k_dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().kvq_wo_packed_bytes(d_model, k_dim, ctypes.byref(out)))
    return int(out.value)


def kvq_pack_wo(w, w_packed, stream=None) -> None:
    """w: bf16 [d_model][k_dim] (e.g. kvq_fold_wo's output); w_packed: kvq_wo_packed_bytes bytes."""
    d_model, k_dim = w.shape
    _check(lib().kvq_pack_wo(d_model, k_dim, _ptr(_contig(w, "w")), _ptr(w_packed), _stream(stream)))


def kvq_out_proj_packed(x, w_packed, y, d_model: int, stream=None) -> None:
    n_rows, k_dim = x.shape
    _check(lib().kvq_out_proj_packed(n_rows, d_model, k_dim, _ptr(_contig(x, "x")), _ptr(w_packed), _ptr(y),
                                     _stream(stream)))
