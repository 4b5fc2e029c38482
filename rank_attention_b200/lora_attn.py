"""Python binding of liblora_attn.so (ctypes; argument marshalling only).

The names match the C ABI in include/lora_attn.h.  Tensors are torch CUDA
tensors; the binding passes their data pointers, sizes and strides, and the
current torch stream.  Every step of the computation runs in the library's
CUDA kernels.  If the compiled library is missing, importing this module
raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "liblora_attn.so")

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CAPACITY = 0, 1, 2, 3
LA_ERR_WORKSPACE, LA_ERR_CUDA, LA_ERR_DEVICE_CHECK, LA_ERR_SCRATCH_LIMIT = 4, 5, 6, 7
LA_STATIC_SCRATCH_BYTES = 4 << 20
LA_F32, LA_BF16 = 0, 1
LA_VALUE_REORDERED, LA_VALUE_REORDERED_GENERIC, LA_VALUE_PER_TILE, LA_VALUE_PER_TILE_GENERIC = 0, 1, 2, 3
LA_DEV_KV_LEN, LA_DEV_PIPE_WAIT, LA_DEV_MERGE_WAIT, LA_DEV_TREE, LA_DEV_SEGMENT = 1, 2, 4, 8, 16
LA_TREE_MAX_NODES = 64

EXPORTED = ("la_status_string", "lr_cache_append", "lora_attn_prefill", "lora_attn_decode",
            "lora_attn_decode_workspace_bytes", "la_device_check",
            "lora_attn_decode_static_scratch", "lora_materialize_agent_kv",
            "lr_cache_append_agents", "lora_query_expand", "lora_output_delta",
            "la_device_check_word", "lora_decode_step_host", "lora_attn_decode_step",
            "lora_attn_decode_combine", "lora_attn_tree", "lora_qk_norm_rope",
            "lora_grouped_delta")


class LoraAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class AttnArgs(ctypes.Structure):
    """Mirror of la_attn_args."""

    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_agents", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("r", ctypes.c_int32),
        ("lora_scale", ctypes.c_float), ("softmax_scale", ctypes.c_float),
        ("rope_base", ctypes.c_double),
        ("L_max", ctypes.c_int64),
        ("k_base", ctypes.c_void_p), ("v_base", ctypes.c_void_p),
        ("kv_seq_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64),
        ("kv_tok_stride", ctypes.c_int64),
        ("lr_cache", ctypes.c_void_p), ("lr_seq_stride", ctypes.c_int64),
        ("B_k", ctypes.c_void_p), ("B_v", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p),
        ("max_kv_len", ctypes.c_int64),
        ("q_pos0", ctypes.c_int64),
        ("n_q_tokens", ctypes.c_int32),
        ("io_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("lr_agent_stride", ctypes.c_int64),
        ("value_path", ctypes.c_int32),
        ("key_pos0", ctypes.c_int64),
        ("row_stats", ctypes.c_void_p),
    ]


class TreeArgs(ctypes.Structure):
    """Mirror of la_tree_args."""

    _fields_ = [("parent", ctypes.c_void_p), ("tree_len", ctypes.c_void_p),
                ("n_trees", ctypes.c_int32)]


class QkArgs(ctypes.Structure):
    """Mirror of la_qk_args."""

    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_agents", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("eps", ctypes.c_float), ("rope_base", ctypes.c_double),
        ("q", ctypes.c_void_p), ("q_seq_stride", ctypes.c_int64),
        ("q_agent_stride", ctypes.c_int64), ("q_tok_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("kv_in_seq_stride", ctypes.c_int64), ("kv_in_tree_stride", ctypes.c_int64),
        ("kv_in_tok_stride", ctypes.c_int64),
        ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
        ("k_base", ctypes.c_void_p), ("v_base", ctypes.c_void_p),
        ("L_max", ctypes.c_int64), ("kv_seq_stride", ctypes.c_int64),
        ("kv_head_stride", ctypes.c_int64), ("kv_tok_stride", ctypes.c_int64),
        ("kv_len", ctypes.c_void_p), ("max_kv_len", ctypes.c_int64), ("dtype", ctypes.c_int),
    ]


class GroupedArgs(ctypes.Structure):
    """Mirror of la_grouped_args."""

    _fields_ = [
        ("n_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_out", ctypes.c_int32),
        ("r", ctypes.c_int32), ("n_agents", ctypes.c_int32), ("n_segs", ctypes.c_int32),
        ("lora_scale", ctypes.c_float),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("A", ctypes.c_void_p), ("a_agent_stride", ctypes.c_int64), ("B", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64),
        ("seg_start", ctypes.c_void_p), ("seg_agent", ctypes.c_void_p), ("dtype", ctypes.c_int),
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"liblora_attn.so is not built ({LIB_PATH}); run "
                          "python -m rank_attention_b200.build_lib")
    lib = ctypes.CDLL(LIB_PATH)
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_status_string.argtypes = [ctypes.c_int]
    lib.lr_cache_append.restype = ctypes.c_int
    lib.lr_cache_append.argtypes = [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.lr_cache_append_agents.restype = ctypes.c_int
    lib.lr_cache_append_agents.argtypes = [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.lora_query_expand.restype = ctypes.c_int
    lib.lora_query_expand.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_float, ctypes.c_double, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    lib.lora_output_delta.restype = ctypes.c_int
    lib.lora_output_delta.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_float, ctypes.c_int, ctypes.c_void_p]
    lib.lora_attn_prefill.restype = ctypes.c_int
    lib.lora_attn_prefill.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p]
    lib.lora_attn_decode.restype = ctypes.c_int
    lib.lora_attn_decode.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]
    lib.lora_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.lora_attn_decode_workspace_bytes.argtypes = [ctypes.POINTER(AttnArgs)]
    lib.la_device_check.restype = ctypes.c_int
    lib.la_device_check.argtypes = []
    lib.la_device_check_word.restype = ctypes.c_int
    lib.lora_decode_step_host.restype = ctypes.c_int
    lib.lora_decode_step_host.argtypes = [
        ctypes.POINTER(AttnArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p]
    lib.la_device_check_word.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    lib.lora_attn_decode_step.restype = ctypes.c_int
    lib.lora_attn_decode_step.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]
    lib.lora_attn_decode_static_scratch.restype = ctypes.c_int
    lib.lora_attn_decode_static_scratch.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p]
    lib.lora_materialize_agent_kv.restype = ctypes.c_int
    lib.lora_materialize_agent_kv.argtypes = [ctypes.POINTER(AttnArgs), ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p]
    lib.lora_attn_decode_combine.restype = ctypes.c_int
    lib.lora_attn_decode_combine.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                                             ctypes.c_void_p, ctypes.c_void_p]
    lib.lora_attn_tree.restype = ctypes.c_int
    lib.lora_attn_tree.argtypes = [ctypes.POINTER(AttnArgs), ctypes.POINTER(TreeArgs),
                                   ctypes.c_void_p]
    lib.lora_qk_norm_rope.restype = ctypes.c_int
    lib.lora_qk_norm_rope.argtypes = [ctypes.POINTER(QkArgs), ctypes.POINTER(TreeArgs),
                                      ctypes.c_void_p]
    lib.lora_grouped_delta.restype = ctypes.c_int
    lib.lora_grouped_delta.argtypes = [ctypes.POINTER(GroupedArgs), ctypes.c_void_p]
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.la_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != LA_OK:
        raise LoraAttnError(status, where)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def lr_cache_append(X: torch.Tensor, A_kv: torch.Tensor, lr_cache: torch.Tensor, pos0: int,
                    stream=None) -> None:
    """lr_cache[:, pos0:pos0+n] = X @ A_kv.

    X [n_seqs, n, H] (last dim contiguous), A_kv [H, 2r] contiguous,
    lr_cache [n_seqs, L_max, 2r] (last two dims contiguous)."""
    n_seqs, n, H = X.shape
    r = A_kv.shape[1] // 2
    assert X.stride(2) == 1 and A_kv.is_contiguous()
    assert lr_cache.stride(2) == 1 and lr_cache.stride(1) == 2 * r
    st = lib.lr_cache_append(X.data_ptr(), X.stride(1), n, H, A_kv.data_ptr(), r,
                             lr_cache.data_ptr(), lr_cache.shape[1], pos0, n_seqs, X.stride(0),
                             lr_cache.stride(0), _dt(X), _stream(stream))
    _check(st, "lr_cache_append")


def lr_cache_append_agents(X: torch.Tensor, A_kv: torch.Tensor, lr_cache: torch.Tensor,
                           pos0: int, stream=None) -> None:
    """lr_cache[a, :, pos0:pos0+n] = X @ A_kv[a] for every agent a.

    X [n_seqs, n, H] (last dim contiguous), A_kv [n_agents, H, 2r] contiguous,
    lr_cache [n_agents, n_seqs, L_max, 2r] (last two dims contiguous)."""
    n_seqs, n, H = X.shape
    n_agents, r = A_kv.shape[0], A_kv.shape[2] // 2
    assert X.stride(2) == 1 and A_kv.is_contiguous()
    assert lr_cache.stride(3) == 1 and lr_cache.stride(2) == 2 * r
    st = lib.lr_cache_append_agents(X.data_ptr(), X.stride(1), n, H, A_kv.data_ptr(), n_agents, r,
                                    lr_cache.data_ptr(), lr_cache.stride(0), lr_cache.shape[2],
                                    pos0, n_seqs, X.stride(0), lr_cache.stride(1), _dt(X),
                                    _stream(stream))
    _check(st, "lr_cache_append_agents")


def lora_query_expand(q_base: torch.Tensor, lr_q: torch.Tensor, B_q: torch.Tensor,
                      q_out: torch.Tensor, pos_end: torch.Tensor, *, lora_scale: float,
                      rope_base: float, stream=None) -> None:
    """q_out = RoPE(q_base + s lr_q B_q^a) per agent and head.

    q_base, q_out [n_seqs, n_agents, n_tok, n_q, d] contiguous (may be the same
    tensor); lr_q [n_seqs, n_agents, n_tok, r]; B_q [n_agents, r, n_q*d];
    pos_end int32 [n_seqs]: token j sits at pos_end - n_tok + j."""
    n_seqs, n_agents, n_tok, n_q, d = q_base.shape
    r = lr_q.shape[-1]
    assert q_base.is_contiguous() and q_out.is_contiguous() and lr_q.is_contiguous()
    assert B_q.is_contiguous() and pos_end.dtype == torch.int32
    st = lib.lora_query_expand(q_base.data_ptr(), lr_q.data_ptr(), B_q.data_ptr(),
                               q_out.data_ptr(), n_seqs, n_agents, n_tok, n_q, d, r, lora_scale,
                               rope_base, pos_end.data_ptr(), _dt(q_base), _stream(stream))
    _check(st, "lora_query_expand")


def lora_output_delta(o: torch.Tensor, A_o: torch.Tensor, B_o: torch.Tensor, y: torch.Tensor, *,
                      lora_scale: float, stream=None) -> None:
    """y += s (o A_o) B_o^a per agent.

    o [n_seqs, n_agents, n_tok, d_in]; A_o [d_in, r] shared, or [n_agents, d_in, r];
    B_o [n_agents, r, d_out]; y [n_seqs, n_agents, n_tok, d_out]; all contiguous."""
    n_seqs, n_agents, n_tok, d_in = o.shape
    r, d_out = B_o.shape[1], B_o.shape[2]
    a_stride = A_o.stride(0) if A_o.dim() == 3 else 0
    assert o.is_contiguous() and A_o.is_contiguous() and B_o.is_contiguous() and y.is_contiguous()
    st = lib.lora_output_delta(o.data_ptr(), A_o.data_ptr(), a_stride, B_o.data_ptr(), y.data_ptr(),
                               n_seqs, n_agents, n_tok, d_in, d_out, r, lora_scale, _dt(o),
                               _stream(stream))
    _check(st, "lora_output_delta")


def _strides(t: torch.Tensor) -> list:
    """t's strides, dense ones in place of those of dimensions with one entry, which are never
    used and may hold anything."""
    shape, st = t.shape, list(t.stride())
    for i in range(len(st) - 2, -1, -1):
        if shape[i] <= 1:
            st[i] = shape[i + 1] * st[i + 1]
    return st


def _same_strides(a: torch.Tensor, b: torch.Tensor) -> bool:
    return a.stride() == b.stride() or _strides(a) == _strides(b)


def make_args(k_base, v_base, lr, B_k, B_v, q, out, *, lora_scale: float, rope_base: float,
              softmax_scale: Optional[float] = None, kv_len: Optional[torch.Tensor] = None,
              max_kv_len: int = 0, q_pos0: int = 0, value_path: int = LA_VALUE_REORDERED,
              key_pos0: int = 0, row_stats: Optional[torch.Tensor] = None) -> AttnArgs:
    """Fill la_attn_args from tensors.

    k_base, v_base [n_seqs, n_kv, L_max, d] (any strides with a unit last
    stride); lr [n_seqs, L_max, 2r], one LR cache shared by every agent, or
    [n_agents, n_seqs, L_max, 2r], one per agent; B_k, B_v [n_agents, r, n_kv*d];
    q, out [n_seqs, n_agents, n_tok, n_q, d] contiguous; kv_len int32 [n_seqs].
    B_k may be None for lora_attn_tree alone (keys without a low-rank part).
    Sequence-sharded decode: key_pos0 is the position of the caches' key row 0;
    row_stats a float32 [n_seqs, n_agents, n_q, 2] tensor the decode fills
    with each row's (M, L) for lora_attn_decode_combine.
    The struct holds addresses; it keeps the tensors alive as long as it lives itself
    (every make_* struct does)."""
    keep = (k_base, v_base, lr, B_k, B_v, q, out, kv_len, row_stats)
    n_seqs, n_kv, L_max, d = k_base.shape
    n_agents, n_tok, n_q = q.shape[1], q.shape[2], q.shape[3]
    per_agent = lr.dim() == 4
    lr_strides, kv_strides = _strides(lr), _strides(k_base)
    lr_agent_stride = lr_strides[0] if per_agent else 0
    if per_agent:
        assert lr.shape[0] == n_agents
    r = lr.shape[-1] // 2
    assert _same_strides(k_base, v_base) and kv_strides[3] == 1
    assert lr_strides[-2:] == [2 * r, 1]
    assert B_k is None or B_k.is_contiguous()
    assert B_v.is_contiguous() and q.is_contiguous() and out.is_contiguous()
    a = AttnArgs()
    a.n_seqs, a.n_agents, a.n_q_heads, a.n_kv_heads = n_seqs, n_agents, n_q, n_kv
    a.head_dim, a.r = d, r
    a.lora_scale = lora_scale
    a.softmax_scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(d)
    a.rope_base = rope_base
    a.L_max = L_max
    a.k_base, a.v_base = k_base.data_ptr(), v_base.data_ptr()
    a.kv_seq_stride, a.kv_head_stride, a.kv_tok_stride = kv_strides[:3]
    a.lr_cache, a.lr_seq_stride = lr.data_ptr(), lr_strides[-3]
    a.B_k, a.B_v = (B_k.data_ptr() if B_k is not None else None), B_v.data_ptr()
    a.q, a.out = q.data_ptr(), out.data_ptr()
    a.kv_len = kv_len.data_ptr() if kv_len is not None else None
    a.max_kv_len = max_kv_len
    a.q_pos0 = q_pos0
    a.n_q_tokens = n_tok
    a.io_dtype, a.out_dtype = _dt(k_base), _dt(out)
    a.lr_agent_stride = lr_agent_stride
    a.value_path = value_path
    a.key_pos0 = key_pos0
    if row_stats is not None:
        assert row_stats.dtype == torch.float32 and row_stats.is_contiguous()
        assert row_stats.numel() == 2 * n_seqs * n_agents * n_q
    a.row_stats = row_stats.data_ptr() if row_stats is not None else None
    a.device = q.device.index
    a.keep = keep
    a.checked = False   # lora_attn_tree's checks of these tensors, on its first call
    return a


def lora_attn_decode_workspace_bytes(args: AttnArgs) -> int:
    return int(lib.lora_attn_decode_workspace_bytes(ctypes.byref(args)))


def decode_workspace(args: AttnArgs, device) -> torch.Tensor:
    """A zero-filled workspace large enough for these decode arguments."""
    n = lora_attn_decode_workspace_bytes(args)
    if n == 0:
        raise LoraAttnError(LA_ERR_INVALID_ARG, "lora_attn_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lora_attn_decode(args: AttnArgs, workspace: torch.Tensor, stream=None) -> None:
    st = lib.lora_attn_decode(ctypes.byref(args), workspace.data_ptr(), workspace.numel(),
                              _stream(stream))
    _check(st, "lora_attn_decode")


def lora_attn_decode_combine(outs: torch.Tensor, stats: torch.Tensor, out: torch.Tensor,
                             stream=None) -> None:
    """Merge the decodes of n_parts key slices of the same queries: outs
    [n_parts, *rows, d] (fp32 or bf16), stats float32 [n_parts, *rows, 2] as
    row_stats holds them, out [*rows, d] of outs' dtype; all contiguous."""
    assert outs.is_contiguous() and stats.is_contiguous() and out.is_contiguous()
    assert stats.dtype == torch.float32 and out.dtype == outs.dtype
    n_parts, d = outs.shape[0], outs.shape[-1]
    rows = out.numel() // d
    assert outs.numel() == n_parts * rows * d and stats.numel() == 2 * n_parts * rows
    st = lib.lora_attn_decode_combine(outs.data_ptr(), stats.data_ptr(), n_parts, rows, d, _dt(out),
                                      out.data_ptr(), _stream(stream))
    _check(st, "lora_attn_decode_combine")


def lora_attn_decode_step(args: AttnArgs, A_kv: torch.Tensor, x_new: torch.Tensor,
                          workspace: torch.Tensor, stream=None) -> None:
    """A decode step on device buffers: the new token's LR row x_new[q] A_kv at
    kv_len[q] - 1 of the LR cache(s), then the decode.  x_new [n_seqs, hidden] contiguous;
    A_kv [hidden, 2r], or [n_agents, hidden, 2r] with per-agent caches."""
    assert x_new.is_contiguous() and A_kv.is_contiguous()
    st = lib.lora_attn_decode_step(ctypes.byref(args), A_kv.data_ptr(), x_new.data_ptr(),
                                   x_new.shape[-1], workspace.data_ptr(), workspace.numel(),
                                   _stream(stream))
    _check(st, "lora_attn_decode_step")


def lora_decode_step_host(args: AttnArgs, workspace: torch.Tensor, A_kv: torch.Tensor,
                          x_dev: torch.Tensor, x_host: torch.Tensor, q_host: torch.Tensor,
                          kv_len_host: torch.Tensor, out_host: torch.Tensor, stream=None) -> None:
    """One decode step from host buffers (copies in, LR append, decode, copy
    out), queued on the stream by one library call.  x_dev is the device
    staging [n_seqs, hidden]; the host tensors are CPU tensors, pinned for
    asynchronous copies."""
    for t in (x_host, q_host, kv_len_host, out_host):
        assert t.device.type == "cpu" and t.is_contiguous()
    assert x_dev.is_contiguous() and kv_len_host.dtype == torch.int32
    st = lib.lora_decode_step_host(ctypes.byref(args), workspace.data_ptr(), workspace.numel(),
                                   A_kv.data_ptr(), x_dev.shape[-1], x_dev.data_ptr(),
                                   x_host.data_ptr(), q_host.data_ptr(), kv_len_host.data_ptr(),
                                   out_host.data_ptr(), _stream(stream))
    _check(st, "lora_decode_step_host")


def packed_step_inputs(x_shape, q_shape, n_seqs: int, dtype: torch.dtype, device,
                       pin: bool = False):
    """x [x_shape], q [q_shape] (dtype) and kv_len int32 [n_seqs] as back-to-back
    views of one buffer: laid out so on both sides, lora_decode_step_host moves
    a step's inputs in one copy.  Returns (buffer, x, q, kv_len)."""
    es = torch.empty(0, dtype=dtype).element_size()
    nx, nq = math.prod(x_shape) * es, math.prod(q_shape) * es
    buf = torch.empty(nx + nq + 4 * n_seqs, dtype=torch.uint8, device=device,
                      pin_memory=pin)
    return (buf, buf[:nx].view(dtype).view(x_shape), buf[nx:nx + nq].view(dtype).view(q_shape),
            buf[nx + nq:].view(torch.int32))


def lora_attn_decode_static_scratch(args: AttnArgs, stream=None) -> None:
    """Decode without a workspace: the split scratch is the library's own device
    array (for callers that cannot allocate device memory; see the header)."""
    st = lib.lora_attn_decode_static_scratch(ctypes.byref(args), _stream(stream))
    _check(st, "lora_attn_decode_static_scratch")


def lora_materialize_agent_kv(args: AttnArgs, k_out: torch.Tensor, v_out: torch.Tensor,
                              stream=None) -> None:
    """Every agent's full K^a, V^a ([n_seqs, n_agents, n_kv, L_max, d] each): the
    non-shared baseline's caches (see the header)."""
    assert k_out.is_contiguous() and v_out.is_contiguous()
    st = lib.lora_materialize_agent_kv(ctypes.byref(args), k_out.data_ptr(), v_out.data_ptr(),
                                       _stream(stream))
    _check(st, "lora_materialize_agent_kv")


def lora_attn_prefill(args: AttnArgs, stream=None) -> None:
    st = lib.lora_attn_prefill(ctypes.byref(args), _stream(stream))
    _check(st, "lora_attn_prefill")


def _same_device(ts) -> int:
    """The one CUDA device that holds every tensor (None entries are skipped)."""
    devs = {t.device for t in ts if t is not None}
    if len(devs) != 1 or next(iter(devs)).type != "cuda":
        raise ValueError(f"expected every tensor on one CUDA device, got {sorted(map(str, devs))}")
    return next(iter(devs)).index


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _on_device(device: int, stream, where: str) -> int:
    """The stream to launch on; the arguments' device must be the current one."""
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"{where}: tensors are on cuda:{device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:   # without building a Stream object (about 2 us a call)
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


def make_tree_args(parent: Optional[torch.Tensor], tree_len: Optional[torch.Tensor] = None, *,
                   n_trees: Optional[int] = None) -> TreeArgs:
    """Fill la_tree_args: drafted trees, one per sequence (n_trees = 1) or one
    per agent.

    parent int32 [n_seqs, n_trees, n], parent[.., j] in [-1, j), or None: every
    tree is a chain; tree_len int32 [n_seqs, n_trees], nodes in use, or None: all
    of them.  n_trees is needed only where both are None (default 1)."""
    shape = None
    for t, dims in ((parent, 3), (tree_len, 2)):
        if t is None:
            continue
        if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"expected a contiguous int32 tensor of {dims} dimensions, got "
                             f"{t.dtype} {tuple(t.shape)}")
        if shape is not None and tuple(t.shape[:2]) != shape:
            raise ValueError("parent and tree_len disagree on [n_seqs, n_trees]")
        shape = tuple(t.shape[:2])
    if shape is not None and n_trees not in (None, shape[1]):
        raise ValueError("n_trees disagrees with parent / tree_len")
    a = TreeArgs()
    a.parent, a.tree_len = _ptr(parent), _ptr(tree_len)
    a.n_trees = shape[1] if shape is not None else (1 if n_trees is None else n_trees)
    a.n_seqs = None if shape is None else shape[0]
    a.n = None if parent is None else parent.shape[2]
    a.device = None if shape is None else _same_device((parent, tree_len))
    a.keep = (parent, tree_len)
    return a


def _check_tree(tree: TreeArgs, n_seqs: int, n: int, where: str) -> None:
    if tree.n_seqs not in (None, n_seqs) or tree.n not in (None, n):
        raise ValueError(f"{where}: the trees' shape [n_seqs, n_trees, n] does not fit the call's "
                         f"n_seqs {n_seqs} and n {n}")


def _check_attn(args: AttnArgs) -> None:
    """The tensors behind make_args' struct: one type, one device, shapes that fit (the
    struct alone does not show them)."""
    k_base, v_base, lr, B_k, B_v, q, out, kv_len, _ = args.keep
    n_seqs, n_kv, L_max, d = k_base.shape
    n_agents, r = q.shape[1], lr.shape[-1] // 2
    for t in (v_base, lr, B_k, B_v, q):
        if t is not None and t.dtype != k_base.dtype:
            raise TypeError(f"lora_attn_tree: expected every input of {k_base.dtype}, got {t.dtype}")
    if kv_len is None or kv_len.dtype != torch.int32 or not kv_len.is_contiguous() or kv_len.numel() < n_seqs:
        raise ValueError("lora_attn_tree: kv_len must be int32 [n_seqs]")

    def holds(t, *shape):   # with room for more agents than the call has, if it likes
        return t.dim() == len(shape) and t.shape[0] >= shape[0] and tuple(t.shape[1:]) == shape[1:]

    if v_base.shape != k_base.shape or q.shape[0] != n_seqs or q.shape[4:] != (d,) or out.numel() < q.numel() or \
            lr.shape[-3] < n_seqs or lr.shape[-2] < L_max or not holds(B_v, n_agents, r, n_kv * d) or \
            (B_k is not None and not holds(B_k, n_agents, r, n_kv * d)):
        raise ValueError("lora_attn_tree: shapes of the caches, LR rows, B_k, B_v, q and out do not fit")
    _same_device(args.keep)


def lora_attn_tree(args: AttnArgs, tree: TreeArgs, stream=None) -> None:
    """Attention of the drafted nodes over the committed context and their own
    branches.  args from make_args, with q and out [n_seqs, n_agents, n, n_q, d],
    kv_len the committed lengths and max_kv_len a bound on kv_len + n_trees * n."""
    if not getattr(args, "checked", True):
        _check_attn(args)
        args.checked = True
    _check_tree(tree, args.n_seqs, args.n_q_tokens, "lora_attn_tree")
    device = getattr(args, "device", None)   # of make_args' tensors
    if tree.device not in (None, device):
        raise ValueError("lora_attn_tree: the trees are on another device")
    s = _stream(stream) if device is None else _on_device(device, stream, "lora_attn_tree")
    st = lib.lora_attn_tree(ctypes.byref(args), ctypes.byref(tree), s)
    _check(st, "lora_attn_tree")


def make_qk_args(q, k, v, w_q, w_k, q_out, k_base, v_base, kv_len, *, rope_base: float,
                 max_kv_len: int, eps: float = 1e-6) -> QkArgs:
    """Fill la_qk_args from tensors.

    q [n_seqs, n_agents, n, n_q, d] (heads contiguous; sequence, agent and token
    strides free: slices of a fused projection's output will do) with q_out of
    that shape, contiguous, or both None; k, v [n_seqs, n_trees, n, n_kv, d] the
    same way, of equal strides, with the base caches k_base, v_base
    [n_seqs, n_kv, L_max, d] of equal strides, or None; w_q, w_k [d] or None;
    kv_len int32 [n_seqs]."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("one of q and k is needed")
    dt = ref.dtype
    for t in (q, k, v, w_q, w_k, q_out, k_base, v_base):
        if t is not None and t.dtype != dt:
            raise TypeError(f"expected every tensor of {dt}, got {t.dtype}")
    a = QkArgs()
    n_seqs, _, n, _, d = ref.shape
    a.n_seqs, a.n_tokens, a.head_dim = n_seqs, n, d
    a.n_agents = a.n_q_heads = a.n_kv_heads = 1
    a.eps, a.rope_base = eps, rope_base
    if (q is None) != (q_out is None) or (k is None) != (k_base is None) or \
            (v is None) != (v_base is None):
        raise ValueError("q and q_out, k and k_base, v and v_base come together")

    def heads(t):
        if t.dim() != 5 or t.shape[0] != n_seqs or t.shape[2] != n or t.shape[4] != d or \
                t.stride(4) != 1 or (t.shape[3] > 1 and t.stride(3) != d):
            raise ValueError("expected [n_seqs, ., n, heads, d] with contiguous heads, got "
                             f"{tuple(t.shape)} with strides {t.stride()}")

    if q is not None:
        heads(q)
        if q_out.shape != q.shape or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous, of q's shape")
        a.n_agents, a.n_q_heads = q.shape[1], q.shape[3]
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
        a.q_seq_stride, a.q_agent_stride, a.q_tok_stride = _strides(q)[:3]
    a.n_trees = None
    if k is not None:
        heads(k)
        a.n_trees = k.shape[1]
        if q is None:
            a.n_agents = k.shape[1]
        a.n_kv_heads = k.shape[3]
        a.k, a.v = k.data_ptr(), _ptr(v)
        a.kv_in_seq_stride, a.kv_in_tree_stride, a.kv_in_tok_stride = _strides(k)[:3]
        if k_base.dim() != 4 or k_base.shape[:2] != (n_seqs, a.n_kv_heads) or \
                k_base.shape[3] != d or k_base.stride(3) != 1:
            raise ValueError("k_base must be [n_seqs, n_kv, L_max, d] with a unit last stride")
        if v is not None and (v.shape != k.shape or not _same_strides(v, k) or v_base.shape != k_base.shape or
                              not _same_strides(v_base, k_base)):
            raise ValueError("v and v_base must have the shapes and strides of k and k_base")
        a.k_base, a.v_base = k_base.data_ptr(), _ptr(v_base)
        a.L_max = k_base.shape[2]
        a.kv_seq_stride, a.kv_head_stride, a.kv_tok_stride = _strides(k_base)[:3]
    elif v is not None:
        raise ValueError("v needs k")
    else:
        a.L_max = max(1, max_kv_len)
    for w in (w_q, w_k):
        if w is not None and (w.shape != (d,) or not w.is_contiguous()):
            raise ValueError("norm weights are contiguous [d]")
    a.w_q, a.w_k = _ptr(w_q), _ptr(w_k)
    if kv_len.dtype != torch.int32 or kv_len.shape != (n_seqs,) or not kv_len.is_contiguous():
        raise ValueError("kv_len must be int32 [n_seqs]")
    a.kv_len, a.max_kv_len, a.dtype = kv_len.data_ptr(), max_kv_len, _dt(ref)
    a.keep = (q, k, v, w_q, w_k, q_out, k_base, v_base, kv_len)
    a.device = _same_device(a.keep)
    return a


def lora_qk_norm_rope(args: QkArgs, tree: Optional[TreeArgs] = None, stream=None) -> None:
    """Norm and rotate new queries and keys per head and write the cache rows
    (args from make_qk_args); tree None: one chain per sequence from kv_len on."""
    if tree is not None:
        _check_tree(tree, args.n_seqs, args.n_tokens, "lora_qk_norm_rope")
        if tree.device not in (None, args.device):
            raise ValueError("lora_qk_norm_rope: the trees are on another device")
    if args.n_trees is not None and args.n_trees != (1 if tree is None else tree.n_trees):
        raise ValueError(f"lora_qk_norm_rope: k has {args.n_trees} trees of rows")
    s = _on_device(args.device, stream, "lora_qk_norm_rope")
    st = lib.lora_qk_norm_rope(ctypes.byref(args), None if tree is None else ctypes.byref(tree), s)
    _check(st, "lora_qk_norm_rope")


def make_grouped_args(x, A, B, y, out, seg_start, seg_agent, *, lora_scale: float) -> GroupedArgs:
    """Fill la_grouped_args from tensors.

    x [n_tokens, hidden], y and out [n_tokens, n_out] (unit last strides; out may
    be y); A [hidden, r] shared, or [n_agents, hidden, r]; B [n_agents, r, n_out]
    contiguous; seg_start int32 [n_segs + 1], seg_agent int32 [n_segs]."""
    T, H = x.shape
    n_agents, r, N = B.shape
    if y.shape != (T, N) or out.shape != (T, N) or tuple(A.shape[-2:]) != (H, r) or \
            A.dim() not in (2, 3) or (A.dim() == 3 and A.shape[0] != n_agents):
        raise ValueError("shapes of x, A, B, y and out do not fit")
    if not (x.stride(1) == y.stride(1) == out.stride(1) == 1) or not B.is_contiguous() or \
            A.stride(-1) != 1 or A.stride(-2) != r:
        raise ValueError("x, y and out need unit last strides, B and each A must be contiguous")
    for t in (A, B, y, out):
        if t.dtype != x.dtype:
            raise TypeError(f"expected every tensor of {x.dtype}, got {t.dtype}")
    n_segs = seg_agent.numel()
    if seg_start.dtype != torch.int32 or seg_agent.dtype != torch.int32 or \
            seg_start.shape != (n_segs + 1,) or seg_agent.dim() != 1 or \
            not seg_start.is_contiguous() or not seg_agent.is_contiguous():
        raise ValueError("seg_start is int32 [n_segs + 1], seg_agent int32 [n_segs]")
    a = GroupedArgs()
    a.n_tokens, a.hidden, a.n_out, a.r, a.n_agents, a.n_segs = T, H, N, r, n_agents, n_segs
    a.lora_scale = lora_scale
    a.x, a.ldx = x.data_ptr(), x.stride(0) if T > 1 else H
    a.A, a.a_agent_stride = A.data_ptr(), (A.stride(0) if A.dim() == 3 and n_agents > 1 else 0)
    a.B = B.data_ptr()
    a.y, a.ldy = y.data_ptr(), y.stride(0) if T > 1 else N
    a.out, a.ldo = out.data_ptr(), out.stride(0) if T > 1 else N
    a.seg_start, a.seg_agent, a.dtype = seg_start.data_ptr(), seg_agent.data_ptr(), _dt(x)
    a.keep = (x, A, B, y, out, seg_start, seg_agent)
    a.device = _same_device(a.keep)
    return a


def lora_grouped_delta(args: GroupedArgs, stream=None) -> None:
    """out = y + s (x A_a) B_a over ragged segments of tokens grouped by agent
    (args from make_grouped_args)."""
    s = _on_device(args.device, stream, "lora_grouped_delta")
    st = lib.lora_grouped_delta(ctypes.byref(args), s)
    _check(st, "lora_grouped_delta")


def la_device_check() -> int:
    return int(lib.la_device_check())


def la_device_check_word() -> tuple:
    """(status, bits of the device error word that fired); reads and clears it."""
    w = ctypes.c_int32(0)
    st = int(lib.la_device_check_word(ctypes.byref(w)))
    return st, int(w.value)


class DecodeStep:
    """One decode step of the hot path: the new token's LR row at kv_len - 1,
    then every agent's query over the shared caches (lora_attn_decode_step:
    one library call: the row append, then the decode).

    Holds the argument struct and the zero-filled split-K workspace.  Tensors
    must stay alive while it is used.  Without x_new / A_kv it is the decode
    alone."""

    def __init__(self, k_base, v_base, lr, B_k, B_v, q, out, kv_len, *, lora_scale, rope_base,
                 max_kv_len, A_kv=None, x_new=None):
        self.args = make_args(k_base, v_base, lr, B_k, B_v, q, out, lora_scale=lora_scale,
                              rope_base=rope_base, kv_len=kv_len, max_kv_len=max_kv_len)
        self.workspace = decode_workspace(self.args, q.device)
        self.lr, self.A_kv = lr, A_kv
        self.x_new = None if x_new is None else x_new.reshape(x_new.shape[0], -1)
        self._keep = (k_base, v_base, lr, B_k, B_v, q, out, kv_len, x_new)

    def __call__(self, stream=None) -> None:
        if self.x_new is not None:
            lora_attn_decode_step(self.args, self.A_kv, self.x_new, self.workspace, stream)
        else:
            lora_attn_decode(self.args, self.workspace, stream)

    def from_host(self, x_host, q_host, kv_len_host, out_host, stream=None) -> None:
        """The same step with its inputs and outputs in host memory: one call
        that copies them in and out around the append and the decode; the new
        rows land at kv_len_host - 1."""
        lora_decode_step_host(self.args, self.workspace, self.A_kv, self.x_new, x_host, q_host,
                              kv_len_host, out_host, stream)
