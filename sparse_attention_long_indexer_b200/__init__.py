"""Python binding of the DSA forward-path C ABI (``include/dsa.h``, ``libdsa.so``).

Argument marshalling only: every step of the path (lightning indexer, top-k selection,
sparse MLA attention) runs in the library's CUDA kernels. PyTorch supplies device memory
and streams. There is no CPU fallback: importing this package raises if ``libdsa.so`` is
missing, and every call raises ``DSAError`` on a non-OK status.

Functions with the C names take torch tensors (device memory, contiguous, the dtypes
stated in ``include/dsa.h``); ``forward`` / ``indexer_topk`` / ``sparse_mla_attn``
allocate outputs for convenience.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdsa.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m sparse_attention_long_indexer_b200.build` "
        "(the DSA path has no CPU fallback)")
_lib = ctypes.CDLL(_LIB_PATH)

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA = 0, 1, 2, 3
DSA_ERR_DEVICE_TIMEOUT, DSA_ERR_INDEX_RANGE, DSA_ERR_WORKSPACE = 4, 5, 6

LIBRARY_PATH = _LIB_PATH
EXPORTED = ("dsa_workspace_bytes", "dsa_workspace_init", "dsa_indexer_topk", "dsa_sparse_mla_attn",
            "dsa_forward", "dsa_get_device_status", "dsa_status_string", "dsa_version",
            "dsa_indexer_topk_decode_noalloc", "dsa_masked_mqa_attn", "dsa_indexer_topk_scores",
            "dsa_indexer_kl_loss", "dsa_set_wait_budget_ns", "dsa_qcache_workspace_bytes", "dsa_qcache_write",
            "dsa_qcache_read", "dsa_sparse_mla_attn_qcache", "dsa_tree_mla_attn", "dsa_tree_mla_attn_qcache")


class dsa_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("n_idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]


class dsa_qcache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rope", ctypes.c_void_p)]


_P = ctypes.c_void_p
_DIMS = ctypes.POINTER(dsa_dims)
_lib.dsa_workspace_bytes.argtypes = [_DIMS, ctypes.c_int32]
_lib.dsa_workspace_bytes.restype = ctypes.c_size_t
_lib.dsa_workspace_init.argtypes = [_P, ctypes.c_size_t, _P]
_lib.dsa_workspace_init.restype = ctypes.c_int
_lib.dsa_indexer_topk.argtypes = [_DIMS, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_indexer_topk.restype = ctypes.c_int
_lib.dsa_indexer_topk_scores.argtypes = [_DIMS, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_indexer_topk_scores.restype = ctypes.c_int
_lib.dsa_indexer_kl_loss.argtypes = [_DIMS, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_indexer_kl_loss.restype = ctypes.c_int
_lib.dsa_sparse_mla_attn.argtypes = [_DIMS, _P, _P, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_sparse_mla_attn.restype = ctypes.c_int
_lib.dsa_masked_mqa_attn.argtypes = [_DIMS, _P, _P, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_masked_mqa_attn.restype = ctypes.c_int
_lib.dsa_forward.argtypes = [_DIMS, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_forward.restype = ctypes.c_int
_QC = ctypes.POINTER(dsa_qcache)
_lib.dsa_qcache_workspace_bytes.argtypes = [_DIMS, ctypes.c_int32]
_lib.dsa_qcache_workspace_bytes.restype = ctypes.c_size_t
_lib.dsa_qcache_write.argtypes = [_DIMS, _P, _P, ctypes.c_int32, _P, _P, _P, _QC, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_qcache_write.restype = ctypes.c_int
_lib.dsa_qcache_read.argtypes = [_DIMS, _QC, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_qcache_read.restype = ctypes.c_int
_lib.dsa_sparse_mla_attn_qcache.argtypes = [_DIMS, _P, _QC, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_sparse_mla_attn_qcache.restype = ctypes.c_int
_lib.dsa_tree_mla_attn.argtypes = [_DIMS, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_tree_mla_attn.restype = ctypes.c_int
_lib.dsa_tree_mla_attn_qcache.argtypes = [_DIMS, _P, _QC, _P, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.dsa_tree_mla_attn_qcache.restype = ctypes.c_int
_lib.dsa_get_device_status.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]
_lib.dsa_get_device_status.restype = ctypes.c_int
_lib.dsa_status_string.argtypes = [ctypes.c_int]
_lib.dsa_status_string.restype = ctypes.c_char_p
_lib.dsa_set_wait_budget_ns.argtypes = [ctypes.c_uint64]
_lib.dsa_set_wait_budget_ns.restype = ctypes.c_int
_lib.dsa_version.argtypes = []
_lib.dsa_version.restype = ctypes.c_int32


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dsa_status_string(status)} (status {status})")


def dsa_status_string(status: int) -> str:
    return _lib.dsa_status_string(int(status)).decode()


def dsa_set_wait_budget_ns(ns: int):
    """Test setting: budget of the pipeline waits of the indexer and of the attention over an 8-bit cache or a
    drafted tree, in ns (0 = the default 2 s)."""
    _check(_lib.dsa_set_wait_budget_ns(int(ns)), "dsa_set_wait_budget_ns")


def dsa_version() -> int:
    return int(_lib.dsa_version())


def make_dims(batch, n_q, max_len, n_idx_heads=64, idx_dim=128, n_heads=128, d_latent=512, d_rope=64,
              softmax_scale=None) -> dsa_dims:
    if softmax_scale is None:
        softmax_scale = 1.0 / float(d_latent + d_rope) ** 0.5
    return dsa_dims(batch, n_q, max_len, n_idx_heads, idx_dim, n_heads, d_latent, d_rope, softmax_scale)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("DSA tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle without a torch.cuda.Stream object around it (3 us of every call), where
# this torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DSAError(status, where)


def _expect(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be device memory")


# ----------------------------------------------------------------------------- C-named calls
def dsa_workspace_bytes(dims: dsa_dims, topk: int) -> int:
    return int(_lib.dsa_workspace_bytes(ctypes.byref(dims), int(topk)))


def dsa_workspace_init(ws: torch.Tensor, stream=None):
    _check(_lib.dsa_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "dsa_workspace_init")


def dsa_indexer_topk(dims, q_idx, w, k_idx, scales, lengths, topk, out_idx, ws, stream=None):
    _check(_lib.dsa_indexer_topk(ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(scales), _ptr(lengths),
                                 int(topk), _ptr(out_idx), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_indexer_topk")


def dsa_indexer_topk_scores(dims, q_idx, w, k_idx, scales, lengths, topk, out_idx, out_scores, ws, stream=None):
    _check(_lib.dsa_indexer_topk_scores(ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(scales),
                                        _ptr(lengths), int(topk), _ptr(out_idx), _ptr(out_scores), _ptr(ws),
                                        ws.numel(), _stream(stream)), "dsa_indexer_topk_scores")


def dsa_indexer_kl_loss(dims, q, latent_kv, idx, idx_scores, lse, topk, loss, ws, stream=None):
    _check(_lib.dsa_indexer_kl_loss(ctypes.byref(dims), _ptr(q), _ptr(latent_kv), _ptr(idx), _ptr(idx_scores),
                                    _ptr(lse), int(topk), _ptr(loss), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_indexer_kl_loss")


def dsa_sparse_mla_attn(dims, q, latent_kv, idx, topk, out, lse, ws, stream=None):
    _check(_lib.dsa_sparse_mla_attn(ctypes.byref(dims), _ptr(q), _ptr(latent_kv), _ptr(idx), int(topk), _ptr(out),
                                    _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), "dsa_sparse_mla_attn")


def dsa_masked_mqa_attn(dims, q, latent_kv, idx, topk, out, lse, ws, stream=None):
    _check(_lib.dsa_masked_mqa_attn(ctypes.byref(dims), _ptr(q), _ptr(latent_kv), _ptr(idx), int(topk), _ptr(out),
                                    _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), "dsa_masked_mqa_attn")


def dsa_forward(dims, q_idx, w, k_idx, scales, lengths, topk, q, latent_kv, out_idx, out, lse, ws, stream=None):
    _check(_lib.dsa_forward(ctypes.byref(dims), _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(scales), _ptr(lengths),
                            int(topk), _ptr(q), _ptr(latent_kv), _ptr(out_idx), _ptr(out), _ptr(lse), _ptr(ws),
                            ws.numel(), _stream(stream)), "dsa_forward")


def dsa_qcache_workspace_bytes(dims: dsa_dims, topk: int) -> int:
    return int(_lib.dsa_qcache_workspace_bytes(ctypes.byref(dims), int(topk)))


def dsa_qcache_write(dims, latent, keys, n_src, src_rows, start, lengths, cache, k_idx, k_scale, ws, stream=None):
    _check(_lib.dsa_qcache_write(ctypes.byref(dims), _ptr(latent), _ptr(keys), int(n_src), _ptr(src_rows), _ptr(start),
                                 _ptr(lengths), ctypes.byref(cache) if cache is not None else None, _ptr(k_idx),
                                 _ptr(k_scale), _ptr(ws), ws.numel(), _stream(stream)), "dsa_qcache_write")


def dsa_qcache_read(dims, cache, rows_listed, start, lengths, out, ws, stream=None):
    _check(_lib.dsa_qcache_read(ctypes.byref(dims), ctypes.byref(cache), _ptr(rows_listed), _ptr(start),
                                _ptr(lengths), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "dsa_qcache_read")


def dsa_sparse_mla_attn_qcache(dims, q, cache, idx, topk, out, lse, ws, stream=None):
    _check(_lib.dsa_sparse_mla_attn_qcache(ctypes.byref(dims), _ptr(q), ctypes.byref(cache), _ptr(idx), int(topk),
                                           _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_sparse_mla_attn_qcache")


def dsa_tree_mla_attn(dims, q, latent_kv, idx, topk, draft, parents, out, lse, ws, stream=None):
    _check(_lib.dsa_tree_mla_attn(ctypes.byref(dims), _ptr(q), _ptr(latent_kv), _ptr(idx), int(topk), _ptr(draft),
                                  _ptr(parents), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_tree_mla_attn")


def dsa_tree_mla_attn_qcache(dims, q, cache, idx, topk, draft, parents, out, lse, ws, stream=None):
    _check(_lib.dsa_tree_mla_attn_qcache(ctypes.byref(dims), _ptr(q), ctypes.byref(cache), _ptr(idx), int(topk),
                                         _ptr(draft), _ptr(parents), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                         _stream(stream)), "dsa_tree_mla_attn_qcache")


def dsa_get_device_status(ws: torch.Tensor, stream=None):
    detail = ctypes.c_uint32(0)
    st = int(_lib.dsa_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(detail)))
    return st, int(detail.value)


# ----------------------------------------------------------------------------- conveniences
@dataclass
class Workspace:
    """A device workspace sized for (dims, topk), status word zeroed."""
    dims: dsa_dims
    topk: int
    buf: torch.Tensor

    @staticmethod
    def create(dims: dsa_dims, topk: int, device=None, stream=None) -> "Workspace":
        n = dsa_workspace_bytes(dims, topk)
        if n == 0:
            raise DSAError(DSA_ERR_INVALID_ARG, "dsa_workspace_bytes")
        buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-buf.data_ptr()) % 256
        buf = buf[off:off + n]
        dsa_workspace_init(buf, stream)
        return Workspace(dims, topk, buf)

    @staticmethod
    def create_qcache(dims: dsa_dims, topk: int, device=None, stream=None) -> "Workspace":
        """A workspace for the calls on an 8-bit cache and on drafted trees, of these sizes and smaller ones."""
        n = dsa_qcache_workspace_bytes(dims, topk)
        if n == 0:
            raise DSAError(DSA_ERR_INVALID_ARG, "dsa_qcache_workspace_bytes")
        buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-buf.data_ptr()) % 256
        buf = buf[off:off + n]
        dsa_workspace_init(buf, stream)
        return Workspace(dims, topk, buf)

    def check(self, stream=None):
        """Raises DSAError if a kernel recorded a device-side error since the last check."""
        st, detail = dsa_get_device_status(self.buf, stream)
        if st != DSA_OK:
            raise DSAError(st, f"device status (detail 0x{detail:08x})")


def _scales(q_scale: torch.Tensor, k_scale: torch.Tensor) -> torch.Tensor:
    return torch.cat([q_scale.reshape(-1), k_scale.reshape(-1)]).to(torch.float32).contiguous()


def indexer_topk(dims, q_idx, w, k_idx, q_scale, k_scale, lengths, topk, ws: Workspace, stream=None):
    """Returns int32 [B, n_q, topk] selected positions (-1 padded, unspecified order)."""
    _expect(q_idx, torch.uint8, "q_idx")
    _expect(k_idx, torch.uint8, "k_idx")
    _expect(w, torch.bfloat16, "w")
    out_idx = torch.empty((dims.batch, dims.n_q, topk), dtype=torch.int32, device=q_idx.device)
    dsa_indexer_topk(dims, q_idx, w, k_idx, _scales(q_scale, k_scale), lengths.to(torch.int32).contiguous(), topk,
                     out_idx, ws.buf, stream)
    return out_idx


def sparse_mla_attn(dims, q, latent_kv, idx, topk, ws: Workspace, stream=None):
    """Returns (out bf16 [B, n_q, H, d_latent], lse fp32 [B, n_q, H])."""
    _expect(q, torch.bfloat16, "q")
    _expect(latent_kv, torch.bfloat16, "latent_kv")
    out = torch.empty((dims.batch, dims.n_q, dims.n_heads, dims.d_latent), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((dims.batch, dims.n_q, dims.n_heads), dtype=torch.float32, device=q.device)
    dsa_sparse_mla_attn(dims, q, latent_kv, idx.to(torch.int32).contiguous(), topk, out, lse, ws.buf, stream)
    return out, lse


def indexer_topk_scores(dims, q_idx, w, k_idx, q_scale, k_scale, lengths, topk, ws: Workspace, stream=None):
    """Returns (idx int32 [B, n_q, topk], scores fp32 [B, n_q, topk]); -1 / -inf padded."""
    _expect(q_idx, torch.uint8, "q_idx")
    _expect(k_idx, torch.uint8, "k_idx")
    _expect(w, torch.bfloat16, "w")
    out_idx = torch.empty((dims.batch, dims.n_q, topk), dtype=torch.int32, device=q_idx.device)
    out_scores = torch.empty((dims.batch, dims.n_q, topk), dtype=torch.float32, device=q_idx.device)
    dsa_indexer_topk_scores(dims, q_idx, w, k_idx, _scales(q_scale, k_scale), lengths.to(torch.int32).contiguous(),
                            topk, out_idx, out_scores, ws.buf, stream)
    return out_idx, out_scores


def indexer_kl_loss(dims, q, latent_kv, idx, idx_scores, lse, topk, ws: Workspace, stream=None):
    """Returns the per-query indexer-alignment KL terms, fp32 [B, n_q]."""
    loss = torch.empty((dims.batch, dims.n_q), dtype=torch.float32, device=q.device)
    dsa_indexer_kl_loss(dims, q, latent_kv, idx.to(torch.int32).contiguous(), idx_scores.contiguous(),
                        lse.contiguous(), topk, loss, ws.buf, stream)
    return loss


def masked_mqa_attn(dims, q, latent_kv, idx, topk, ws: Workspace, stream=None):
    """The masked dense mode of the attention. Returns (out, lse) like ``sparse_mla_attn``."""
    _expect(q, torch.bfloat16, "q")
    _expect(latent_kv, torch.bfloat16, "latent_kv")
    out = torch.empty((dims.batch, dims.n_q, dims.n_heads, dims.d_latent), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((dims.batch, dims.n_q, dims.n_heads), dtype=torch.float32, device=q.device)
    dsa_masked_mqa_attn(dims, q, latent_kv, idx.to(torch.int32).contiguous(), topk, out, lse, ws.buf, stream)
    return out, lse


def forward(dims, q_idx, w, k_idx, q_scale, k_scale, lengths, topk, q, latent_kv, ws: Workspace, stream=None,
            return_idx: bool = True):
    """The whole DSA forward path. Returns (idx or None, out, lse)."""
    dev = q.device
    out = torch.empty((dims.batch, dims.n_q, dims.n_heads, dims.d_latent), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((dims.batch, dims.n_q, dims.n_heads), dtype=torch.float32, device=dev)
    out_idx = torch.empty((dims.batch, dims.n_q, topk), dtype=torch.int32, device=dev) if return_idx else None
    dsa_forward(dims, q_idx, w, k_idx, _scales(q_scale, k_scale), lengths.to(torch.int32).contiguous(), topk, q,
                latent_kv, out_idx, out, lse, ws.buf, stream)
    return out_idx, out, lse


# ----------------------------------------------------------------------------- 8-bit cache, drafted trees
_SCALE_GROUP = 128      # latent dims per scale


def _same(name: str, t: torch.Tensor, dtype, numel: int, device: int):
    """Checks one tensor of a call: dtype, size and device, so that no kernel reads past its end."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()} in {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{device}")


def _call_device(t: torch.Tensor) -> int:
    """The device of a call's tensors, which must be the current one (its stream takes the launch)."""
    device = t.get_device()                       # -1 on the CPU
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError(f"tensors on {t.device}: make it the current device first (torch.cuda.device)")
    return device


def _workspace(ws: Workspace, device: int) -> torch.Tensor:
    """A workspace's buffer, checked like the call's tensors: kernels write to it."""
    buf = ws.buf
    if buf.dtype is not torch.uint8:
        raise TypeError(f"workspace: expected torch.uint8, got {buf.dtype}")
    if buf.get_device() != device:
        raise ValueError(f"the workspace is on {buf.device}, the call runs on cuda:{device}")
    return buf


@dataclass
class QCache:
    """An 8-bit latent cache (see ``dsa_qcache`` in ``include/dsa.h``), with the index keys beside it.

    codes   uint8 (E4M3) [B, max_len, d_latent]
    scales  fp32 [B, max_len, ceil(d_latent / 128)]
    rope    bf16 [B, max_len, d_rope]
    k_idx   uint8 (E4M3) [B, max_len, idx_dim], k_scale fp32 [B, max_len], or None without an indexer
    """
    codes: torch.Tensor
    scales: torch.Tensor
    rope: torch.Tensor
    k_idx: Optional[torch.Tensor] = None
    k_scale: Optional[torch.Tensor] = None

    @staticmethod
    def create(dims: dsa_dims, device=None) -> "QCache":
        """An empty cache for these dims: rows of zeros."""
        device = device or "cuda"
        b, n = dims.batch, dims.max_len
        groups = -(-dims.d_latent // _SCALE_GROUP)
        return QCache(torch.zeros((b, n, dims.d_latent), dtype=torch.uint8, device=device),
                      torch.ones((b, n, groups), dtype=torch.float32, device=device),
                      torch.zeros((b, n, dims.d_rope), dtype=torch.bfloat16, device=device),
                      torch.zeros((b, n, dims.idx_dim), dtype=torch.uint8, device=device),
                      torch.ones((b, n), dtype=torch.float32, device=device))

    def _struct(self, dims: dsa_dims, device: int) -> dsa_qcache:
        rows = dims.batch * dims.max_len
        _same("cache.codes", self.codes, torch.uint8, rows * dims.d_latent, device)
        _same("cache.scales", self.scales, torch.float32, rows * -(-dims.d_latent // _SCALE_GROUP), device)
        _same("cache.rope", self.rope, torch.bfloat16, rows * dims.d_rope, device)
        return dsa_qcache(_ptr(self.codes), _ptr(self.scales), _ptr(self.rope))


def _allocating(stream):
    """Outputs of a call on ``stream`` come from that stream's memory: memory of the current stream could still
    be in use there by earlier work that the call does not wait for."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _per_sequence(dims, device, **tensors):
    for name, t in tensors.items():
        if t is not None:
            _same(name, t, torch.int32, dims.batch, device)


def qcache_write(dims, cache: QCache, latent, keys, ws: Workspace, start=None, lengths=None, src_rows=None,
                 stream=None):
    """Quantises new rows into ``cache``: row j of sequence b goes to position start[b] + j if that is below
    lengths[b]. ``latent`` bf16 [B, n_src, d_latent + d_rope] and ``keys`` bf16 [B, n_src, idx_dim], either of
    them None; ``src_rows`` int32 [B, n_q] lists the source row of each written one (< 0: none)."""
    if latent is None and keys is None:
        raise ValueError("qcache_write: neither latent nor keys")
    first = latent if latent is not None else keys
    device = _call_device(first)
    if first.dim() != 3:
        raise ValueError(f"qcache_write: expected [B, n_src, dims] rows, got {tuple(first.shape)}")
    n_src = first.shape[1]
    if latent is not None:
        _same("latent", latent, torch.bfloat16, dims.batch * n_src * (dims.d_latent + dims.d_rope), device)
    if keys is not None:
        if cache.k_idx is None or cache.k_scale is None:
            raise ValueError("qcache_write: the cache holds no index keys")
        _same("keys", keys, torch.bfloat16, dims.batch * n_src * dims.idx_dim, device)
        _same("cache.k_idx", cache.k_idx, torch.uint8, dims.batch * dims.max_len * dims.idx_dim, device)
        _same("cache.k_scale", cache.k_scale, torch.float32, dims.batch * dims.max_len, device)
    if src_rows is not None:
        _same("src_rows", src_rows, torch.int32, dims.batch * dims.n_q, device)
    _per_sequence(dims, device, start=start, lengths=lengths)
    dsa_qcache_write(dims, latent, keys, n_src, src_rows, start, lengths, cache._struct(dims, device),
                     cache.k_idx if keys is not None else None, cache.k_scale if keys is not None else None,
                     _workspace(ws, device), stream)


def qcache_read(dims, cache: QCache, ws: Workspace, rows=None, start=None, lengths=None, stream=None):
    """bf16 [B, n_q, d_latent + d_rope]: the listed positions (``rows`` int32 [B, n_q], < 0: zeros), or
    start[b] .. start[b] + n_q - 1, zeros from lengths[b] on."""
    device = _call_device(cache.codes)
    if rows is not None:
        _same("rows", rows, torch.int32, dims.batch * dims.n_q, device)
    _per_sequence(dims, device, start=start, lengths=lengths)
    with _allocating(stream):
        out = cache.rope.new_empty((dims.batch, dims.n_q, dims.d_latent + dims.d_rope))
    dsa_qcache_read(dims, cache._struct(dims, device), rows, start, lengths, out, _workspace(ws, device), stream)
    return out


def _attention_inputs(dims, q, idx, topk, stream):
    device = _call_device(q)
    queries = dims.batch * dims.n_q
    _same("q", q, torch.bfloat16, queries * dims.n_heads * (dims.d_latent + dims.d_rope), device)
    _same("idx", idx, torch.int32, queries * topk, device)
    with _allocating(stream):
        out = q.new_empty((dims.batch, dims.n_q, dims.n_heads, dims.d_latent))
        lse = q.new_empty((dims.batch, dims.n_q, dims.n_heads), dtype=torch.float32)
    return device, out, lse


def sparse_mla_attn_qcache(dims, q, cache: QCache, idx, topk, ws: Workspace, stream=None):
    """``sparse_mla_attn`` over an 8-bit cache. Returns (out bf16 [B, n_q, H, d_latent], lse fp32 [B, n_q, H])."""
    device, out, lse = _attention_inputs(dims, q, idx, topk, stream)
    dsa_sparse_mla_attn_qcache(dims, q, cache._struct(dims, device), idx, topk, out, lse, _workspace(ws, device),
                               stream)
    return out, lse


def tree_mla_attn(dims, q, cache, idx, topk, draft, parents, ws: Workspace, stream=None):
    """Attention of drafted trees: query i of a sequence is node i, attending to the cache rows its list names and
    to the drafted rows on its path. ``cache`` is a ``QCache`` or a bf16 latent cache [B, max_len, d]; ``draft``
    bf16 [B, n_q, d]; ``parents`` int32 [B, n_q] (-1: child of the last committed token, < -1: absent node).
    Returns (out, lse) like ``sparse_mla_attn``."""
    device, out, lse = _attention_inputs(dims, q, idx, topk, stream)
    width = dims.d_latent + dims.d_rope
    _same("draft", draft, torch.bfloat16, dims.batch * dims.n_q * width, device)
    _same("parents", parents, torch.int32, dims.batch * dims.n_q, device)
    if isinstance(cache, QCache):
        dsa_tree_mla_attn_qcache(dims, q, cache._struct(dims, device), idx, topk, draft, parents, out, lse,
                                 _workspace(ws, device), stream)
    else:
        _same("cache", cache, torch.bfloat16, dims.batch * dims.max_len * width, device)
        dsa_tree_mla_attn(dims, q, cache, idx, topk, draft, parents, out, lse, _workspace(ws, device), stream)
    return out, lse


def dims_for(cfg) -> dsa_dims:
    """dsa_dims of a workload description with the fields of ``synthetic.DSAConfig``."""
    return make_dims(cfg.batch, cfg.n_q, cfg.max_len, cfg.n_idx_heads, cfg.idx_dim, cfg.n_heads, cfg.d_latent,
                     cfg.d_rope, cfg.softmax_scale)
