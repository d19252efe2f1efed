"""Python binding of libpkv.so: paged decode attention over a chunked-slab KV pool on
GB300 (sm_103a).

Argument marshalling only: every step runs in the library's CUDA kernels.  PyTorch
supplies device memory and streams (tensors are passed by ``data_ptr()`` and the
current stream's handle).  There is no CPU fallback: without the compiled library
every call raises.  Names follow the C ABI in ``include/pkv.h`` without the ``pkv_``
prefix.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpkv.so")

FORMATS = {"bf16": 0, "k4v4": 1, "k8v4": 2, "k8v8": 3, "latent": 4}
FORMAT_NAMES = {v: k for k, v in FORMATS.items()}
KIND_K, KIND_V, KIND_KMETA, KIND_VMETA = 0, 1, 2, 3

STATUS = {0: "ok", -1: "invalid argument", -2: "allocation failed", -3: "CUDA error",
          -4: "format mismatch", -5: "out of range", -6: "device error word set"}
PKV_OK, PKV_ERR_INVALID, PKV_ERR_OOM, PKV_ERR_CUDA, PKV_ERR_FORMAT, PKV_ERR_RANGE, PKV_ERR_DEVICE = \
    0, -1, -2, -3, -4, -5, -6
ERR_ROW, ERR_CTX, ERR_SLOT, ERR_TIMEOUT, ERR_POS, ERR_PATH = 1, 2, 4, 8, 16, 32
LATENT_HEAD = 128  # values of a head's expanded key (without its position part) and value


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        msg = f"{what}: {STATUS.get(status, status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class PoolConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("slab_blocks", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("format", ctypes.c_int32), ("max_slabs", ctypes.c_int32), ("hadamard_seed", ctypes.c_uint64)]


class Stats(ctypes.Structure):
    _fields_ = [("n_slabs", ctypes.c_int32), ("n_kinds", ctypes.c_int32),
                ("slab_append_events", ctypes.c_int64), ("rows_capacity", ctypes.c_int64),
                ("rows_in_use", ctypes.c_int64), ("bytes_reserved", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64 * 4)]

    def as_dict(self):
        return {"n_slabs": self.n_slabs, "n_kinds": self.n_kinds, "slab_append_events": self.slab_append_events,
                "rows_capacity": self.rows_capacity, "rows_in_use": self.rows_in_use,
                "bytes_reserved": self.bytes_reserved, "row_bytes": list(self.row_bytes)}


ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
RELEASE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)


class Request(ctypes.Structure):
    _fields_ = [("new_blocks", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("n_q", ctypes.c_int32), ("max_blocks", ctypes.c_int32)]


class Price(ctypes.Structure):
    _fields_ = [("slabs_to_append", ctypes.c_int32), ("free_rows", ctypes.c_int64),
                ("storage_bytes", ctypes.c_uint64), ("page_bytes", ctypes.c_uint64),
                ("fixed_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {k: int(getattr(self, k)) for k, _ in self._fields_}


class Allocator(ctypes.Structure):
    _fields_ = [("alloc", ALLOC_FN), ("release", RELEASE_FN), ("ctx", ctypes.c_void_p)]


# Every symbol of include/pkv.h with its ctypes signature.
_P, _I, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "pkv_pool_create": ([ctypes.POINTER(PoolConfig), ctypes.POINTER(Allocator), _P, ctypes.POINTER(_P)], _I),
    "pkv_pool_destroy": ([_P], None),
    "pkv_append_slab": ([_P, _I, _P], _I),
    "pkv_alloc_rows": ([_P, _I, _P, _P], _I),
    "pkv_retain_row": ([_P, ctypes.c_int32], _I),
    "pkv_release_row": ([_P, ctypes.c_int32], _I),
    "pkv_slab_runs": ([_P, _I, _I, _P], _I),
    "pkv_write_block": ([_P, _I, _I, _P, _P, _P, _P, _P], _I),
    "pkv_copy_on_write_block": ([_P, _I, _P, _P, _P], _I),
    "pkv_gather_visible": ([_P, _I, _P, _I, _P, _P, _P, _P, _P], _I),
    "pkv_decode_workspace_bytes": ([_P, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "pkv_paged_decode_attention": ([_P, _I, _I, _I, _P, _P, _I, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "pkv_paged_decode_attention_noalloc": ([_P, _I, _I, _I, _P, _P, _I, _P, _I, _F, _P, _P], _I),
    "pkv_decode_set_ctas": ([_P, _I], _I),
    "pkv_pool_stats": ([_P, ctypes.POINTER(Stats)], _I),
    "pkv_slab_address": ([_P, _I, _I, _I, ctypes.POINTER(_P)], _I),
    "pkv_pool_check_identity": ([_P, ctypes.POINTER(PoolConfig)], _I),
    "pkv_price_request": ([_P, ctypes.POINTER(Request), ctypes.POINTER(Price)], _I),
    "pkv_pool_check_errors": ([_P, _P, ctypes.POINTER(ctypes.c_int32)], _I),
    "pkv_pool_get_config": ([_P, ctypes.POINTER(PoolConfig)], _I),
    "pkv_prefill_workspace_bytes": ([_P, _I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "pkv_paged_prefill_attention": ([_P, _I, _I, _I, _I, _P, _P, _I, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "pkv_block_record_bytes": ([_P, ctypes.POINTER(_SZ)], _I),
    "pkv_export_blocks": ([_P, _I, _P, _P, _SZ, _P], _I),
    "pkv_import_blocks": ([_P, ctypes.POINTER(PoolConfig), _I, _P, _P, _SZ, _P], _I),
    "pkv_write_latent": ([_P, _I, _I, _P, _P, _P, _I64, _P, _P, _I, _P, _F, _I, _I, _P, _I64, _I64, _P, _I64, _I64,
                          _P], _I),
    "pkv_latent_workspace_bytes": ([_P, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "pkv_paged_latent_attention": ([_P, _I, _I, _I, _I, _P, _I64, _P, _I64, _P, _I, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "pkv_latent_prefill_workspace_bytes": ([_P, _I, _I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "pkv_price_latent_prefill": ([_P, ctypes.POINTER(Request), _I, ctypes.POINTER(Price)], _I),
    "pkv_latent_prefill_attention": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "pkv_write_rotated": ([_P, _I, _I, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I, _I, _I, _P, _P, _F, _I, _P,
                           _I64, _I64, _P, _I64, _I64, _P], _I),
    "pkv_tree_workspace_bytes": ([_P, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "pkv_paged_tree_attention": ([_P, _I, _I, _I, _I, _P, _P, _I64, _P, _I, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "pkv_accept_drafts": ([_P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P], _I),
    "pkv_status_string": ([_I], ctypes.c_char_p),
    "pkv_last_error": ([], ctypes.c_char_p),
}

_lock = threading.Lock()
_lib_handle = None


def lib():
    """The loaded libpkv.so (raises if it has not been built)."""
    global _lib_handle
    with _lock:
        if _lib_handle is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m paged_kv_cache_split_gb300.build` (nvcc, sm_103a)")
            h = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(h, name)
                fn.argtypes = args
                fn.restype = res
            _lib_handle = h
        return _lib_handle


def _check(status: int, what: str):
    if status != PKV_OK:
        detail = ""
        if status == PKV_ERR_CUDA:
            detail = lib().pkv_last_error().decode(errors="replace")
        raise PkvError(status, what, detail)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_raw_stream = None  # (device -> handle of its current stream, current device), once CUDA runs


def _stream(stream=None) -> int:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            torch = _torch()
            handle = torch.cuda.current_stream().cuda_stream  # initialises CUDA, or raises
            _raw_stream = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
            return handle
        return _raw_stream[0](_raw_stream[1]())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t, dtype, name: str, shape=None):
    try:
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _dev_strided(t, dtype, name: str, shape):
    """Like _dev, for a tensor whose last dimension alone has to be contiguous."""
    try:
        if t.is_cuda and t.dtype is dtype and t.shape == shape and t.stride(-1) == 1:
            return t.data_ptr()
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def _row_stride(t, name: str) -> int:
    """The one distance between consecutive rows (every leading dimension) of `t`."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 4:
        a, b, c, _ = shape
        sa, sb, sc, _ = strides
        if c > 1 and (b == 1 or sb == c * sc) and (a == 1 or sa == b * c * sc):
            return sc
    step, rows = None, 1
    for i in range(len(shape) - 2, -1, -1):
        n = shape[i]
        if n != 1:
            if step is None:
                step = strides[i]
            elif strides[i] != step * rows:
                raise ValueError(f"{name}: its rows must be evenly spaced (strides {strides})")
        rows *= n
    return shape[-1] if step is None else step


def slab_runs(rows, slab_blocks: int = 32) -> np.ndarray:
    """Start index of each maximal same-slab run of a block-table row list (host)."""
    r = np.ascontiguousarray(rows, np.int32)
    out = np.zeros(max(1, r.size), np.int32)
    n = lib().pkv_slab_runs(r.ctypes.data_as(_P), r.size, slab_blocks, out.ctypes.data_as(_P))
    if n < 0:
        raise PkvError(PKV_ERR_INVALID, "slab_runs")
    return out[:n].copy()


def tree_masks(parents):
    """Mask words and depths of trees given by parents (host): parents [..., n_q] holds each
    drafted token's parent, an earlier token of the tree, or a negative number for one that
    follows the context.  Returns (masks [..., n_q, ceil(n_q / 32)] int32, depths [..., n_q]
    int32): a token's mask names its ancestors and itself, and its position is that of the
    first drafted token plus its depth."""
    p = np.asarray(parents)
    if p.ndim < 1 or not np.issubdtype(p.dtype, np.integer):
        raise TypeError("parents must be integers, [..., n_q]")
    n = p.shape[-1]
    if n and (p >= np.arange(n)).any():
        raise ValueError("a token's parent comes before it")
    flat = p.reshape(int(np.prod(p.shape[:-1], dtype=np.int64)), n)
    masks = np.zeros((flat.shape[0], n, -(-n // 32)), np.uint32)
    depths = np.zeros(flat.shape, np.int32)
    every = np.arange(flat.shape[0])
    for i in range(n):
        up = flat[:, i]
        has = up >= 0
        masks[has, i] = masks[every[has], up[has]]
        depths[has, i] = depths[every[has], up[has]] + 1
        masks[:, i, i // 32] |= np.uint32(1 << i % 32)
    return masks.view(np.int32).reshape(*p.shape, masks.shape[-1]), depths.reshape(p.shape)


def make_config(n_layers: int, n_kv_heads: int, head_dim: int, format="bf16", hadamard_seed: int = 0,
                slab_blocks: int = 32, max_slabs: int = 1024, block_size: int = 32, group_size: int = 32):
    fmt = FORMATS[format] if isinstance(format, str) else int(format)
    return PoolConfig(n_layers, n_kv_heads, head_dim, block_size, slab_blocks, group_size, fmt, max_slabs,
                      hadamard_seed & (2**64 - 1))


class Pool:
    """A chunked-slab KV pool on the current CUDA device (see pkv_pool_create)."""

    def __init__(self, n_layers: int, n_kv_heads: int, head_dim: int, format="bf16", hadamard_seed: int = 0,
                 slab_blocks: int = 32, max_slabs: int = 1024, allocator: Optional[Allocator] = None,
                 stream=None, group_size: int = 32, rope_dim: Optional[int] = None):
        """For format "latent", n_kv_heads is 1, head_dim the latent vector's width and
        rope_dim (default 64) the position key's; the other formats take no rope_dim."""
        self._lib = lib()
        if FORMATS.get(format, format) == FORMATS["latent"]:
            group_size = 64 if rope_dim is None else rope_dim
        elif rope_dim is not None:
            raise ValueError("rope_dim belongs to the latent format")
        self.cfg = make_config(n_layers, n_kv_heads, head_dim, format, hadamard_seed, slab_blocks, max_slabs,
                               group_size=group_size)
        self.n_layers, self.n_kv_heads, self.head_dim = n_layers, n_kv_heads, head_dim
        self.format = FORMAT_NAMES[self.cfg.format]
        self.slab_blocks = slab_blocks
        self._allocator = allocator  # keep callbacks alive
        h = _P()
        st = self._lib.pkv_pool_create(ctypes.byref(self.cfg), ctypes.byref(allocator) if allocator else None,
                                       _stream(stream), ctypes.byref(h))
        _check(st, "pool_create")
        self._h = h
        self._ws = {}
        self._ws_bytes = {}  # workspace sizes of the latent and tree calls by their arguments
        self._latent_dims = (head_dim, int(group_size)) if self.format == "latent" else None
        self._device = _torch().cuda.current_device()
        s = self.stats()
        self.row_bytes = s["row_bytes"][: s["n_kinds"]]

    # -- lifetime ------------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            self._lib.pkv_pool_destroy(self._h)
            self._h = None
            self._ws = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # -- growth and rows -----------------------------------------------------
    def append_slab(self, n_slabs: int = 1, stream=None):
        _check(self._lib.pkv_append_slab(self._h, n_slabs, _stream(stream)), "append_slab")

    def reserve_rows(self, rows: int, stream=None):
        """Append slabs until the pool has at least `rows` rows."""
        have = self.stats()["rows_capacity"]
        if rows > have:
            self.append_slab(-(-(rows - have) // self.slab_blocks), stream)

    def alloc_rows(self, n: int, stream=None) -> np.ndarray:
        out = np.zeros(max(1, n), np.int32)
        _check(self._lib.pkv_alloc_rows(self._h, n, out.ctypes.data_as(_P), _stream(stream)), "alloc_rows")
        return out[:n].copy()

    def retain_row(self, row: int):
        _check(self._lib.pkv_retain_row(self._h, int(row)), "retain_row")

    def release_row(self, row: int):
        _check(self._lib.pkv_release_row(self._h, int(row)), "release_row")

    # -- data movement -------------------------------------------------------
    def write_block(self, layer: int, rows, slots, k, v, stream=None):
        torch = _torch()
        n = int(rows.numel())
        shape = (n, self.n_kv_heads, self.head_dim)
        _check(self._lib.pkv_write_block(self._h, layer, n, _dev(rows, torch.int32, "rows"),
                                         _dev(slots, torch.int32, "slots"), _dev(k, torch.bfloat16, "k", shape),
                                         _dev(v, torch.bfloat16, "v", shape), _stream(stream)), "write_block")

    def copy_on_write_block(self, src_rows, dst_rows, stream=None):
        torch = _torch()
        n = int(src_rows.numel())
        if int(dst_rows.numel()) != n:
            raise ValueError("src_rows and dst_rows differ in length")
        _check(self._lib.pkv_copy_on_write_block(self._h, n, _dev(src_rows, torch.int32, "src_rows"),
                                                 _dev(dst_rows, torch.int32, "dst_rows"), _stream(stream)),
               "copy_on_write_block")

    def gather_visible(self, layer: int, bt_row, ctx_len: int, stream=None):
        """Dense [Hkv, ctx, row_bytes] uint8 tensors (K, V[, K meta, V meta])."""
        torch = _torch()
        outs = [torch.empty((self.n_kv_heads, ctx_len, rb), dtype=torch.uint8, device=bt_row.device)
                for rb in self.row_bytes]
        ptrs = [o.data_ptr() for o in outs] + [None] * (4 - len(outs))
        _check(self._lib.pkv_gather_visible(self._h, layer, _dev(bt_row, torch.int32, "bt_row"), ctx_len,
                                            *ptrs, _stream(stream)), "gather_visible")
        return outs

    # -- block records (export / import) ---------------------------------------
    def config(self) -> PoolConfig:
        """The pool's configuration (storage identity, layer count, table size)."""
        c = PoolConfig()
        _check(self._lib.pkv_pool_get_config(self._h, ctypes.byref(c)), "pool_get_config")
        return c

    def block_record_bytes(self) -> int:
        n = _SZ()
        _check(self._lib.pkv_block_record_bytes(self._h, ctypes.byref(n)), "block_record_bytes")
        return int(n.value)

    def export_blocks(self, rows, out=None, stream=None):
        """[n, record_bytes] uint8 device tensor with the records of blocks `rows`."""
        torch = _torch()
        n, rec = int(rows.numel()), self.block_record_bytes()
        if out is None:
            out = torch.empty((n, rec), dtype=torch.uint8, device=rows.device)
        _check(self._lib.pkv_export_blocks(self._h, n, _dev(rows, torch.int32, "rows"),
                                           _dev(out, torch.uint8, "out"), out.numel(), _stream(stream)),
               "export_blocks")
        return out

    def import_blocks(self, identity: PoolConfig, rows, records, stream=None):
        """Write records (layout of export_blocks) into blocks `rows`; raises PkvError
        (status PKV_ERR_FORMAT) before any device work if `identity` differs."""
        torch = _torch()
        _check(self._lib.pkv_import_blocks(self._h, ctypes.byref(identity), int(rows.numel()),
                                           _dev(rows, torch.int32, "rows"), _dev(records, torch.uint8, "records"),
                                           records.numel(), _stream(stream)), "import_blocks")

    # -- attention -----------------------------------------------------------
    def decode_workspace_bytes(self, B: int, Hq: int, max_ctx: int = 0) -> int:
        n = _SZ()
        _check(self._lib.pkv_decode_workspace_bytes(self._h, B, Hq, max_ctx, ctypes.byref(n)),
               "decode_workspace_bytes")
        return int(n.value)

    def workspace(self, B: int, Hq: int, device=None):
        """A zero-filled workspace tensor for (B, Hq), cached on the pool."""
        torch = _torch()
        nbytes = self.decode_workspace_bytes(B, Hq)
        key = (B, Hq)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")
            self._ws[key] = ws
        return ws

    def decode_set_ctas(self, n_ctas: int):
        _check(self._lib.pkv_decode_set_ctas(self._h, n_ctas), "decode_set_ctas")
        self._ws = {}
        self._ws_bytes = {}

    def paged_decode_attention(self, layer: int, q, block_table, ctx_lens, scale: float, max_ctx: int = 0,
                               out=None, workspace=None, stream=None):
        torch = _torch()
        B, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError(f"q head_dim {D} != pool head_dim {self.head_dim}")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = self.workspace(B, Hq, q.device)
        _check(self._lib.pkv_paged_decode_attention(
            self._h, layer, B, Hq, _dev(q, torch.bfloat16, "q"), _dev(block_table, torch.int32, "block_table"),
            int(block_table.shape[1]), _dev(ctx_lens, torch.int32, "ctx_lens", (B,)), int(max_ctx), float(scale),
            _dev(out, torch.bfloat16, "out", (B, Hq, D)), workspace.data_ptr(), int(workspace.numel()),
            _stream(stream)), "paged_decode_attention")
        return out

    def prefill_workspace_bytes(self, B: int, n_q: int, Hq: int, max_blocks: int) -> int:
        n = _SZ()
        _check(self._lib.pkv_prefill_workspace_bytes(self._h, B, n_q, Hq, max_blocks, ctypes.byref(n)),
               "prefill_workspace_bytes")
        return int(n.value)

    def paged_prefill_attention(self, layer: int, q, block_table, ctx_lens, scale: float, max_ctx: int = 0,
                                out=None, workspace=None, stream=None):
        """Causal attention of the last n_q tokens of each sequence: q [B, n_q, Hq, D] bf16."""
        torch = _torch()
        B, n_q, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError(f"q head_dim {D} != pool head_dim {self.head_dim}")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        if out is None:
            out = torch.empty_like(q)
        mb = int(block_table.shape[1])
        if workspace is None:
            n = self.prefill_workspace_bytes(B, n_q, Hq, mb)
            workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
        _check(self._lib.pkv_paged_prefill_attention(
            self._h, layer, B, n_q, Hq, _dev(q, torch.bfloat16, "q"), _dev(block_table, torch.int32, "block_table"), mb,
            _dev(ctx_lens, torch.int32, "ctx_lens", (B,)), int(max_ctx), float(scale),
            _dev(out, torch.bfloat16, "out", (B, n_q, Hq, D)), workspace.data_ptr(), int(workspace.numel()),
            _stream(stream)), "paged_prefill_attention")
        return out

    def paged_decode_attention_noalloc(self, layer: int, q, block_table, ctx_lens, scale: float,
                                       max_ctx: int = 0, out=None, stream=None):
        """Decode attention with no workspace argument: the library's fixed device
        scratch array is used instead (see pkv_paged_decode_attention_noalloc)."""
        torch = _torch()
        B, Hq, D = q.shape
        if out is None:
            out = torch.empty_like(q)
        _check(self._lib.pkv_paged_decode_attention_noalloc(
            self._h, layer, B, Hq, _dev(q, torch.bfloat16, "q"), _dev(block_table, torch.int32, "block_table"),
            int(block_table.shape[1]), _dev(ctx_lens, torch.int32, "ctx_lens", (B,)), int(max_ctx), float(scale),
            _dev(out, torch.bfloat16, "out", (B, Hq, D)), _stream(stream)), "paged_decode_attention_noalloc")
        return out

    # -- latent pools ----------------------------------------------------------
    def _latent(self):
        if self._latent_dims is None:
            raise PkvError(PKV_ERR_FORMAT, f"a {self.format} pool has no latent rows")
        return self._latent_dims

    def _same_device(self, *tensors):
        """The kernels run on the pool's device and reach no other's memory."""
        for t in tensors:
            if t is not None and t.get_device() != self._device:
                raise ValueError(f"a tensor on {t.device}, the pool is on cuda:{self._device}")

    def write_latent(self, layer: int, rows, slots, kv, positions, cos_sin, norm_weight=None, eps: float = 1e-6,
                     interleaved: bool = True, q_rope=None, q_out=None, stream=None):
        """Store token i's row kv[i] = (latent, position key) at (rows[i], slots[i]): the latent
        normalised (with norm_weight), the position key turned by the angles of positions[i];
        q_rope [n, Hq, P] is turned by the same angles into q_out (which may be q_rope; a new
        tensor by default).  kv may have any row stride, q_rope and q_out any token and head
        strides, in multiples of 8 values.  Tokens of one call have places of their own: two at
        one place leave a mix of both.  Returns q_out (None without q_rope)."""
        torch = _torch()
        R, P = self._latent()
        bf16, i32 = torch.bfloat16, torch.int32
        n = rows.numel()
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, P]")
        one = (n,)
        kvp = _dev_strided(kv, bf16, "kv", (n, R + P))
        Hq, q, o = 0, None, None
        qt = qh = ot = oh = 0  # a dimension of one entry is never stepped over: its stride says nothing
        if q_rope is not None:
            if q_rope.dim() != 3:
                raise ValueError("q_rope must be [n, Hq, P]")
            Hq = q_rope.shape[1]
            shape = (n, Hq, P)
            if q_out is None:
                q_out = self._own(shape, bf16, q_rope.device, stream)
            q, o = _dev_strided(q_rope, bf16, "q_rope", shape), _dev_strided(q_out, bf16, "q_out", shape)
            if n > 1:
                qt, ot = q_rope.stride(0), q_out.stride(0)
            if Hq > 1:
                qh, oh = q_rope.stride(1), q_out.stride(1)
        elif q_out is not None:
            raise ValueError("q_out without q_rope")
        self._same_device(rows, slots, kv, positions, cos_sin, norm_weight, q_rope, q_out)
        n_pos = cos_sin.shape[0]
        st = self._lib.pkv_write_latent(
            self._h, layer, n, _dev(rows, i32, "rows", one), _dev(slots, i32, "slots", one), kvp,
            kv.stride(0) if n > 1 else R + P, _dev(positions, i32, "positions", one),
            _dev(cos_sin, torch.float32, "cos_sin", (n_pos, P)), n_pos,
            None if norm_weight is None else _dev(norm_weight, bf16, "norm_weight", (R,)), float(eps),
            1 if interleaved else 0, Hq, q, qt, qh, o, ot, oh, _stream(stream))
        if st:
            _check(st, "write_latent")
        return q_out

    def latent_workspace_bytes(self, B: int, n_q: int, Hq: int) -> int:
        n = _SZ()
        _check(self._lib.pkv_latent_workspace_bytes(self._h, B, n_q, Hq, ctypes.byref(n)), "latent_workspace_bytes")
        return int(n.value)

    def paged_latent_attention(self, layer: int, q_latent, q_rope, block_table, ctx_lens, scale: float,
                               max_ctx: int = 0, out=None, workspace=None, stream=None):
        """Absorbed attention over the latent rows: q_latent [B, Hq, R] and q_rope [B, Hq, P], or
        [B, n_q, Hq, .] for the n_q newest tokens of each sequence, any even row stride (views
        of one [.., R + P] tensor, for instance).  Returns out, shaped as q_latent."""
        torch = _torch()
        R, P = self._latent()
        bf16, i32 = torch.bfloat16, torch.int32
        lead = tuple(q_latent.shape)[:-1]
        if len(lead) == 3:
            B, n_q, Hq = lead
        elif len(lead) == 2:
            (B, Hq), n_q = lead, 1
        else:
            raise ValueError("q_latent must be [B, Hq, R] or [B, n_q, Hq, R]")
        rows = lead + (R,)
        ql = _dev_strided(q_latent, bf16, "q_latent", rows)
        qr = _dev_strided(q_rope, bf16, "q_rope", lead + (P,))
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        self._same_device(q_latent, q_rope, block_table, ctx_lens, out, workspace)
        if out is None:
            out = self._own(rows, bf16, q_latent.device, stream)
            o = out.data_ptr()
        else:
            o = _dev(out, bf16, "out", rows)
        if workspace is None:
            key = (B, n_q, Hq)
            need = self._ws_bytes.get(key)
            if need is None:
                need = self._keep_size(key, self.latent_workspace_bytes(B, n_q, Hq))
            workspace = self._own(need, torch.uint8, q_latent.device, stream)
        st = self._lib.pkv_paged_latent_attention(
            self._h, layer, B, n_q, Hq, ql, _row_stride(q_latent, "q_latent"), qr, _row_stride(q_rope, "q_rope"),
            _dev(block_table, i32, "block_table"), block_table.shape[1], _dev(ctx_lens, i32, "ctx_lens", (B,)),
            int(max_ctx), float(scale), o, _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
        if st:
            _check(st, "paged_latent_attention")
        return out

    def latent_prefill_workspace_bytes(self, B: int, n_q: int, Hq: int, max_blocks: int, max_ctx: int = 0) -> int:
        n = _SZ()
        _check(self._lib.pkv_latent_prefill_workspace_bytes(self._h, B, n_q, Hq, max_blocks, max_ctx, ctypes.byref(n)),
               "latent_prefill_workspace_bytes")
        return int(n.value)

    def latent_prefill_attention(self, layer: int, q, w_k, w_v, block_table, ctx_lens, scale: float, max_ctx: int = 0,
                                 out=None, workspace=None, stream=None):
        """Expanded causal attention of the n_q newest tokens of each sequence: q [B, n_q, Hq,
        128 + P], w_k and w_v [Hq, 128, R]; max_ctx bounds ctx_lens and sizes the workspace.
        Returns out [B, n_q, Hq, 128]."""
        torch = _torch()
        R, P = self._latent()
        D = LATENT_HEAD
        if q.dim() != 4:
            raise ValueError("q must be [B, n_q, Hq, 128 + P]")
        B, n_q, Hq = (int(x) for x in q.shape[:3])
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        mb = int(block_table.shape[1])
        self._same_device(q, w_k, w_v, block_table, ctx_lens, out, workspace)
        if out is None:
            out = self._own((B, n_q, Hq, D), torch.bfloat16, q.device, stream)
        if workspace is None:
            key = (B, n_q, Hq, mb, int(max_ctx))
            need = self._ws_bytes.get(key)
            if need is None:
                need = self._keep_size(key, self.latent_prefill_workspace_bytes(*key))
            workspace = self._own(need, torch.uint8, q.device, stream)
        _check(self._lib.pkv_latent_prefill_attention(
            self._h, layer, B, n_q, Hq, _dev(q, torch.bfloat16, "q", (B, n_q, Hq, D + P)),
            _dev(w_k, torch.bfloat16, "w_k", (Hq, D, R)), _dev(w_v, torch.bfloat16, "w_v", (Hq, D, R)),
            _dev(block_table, torch.int32, "block_table"), mb, _dev(ctx_lens, torch.int32, "ctx_lens", (B,)),
            int(max_ctx), float(scale), _dev(out, torch.bfloat16, "out", (B, n_q, Hq, D)),
            _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "latent_prefill_attention")
        return out

    # -- drafted tokens --------------------------------------------------------
    def write_rotated(self, layer: int, rows, slots, k, v, positions, cos_sin, q=None, k_norm=None, q_norm=None,
                      eps: float = 1e-6, interleaved: bool = False, q_out=None, stream=None):
        """Store token i's keys k[i], normalised (with k_norm) and turned by the angles of
        positions[i], and its values v[i] at (rows[i], slots[i]); a packed pool quantises them.  The
        queries q [n, Hq, D] are normalised (q_norm) and turned likewise into q_out (which may be
        q; a new tensor by default).  cos_sin is [positions, rotary_dim]: the first rotary_dim
        values of a head are turned.  k, v, q and q_out may have any token and head strides, in
        multiples of 8 values.  Returns q_out (None without q)."""
        torch = _torch()
        bf16, i32 = torch.bfloat16, torch.int32
        n, Hk, D = rows.numel(), self.n_kv_heads, self.head_dim
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, rotary_dim]")
        one, kv = (n,), (n, Hk, D)
        kp, vp = _dev_strided(k, bf16, "k", kv), _dev_strided(v, bf16, "v", kv)
        # a dimension of one entry is never stepped over: its stride says nothing
        (kt, kh, _), (vt, vh, _) = k.stride(), v.stride()
        if n < 2:
            kt = vt = 0
        if Hk < 2:
            kh = vh = 0
        Hq, qp, op = 0, None, None
        qt = qh = ot = oh = 0
        if q is not None:
            if q.dim() != 3:
                raise ValueError("q must be [n, Hq, head_dim]")
            Hq = q.shape[1]
            shape = (n, Hq, D)
            if q_out is None:
                q_out = self._own(shape, bf16, q.device, stream)
            qp, op = _dev_strided(q, bf16, "q", shape), _dev_strided(q_out, bf16, "q_out", shape)
            (qt, qh, _), (ot, oh, _) = q.stride(), q_out.stride()
            if n < 2:
                qt = ot = 0
            if Hq < 2:
                qh = oh = 0
        elif q_out is not None or q_norm is not None:
            raise ValueError("q_out or q_norm without q")
        self._same_device(rows, slots, k, v, positions, cos_sin, q, k_norm, q_norm, q_out)
        n_pos, rot = cos_sin.shape
        st = self._lib.pkv_write_rotated(
            self._h, layer, n, _dev(rows, i32, "rows", one), _dev(slots, i32, "slots", one), kp, kt, kh, vp, vt, vh,
            _dev(positions, i32, "positions", one), _dev(cos_sin, torch.float32, "cos_sin"), n_pos, rot,
            1 if interleaved else 0, None if k_norm is None else _dev(k_norm, bf16, "k_norm", (D,)),
            None if q_norm is None else _dev(q_norm, bf16, "q_norm", (D,)), float(eps), Hq, qp, qt, qh, op, ot, oh,
            _stream(stream))
        if st:
            _check(st, "write_rotated")
        return q_out

    def tree_workspace_bytes(self, B: int, n_q: int, Hq: int) -> int:
        n = _SZ()
        _check(self._lib.pkv_tree_workspace_bytes(self._h, B, n_q, Hq, ctypes.byref(n)), "tree_workspace_bytes")
        return int(n.value)

    def paged_tree_attention(self, layer: int, q, tree_mask, block_table, ctx_lens, scale: float, max_ctx: int = 0,
                             out=None, workspace=None, stream=None):
        """Attention of each sequence's last n_q tokens, drafted as a tree: q [B, n_q, Hq, D], contiguous;
        tree_mask int32 [B, n_q, ceil(n_q / 32)], or [n_q, ceil(n_q / 32)] for one tree in all
        sequences (tree_masks makes them from parents).  Query i sees every token before the
        drafted ones and drafted token j where bit j of its mask row is set.  Returns out, shaped
        as q."""
        torch = _torch()
        bf16, i32 = torch.bfloat16, torch.int32
        if q.dim() != 4:
            raise ValueError("q must be [B, n_q, Hq, head_dim]")
        B, n_q, Hq, D = q.shape
        if D != self.head_dim:
            raise ValueError(f"q head_dim {D} != pool head_dim {self.head_dim}")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        words = -(-n_q // 32)
        shared = tree_mask.dim() == 2
        maskp = _dev(tree_mask, i32, "tree_mask", (n_q, words) if shared else (B, n_q, words))
        qp = _dev(q, bf16, "q")
        self._same_device(q, tree_mask, block_table, ctx_lens, out, workspace)
        if out is None:
            out = self._own(q.shape, bf16, q.device, stream)
            o = out.data_ptr()
        else:
            o = _dev(out, bf16, "out", q.shape)
        if workspace is None:
            key = ("tree", B, n_q, Hq)
            need = self._ws_bytes.get(key)
            if need is None:
                need = self._keep_size(key, self.tree_workspace_bytes(B, n_q, Hq))
            workspace = self._own(need, torch.uint8, q.device, stream)
        st = self._lib.pkv_paged_tree_attention(
            self._h, layer, B, n_q, Hq, qp, maskp, 0 if shared else n_q * words,
            _dev(block_table, i32, "block_table"), block_table.shape[1], _dev(ctx_lens, i32, "ctx_lens", (B,)),
            int(max_ctx), float(scale), o, _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
        if st:
            _check(st, "paged_tree_attention")
        return out

    def accept_drafts(self, path, path_lens, block_table, ctx_lens, n_q: int, new_lens=None, stream=None):
        """Move the drafted tokens of each sequence's accepted path, path[b, :path_lens[b]] (rising
        indices of its n_q drafted tokens), to the places behind the tokens before them, in
        every layer.  Returns the new lengths [B] int32 (new_lens, or a new tensor)."""
        torch = _torch()
        i32 = torch.int32
        B = path_lens.numel()
        if path.dim() != 2 or path.shape[0] != B:
            raise ValueError("path must be [B, max_path]")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        self._same_device(path, path_lens, block_table, ctx_lens, new_lens)
        if new_lens is None:
            new_lens = self._own((B,), i32, ctx_lens.device, stream)
        _check(self._lib.pkv_accept_drafts(
            self._h, B, int(n_q), path.shape[1], _dev(path, i32, "path"), _dev(path_lens, i32, "path_lens", (B,)),
            _dev(block_table, i32, "block_table"), block_table.shape[1], _dev(ctx_lens, i32, "ctx_lens", (B,)),
            _dev(new_lens, i32, "new_lens", (B,)), _stream(stream)), "accept_drafts")
        return new_lens

    def _keep_size(self, key, nbytes: int) -> int:
        """Sizes are kept for the next call with the same arguments: 1024 at most, as
        batches and bounds of a long-running server differ from step to step."""
        if len(self._ws_bytes) >= 1024:
            self._ws_bytes = {}
        self._ws_bytes[key] = nbytes
        return nbytes

    @staticmethod
    def _own(shape, dtype, device, stream):
        """Memory of one call alone (its output, its workspace): two calls on two streams, or in
        two captured graphs, share none."""
        torch = _torch()
        t = torch.empty(shape, dtype=dtype, device=device)
        if stream is not None:
            # made on the current stream, used on another
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream))
            if s != torch.cuda.current_stream():
                s.wait_stream(torch.cuda.current_stream())
                t.record_stream(s)
        return t

    # -- introspection -------------------------------------------------------
    def stats(self) -> dict:
        s = Stats()
        _check(self._lib.pkv_pool_stats(self._h, ctypes.byref(s)), "pool_stats")
        return s.as_dict()

    def slab_address(self, layer: int, kind: int, slab: int) -> int:
        a = _P()
        _check(self._lib.pkv_slab_address(self._h, layer, kind, slab, ctypes.byref(a)), "slab_address")
        return int(a.value or 0)

    def price_request(self, new_blocks: int, B: int, Hq: int, n_q: int = 1, max_blocks: int = 0) -> dict:
        """Admission price of a request (see pkv_price_request): slabs to append, free
        rows, and the storage, page, fixed and workspace bytes."""
        req = Request(int(new_blocks), int(B), int(Hq), int(n_q), int(max_blocks))
        out = Price()
        _check(self._lib.pkv_price_request(self._h, ctypes.byref(req), ctypes.byref(out)), "price_request")
        return out.as_dict()

    def price_latent_prefill(self, new_blocks: int, B: int, Hq: int, n_q: int, max_blocks: int, max_ctx: int = 0) -> dict:
        """price_request for a step in expanded form (see pkv_price_latent_prefill)."""
        req = Request(int(new_blocks), int(B), int(Hq), int(n_q), int(max_blocks))
        out = Price()
        _check(self._lib.pkv_price_latent_prefill(self._h, ctypes.byref(req), int(max_ctx), ctypes.byref(out)),
               "price_latent_prefill")
        return out.as_dict()

    def check_identity(self, cfg: PoolConfig) -> bool:
        st = self._lib.pkv_pool_check_identity(self._h, ctypes.byref(cfg))
        if st == PKV_ERR_FORMAT:
            return False
        _check(st, "pool_check_identity")
        return True

    def check_errors(self, stream=None) -> int:
        """Synchronise, then return and clear the device error word (0 if clean)."""
        w = ctypes.c_int32(0)
        st = self._lib.pkv_pool_check_errors(self._h, _stream(stream), ctypes.byref(w))
        if st not in (PKV_OK, PKV_ERR_DEVICE):
            _check(st, "pool_check_errors")
        return int(w.value)


def pool_create(*args, **kw) -> Pool:
    return Pool(*args, **kw)
