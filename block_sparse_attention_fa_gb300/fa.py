"""Thin ctypes binding over the C ABI in ``include/fa.h`` and
``include/fa_paged.h``.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``_lib/libfa_gb300.so``.  PyTorch supplies device memory and the
current stream.  If the library is missing or fails to load this module
raises; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libfa_gb300.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE_CHECK = range(6)
BF16, FP32 = 0, 1
MASK_KINDS = {"full": 0, "causal": 1, "sliding_window": 2, "document": 3, "prefix_lm": 4, "table": 5,
              "sink_window": 6}
SCORE_KINDS = {"none": 0, "softcap": 1, "alibi": 2, "rel_bias": 3, "alibi_softcap": 4}
OUT_FP32 = 1
DEBUG_DROP_FIRST_LOAD = 1
BLOCK = 128

SYMBOLS = ("fa_workspace_bytes", "fa_block_mask_shape", "fa_block_mask_size", "fa_block_mask_build", "fa_fwd",
           "fa_fwd_noalloc", "fa_fwd_decode", "fa_decode_partials_bytes", "fa_decode_splits", "fa_bwd",
           "fa_block_mask_build_cols", "fa_bwd_rowstats_bytes", "fa_workspace_check", "fa_last_error", "fa_version")

PAGED_SYMBOLS = ("fa_kv_append", "fa_fwd_paged", "fa_paged_scratch_bytes", "fa_kv_append_scaled", "fa_fwd_paged_scaled",
                 "fa_paged_step")


class FAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"fa status {status}: {msg}")
        self.status = status


class MaskDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("window", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
                ("seg_batch", ctypes.c_int32), ("seg_ids", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_batch", ctypes.c_int32)]


class BlockMaskStruct(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("block_q", ctypes.c_int32), ("block_kv", ctypes.c_int32),
                ("nq", ctypes.c_int32), ("nkv", ctypes.c_int32),
                ("kv_num_blocks", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("full_kv_num_blocks", ctypes.c_void_p), ("full_kv_indices", ctypes.c_void_p),
                ("mask", MaskDesc)]


class ScoreDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("rel_bias", ctypes.c_void_p), ("rel_max", ctypes.c_int32)]


class FwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("q_len", ctypes.c_int32), ("kv_len", ctypes.c_int32),
                ("D", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("timeout_ms", ctypes.c_uint32), ("flags", ctypes.c_uint32),
                ("debug_flags", ctypes.c_uint32)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("D", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("dout", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("dq", ctypes.c_void_p),
                ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p), ("rowstats", ctypes.c_void_p),
                ("timeout_ms", ctypes.c_uint32)]


class BlockMaskColsStruct(ctypes.Structure):
    _fields_ = [("q_num_blocks", ctypes.c_void_p), ("q_indices", ctypes.c_void_p),
                ("full_q_num_blocks", ctypes.c_void_p), ("full_q_indices", ctypes.c_void_p)]


# The paged calls' structs are packed by these (a ctypes structure costs some
# microseconds to fill); the layouts are those of the classes below.
_PAGED_KV = struct.Struct("7i5P")
_KV_APPEND = struct.Struct("4i4P8q3P")
_PAGED_FWD = struct.Struct("3ifP2q2P2I")
_PAGED_SCALES = struct.Struct("2P")
_PAGED_STEP = struct.Struct("6i11P")
_MASK = struct.Struct("4i2Pi0P")
_SCORE = struct.Struct("if2Pi0P")


class PagedKVStruct(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


class KVAppendArgs(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("rope_len", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 2),
                ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2),
                ("q_out_stride", ctypes.c_int64 * 2), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


class PagedFwdArgs(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("max_q_len", ctypes.c_int32), ("shared_len", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 2),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("timeout_ms", ctypes.c_uint32),
                ("flags", ctypes.c_uint32)]


class PagedScales(ctypes.Structure):
    _fields_ = [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class PagedStepArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("shared_pages", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("new_len", ctypes.c_void_p), ("keep_len", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
                ("kv_len_out", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run `python -m block_sparse_attention_fa_gb300.build`)")
    h = ctypes.CDLL(path)
    h.fa_workspace_bytes.restype = ctypes.c_size_t
    h.fa_workspace_bytes.argtypes = []
    h.fa_block_mask_shape.restype = ctypes.c_int
    h.fa_block_mask_shape.argtypes = [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_int32)] * 2 + \
        [ctypes.POINTER(ctypes.c_int64)]
    h.fa_block_mask_size.restype = ctypes.c_int
    h.fa_block_mask_size.argtypes = [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_int32)] * 2 + \
        [ctypes.POINTER(ctypes.c_size_t)]
    h.fa_block_mask_build.restype = ctypes.c_int
    h.fa_block_mask_build.argtypes = [ctypes.POINTER(BlockMaskStruct), ctypes.c_void_p, ctypes.c_void_p]
    h.fa_fwd.restype = ctypes.c_int
    h.fa_fwd.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(BlockMaskStruct),
                         ctypes.POINTER(ScoreDesc), ctypes.c_void_p, ctypes.c_void_p]
    h.fa_fwd_noalloc.restype = ctypes.c_int
    h.fa_fwd_noalloc.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(BlockMaskStruct),
                                 ctypes.POINTER(ScoreDesc), ctypes.c_void_p]
    h.fa_fwd_decode.restype = ctypes.c_int
    h.fa_fwd_decode.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(BlockMaskStruct),
                                ctypes.POINTER(ScoreDesc), ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p, ctypes.c_void_p]
    h.fa_decode_partials_bytes.restype = ctypes.c_size_t
    h.fa_decode_partials_bytes.argtypes = [ctypes.POINTER(FwdArgs), ctypes.c_int32]
    h.fa_decode_splits.restype = ctypes.c_int32
    h.fa_decode_splits.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(BlockMaskStruct)]
    h.fa_block_mask_build_cols.restype = ctypes.c_int
    h.fa_block_mask_build_cols.argtypes = [ctypes.POINTER(BlockMaskStruct), ctypes.POINTER(BlockMaskColsStruct),
                                           ctypes.c_void_p, ctypes.c_void_p]
    h.fa_bwd_rowstats_bytes.restype = ctypes.c_size_t
    h.fa_bwd_rowstats_bytes.argtypes = [ctypes.c_int32] * 3
    h.fa_bwd.restype = ctypes.c_int
    h.fa_bwd.argtypes = [ctypes.POINTER(BwdArgs), ctypes.POINTER(BlockMaskStruct),
                         ctypes.POINTER(BlockMaskColsStruct), ctypes.POINTER(ScoreDesc), ctypes.c_void_p,
                         ctypes.c_void_p]
    h.fa_kv_append.restype = ctypes.c_int
    h.fa_kv_append.argtypes = [ctypes.c_void_p] * 4
    h.fa_paged_scratch_bytes.restype = ctypes.c_size_t
    h.fa_paged_scratch_bytes.argtypes = [ctypes.c_void_p] * 2
    h.fa_fwd_paged.restype = ctypes.c_int
    h.fa_fwd_paged.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2
    h.fa_kv_append_scaled.restype = ctypes.c_int
    h.fa_kv_append_scaled.argtypes = [ctypes.c_void_p] * 5
    h.fa_fwd_paged_scaled.restype = ctypes.c_int
    h.fa_fwd_paged_scaled.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2
    h.fa_paged_step.restype = ctypes.c_int
    h.fa_paged_step.argtypes = [ctypes.c_void_p] * 3
    h.fa_internal_capture_id.restype = ctypes.c_uint64
    h.fa_internal_capture_id.argtypes = [ctypes.c_void_p]
    h.fa_internal_capture_mode.restype = ctypes.c_int
    h.fa_internal_capture_mode.argtypes = [ctypes.c_int]
    h.fa_workspace_check.restype = ctypes.c_int
    h.fa_workspace_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    h.fa_last_error.restype = ctypes.c_char_p
    h.fa_last_error.argtypes = []
    h.fa_version.restype = ctypes.c_char_p
    h.fa_version.argtypes = []
    _lib = h
    return h


def _check(status: int):
    if status != OK:
        raise FAError(status, load_library().fa_last_error().decode())


_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)

# The current device and stream without building Python objects for them (a
# microsecond or two each, as much as a small kernel); the public calls where
# these are missing.
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda idx: torch.cuda.current_stream(idx).cuda_stream)


def _stream_ptr(stream) -> Optional[int]:
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Workspace:
    """fa_workspace_bytes() zero-filled device bytes for status flags."""

    def __init__(self, device=None, tensor: Optional[torch.Tensor] = None):
        if tensor is None:
            tensor = torch.zeros(load_library().fa_workspace_bytes(), dtype=torch.uint8, device=device or "cuda")
        self.tensor = tensor
        self.graphs = []          # a default workspace: those of the graphs captured on its stream

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    def check(self, stream=None):
        """Synchronise and raise FAError if a kernel flagged a device-side failure."""
        for ws in (self, *self.graphs):
            _check(load_library().fa_workspace_check(ws.ptr, _stream_ptr(stream)))


_default_ws = {}
_ws_slots = {}
_ws_lock = threading.Lock()
_WS_SLOTS = 64
_CAPTURE_RELAXED = 2           # cudaStreamCaptureModeRelaxed


def default_workspace(device, stream=None) -> Workspace:
    """The binding's workspace for (device, stream).  Launches that may run
    concurrently must not share a workspace (the forward keeps its work
    queue there), so each stream gets its own, and each graph that is captured
    on it: graphs may be replayed at once.  The stream's check() covers those of
    its graphs."""
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    raw = _raw_stream(idx) if stream is None else stream.cuda_stream
    return _workspace_of(idx, raw, _capture_of(idx, raw, stream is not None))


def _capture_of(idx: int, raw: int, other: bool) -> int:
    """The capture that a call on the stream becomes part of (0: none).  ``other``: not the current device's current
    stream."""
    if not other and not _capturing() and idx == _device_now():
        return 0
    return load_library().fa_internal_capture_id(raw)


def _workspace_of(idx: int, raw: int, capture: int) -> Workspace:
    ws = _default_ws.get((idx, raw, capture))
    if ws is None:
        with _ws_lock:
            ws = _default_ws.get((idx, raw, 0))
            if ws is None:
                ws = _default_ws[(idx, raw, 0)] = Workspace(tensor=_ws_slot(idx))
            if capture:
                eager, ws = ws, _default_ws.get((idx, raw, capture))
                if ws is None:
                    ws = _default_ws[(idx, raw, capture)] = Workspace(tensor=_ws_slot(idx))
                    eager.graphs.append(ws)
    return ws


def _ws_slot(idx: int) -> torch.Tensor:
    """A zero-filled piece for one workspace.  They are made several at a time and filled before they are handed out,
    outside any capture, since no fill on one stream comes before a launch on another."""
    free = _ws_slots.setdefault(idx, [])
    if not free:
        lib = load_library()
        with torch.cuda.device(idx):
            while True:                            # (streams come round, and this one might be in a capture)
                side = torch.cuda.Stream(idx)
                if not lib.fa_internal_capture_id(side.cuda_stream):
                    break
            mode = lib.fa_internal_capture_mode(_CAPTURE_RELAXED)
            try:
                with torch.cuda.stream(side):
                    slab = torch.zeros((_WS_SLOTS, lib.fa_workspace_bytes()), dtype=torch.uint8,
                                       device=torch.device("cuda", idx))
                side.synchronize()
            finally:
                lib.fa_internal_capture_mode(mode)
        free.extend(slab.unbind(0))
    return free.pop()


def _launch(device: torch.device, stream, workspace):
    """The workspace's address and the stream of a call on tensors of ``device``."""
    if stream is None and device.index == _device_now():
        raw = _raw_stream(device.index)
        if workspace is None:
            workspace = _workspace_of(device.index, raw, _capture_of(device.index, raw, False))
        return workspace.tensor.data_ptr(), raw
    if workspace is None:
        workspace = default_workspace(device, stream)
    return workspace.tensor.data_ptr(), _raw_stream(_device_now()) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """An output or scratch of a call on ``stream`` (None: the current one).  Memory of another stream is that
    stream's: what the current one still does with the block's last tenant must not reach it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    now = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(now)                          # where the caller goes on with it
    return t


class _IndexArrays:
    """The two count and two index arrays of a (transposed) BlockMask in one allocation: four would take longer to
    allocate than the arrays of a short sequence take to build.  Each starts on a 16-byte boundary."""

    def __init__(self, counts, indices, device, stream):
        self.shapes = (counts, indices, counts, indices)
        at = [0]
        for s in self.shapes:
            at.append(at[-1] + (math.prod(s) + 3) // 4 * 4)
        self.at = at
        self.buf = _new((at[-1],), torch.int32, device, stream)
        base = self.buf.data_ptr()
        self.ptrs = [base + 4 * x for x in at[:-1]]

    def __getitem__(self, k) -> torch.Tensor:
        return self.buf[self.at[k]:self.at[k] + math.prod(self.shapes[k])].view(self.shapes[k])


class BlockMask:
    """A BlockMask over 128 x 128 tiles (device int32 arrays + the mask_mod)."""

    kv_num_blocks = property(lambda self: self._arrays[0])
    kv_indices = property(lambda self: self._arrays[1])
    full_kv_num_blocks = property(lambda self: self._arrays[2])
    full_kv_indices = property(lambda self: self._arrays[3])

    def __init__(self, B, H, q_len, kv_len, mask, window, prefix_len, seg_ids, device, table=None, stream=None):
        if min(B, H, q_len, kv_len) < 1:          # the library says what is wrong
            _check(load_library().fa_block_mask_shape(B, H, q_len, kv_len, None, None, None))
        self.B, self.H, self.q_len, self.kv_len = B, H, q_len, kv_len
        self.nq, self.nkv = -(-q_len // BLOCK), -(-kv_len // BLOCK)
        self.mask, self.window, self.prefix_len = mask, window, prefix_len
        self.seg_ids = seg_ids
        self.table = table
        self._arrays = _IndexArrays((B, H, self.nq), (B, H, self.nq, self.nkv), device, stream)
        self.device = self._arrays.buf.device
        self._cols = None
        s = BlockMaskStruct()
        s.B, s.H, s.q_len, s.kv_len = B, H, q_len, kv_len
        s.block_q = s.block_kv = BLOCK
        s.nq, s.nkv = self.nq, self.nkv
        s.kv_num_blocks, s.kv_indices, s.full_kv_num_blocks, s.full_kv_indices = self._arrays.ptrs
        m = s.mask
        m.kind, m.window, m.prefix_len = MASK_KINDS[mask], window, prefix_len
        if seg_ids is not None:
            m.seg_batch, m.seg_ids = seg_ids.shape[0], seg_ids.data_ptr()
        if table is not None:
            m.table_batch, m.table = table.shape[0], table.data_ptr()
        self.struct = s

    def rebuild(self, stream=None, workspace: Optional["Workspace"] = None):
        """Run fa_block_mask_build again into this BlockMask's own buffers
        (e.g. after the segment ids changed in place); capturable in a CUDA
        graph since it allocates nothing."""
        ws, raw = _launch(self.device, stream, workspace)
        _check(load_library().fa_block_mask_build(ctypes.byref(self.struct), ws, raw))
        return self

    def cols(self, stream=None, workspace: Optional["Workspace"] = None, rebuild: bool = False) -> dict:
        """The transposed lists (fa_block_mask_build_cols: the q-blocks that
        visit each kv block), built on first use and kept with the mask."""
        self._build_cols(stream, workspace, rebuild)
        return {name: self._cols[k] for k, (name, _) in enumerate(BlockMaskColsStruct._fields_)}

    def _build_cols(self, stream, workspace, rebuild=False):
        if self._cols is None or rebuild:
            if self._cols is None:
                self._cols = _IndexArrays((self.B, self.H, self.nkv), (self.B, self.H, self.nkv, self.nq), self.device,
                                          stream)
                self._cols_struct = BlockMaskColsStruct(*self._cols.ptrs)
            ws, raw = _launch(self.device, stream, workspace)
            _check(load_library().fa_block_mask_build_cols(ctypes.byref(self.struct), ctypes.byref(self._cols_struct),
                                                           ws, raw))

    def visited_tiles(self) -> int:
        return int(self.kv_num_blocks.sum().item() + self.full_kv_num_blocks.sum().item())

    def numpy(self) -> dict:
        return {k: getattr(self, k).cpu().numpy() for k in
                ("kv_num_blocks", "kv_indices", "full_kv_num_blocks", "full_kv_indices")}


def block_mask(mask: str, B: int, H: int, q_len: int, kv_len: int, *, window: int = 0, prefix_len: int = 0,
               seg_ids: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None, device=None,
               stream=None, workspace: Optional[Workspace] = None, sinks: int = 0) -> BlockMask:
    """Build a BlockMask (fa_block_mask_build) for a built-in mask_mod.

    mask "sink_window": causal, and a key is visible while i - j <= ``window``
    or j < ``sinks`` (the C ABI's prefix_len).

    mask "table": ``table`` is the packed lookup table of the C ABI, a CUDA
    int32 tensor [table_batch, q_len, ceil(kv_len / 32)] whose bit j % 32 of
    word j // 32 in row i says whether query i attends to key j."""
    if table is not None:
        if table.dim() == 2:
            table = table[None]
        if table.dtype != torch.int32 or not table.is_cuda or tuple(table.shape[1:]) != (q_len, (kv_len + 31) // 32):
            raise ValueError("table must be a CUDA int32 tensor [batch, q_len, ceil(kv_len / 32)]")
        table = table.contiguous()
        device = table.device
    if seg_ids is not None:
        if seg_ids.dim() == 1:
            seg_ids = seg_ids[None]
        if seg_ids.dtype != torch.int32 or not seg_ids.is_cuda or seg_ids.dim() != 2:
            raise ValueError("seg_ids must be a CUDA int32 tensor [seg_batch, kv_len]")
        if seg_ids.shape[1] != kv_len or seg_ids.shape[0] not in (1, B):
            raise ValueError(f"seg_ids must hold kv_len={kv_len} ids per row and 1 or B={B} rows "
                             f"(got {tuple(seg_ids.shape)})")
        seg_ids = seg_ids.contiguous()
        device = seg_ids.device
    if sinks:
        if mask != "sink_window" or prefix_len:
            raise ValueError("sinks applies to the sink_window mask (and excludes prefix_len)")
        prefix_len = sinks
    # (a field of a ctypes structure would take the low 32 bits of a larger number)
    for name, x in (("window", window), ("sinks" if sinks else "prefix_len", prefix_len)):
        if not -2**31 <= x < 2**31:
            raise ValueError(f"{name} must be a 32-bit integer (got {x})")
    bm = BlockMask(B, H, q_len, kv_len, mask, window, prefix_len, seg_ids, device or "cuda", table=table, stream=stream)
    return bm.rebuild(stream, workspace)


def _check_fwd_tensors(q, k, v, out, lse, out_fp32, alibi_slopes, rel_bias, rel_max, bm):
    """The shapes, dtypes and placement fa_fwd / fa_fwd_noalloc read and write
    through raw pointers, which the C ABI cannot see: anything wrong here
    would become an out-of-bounds device access, so it is rejected first."""
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"unsupported dtype {dtype}")
    if k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k and v must share a dtype")
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4):
            raise ValueError("q, k, v must be contiguous CUDA tensors [B, H, T, D]")
    shape, kv_shape = q.shape, k.shape
    B, Hq, Tq, D = shape
    if kv_shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if kv_shape[0] != B or kv_shape[3] != D:
        raise ValueError("k and v must be [B, Hkv, kv_len, D] with q's B and D")
    if out_fp32 and dtype is not torch.bfloat16:
        raise ValueError("out_fp32 applies to bf16 inputs only")
    want = torch.float32 if out_fp32 else dtype
    if out.dtype is not want or not out.is_cuda or not out.is_contiguous() or out.shape != shape:
        raise ValueError(f"out must be a contiguous CUDA {want} tensor of q's shape")
    if lse.dtype is not torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, Hq, Tq):
        raise ValueError("lse must be a contiguous CUDA float32 tensor [B, Hq, q_len]")
    if alibi_slopes is not None:
        if alibi_slopes.dtype != torch.float32 or not alibi_slopes.is_cuda or not alibi_slopes.is_contiguous() \
                or alibi_slopes.numel() < Hq:
            raise ValueError("alibi_slopes must be a contiguous CUDA float32 tensor of at least Hq entries")
    if rel_bias is not None:
        if rel_bias.dtype != torch.float32 or not rel_bias.is_cuda or not rel_bias.is_contiguous() \
                or rel_bias.numel() < Hq * (2 * rel_max + 1):
            raise ValueError("rel_bias must be a contiguous CUDA float32 tensor [Hq, 2 rel_max + 1]")
    if bm.q_len != Tq or bm.kv_len != kv_shape[2]:
        raise ValueError(f"the BlockMask was built for ({bm.q_len}, {bm.kv_len}), not ({Tq}, {kv_shape[2]})")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, bm: BlockMask, *, score: str = "none",
        softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
        rel_bias: Optional[torch.Tensor] = None, rel_max: int = 0, scale: Optional[float] = None,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
        workspace: Optional[Workspace] = None, stream=None, timeout_ms: int = 0, debug_flags: int = 0,
        out_fp32: bool = False):
    """Block-sparse attention forward (fa_fwd); returns (o, lse).

    ``out_fp32`` writes O in fp32 for bf16 inputs (FA_OUT_FP32)."""
    dt = {torch.bfloat16: BF16, torch.float32: FP32}.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, D]")
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    if out is None:
        out = _new(q.shape, torch.float32 if out_fp32 else q.dtype, q.device, stream)
    if lse is None:
        lse = _new((B, Hq, Tq), torch.float32, q.device, stream)
    _check_fwd_tensors(q, k, v, out, lse, out_fp32, alibi_slopes, rel_bias, rel_max, bm)
    a = FwdArgs()
    a.dtype, a.B, a.Hq, a.Hkv, a.q_len, a.kv_len, a.D = dt, B, Hq, Hkv, Tq, Tkv, D
    a.scale = 0.0 if scale is None else float(scale)
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.timeout_ms, a.debug_flags = timeout_ms, debug_flags
    a.flags = OUT_FP32 if out_fp32 else 0
    sc = ScoreDesc()
    sc.kind = SCORE_KINDS[score]
    sc.softcap = softcap
    if alibi_slopes is not None:
        sc.alibi_slopes = alibi_slopes.data_ptr()
    if rel_bias is not None:
        sc.rel_bias = rel_bias.data_ptr()
        sc.rel_max = rel_max
    ws, raw = _launch(q.device, stream, workspace)
    _check(load_library().fa_fwd(ctypes.byref(a), ctypes.byref(bm.struct), ctypes.byref(sc), ws, raw))
    return out, lse


def fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, bm: BlockMask, *, out: torch.Tensor,
                lse: torch.Tensor, score: str = "none", softcap: float = 0.0,
                alibi_slopes: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None,
                rel_max: int = 0, scale: Optional[float] = None, stream=None, out_fp32: bool = False):
    """fa_fwd_noalloc: the forward for callers that cannot allocate device
    memory.  The caller passes preallocated `out` and `lse`; no workspace is
    taken (the library's scratch is a static device array)."""
    dt = {torch.bfloat16: BF16, torch.float32: FP32}.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    _check_fwd_tensors(q, k, v, out, lse, out_fp32, alibi_slopes, rel_bias, rel_max, bm)
    B, Hq, Tq, D = q.shape
    a = FwdArgs()
    a.dtype, a.B, a.Hq, a.Hkv, a.q_len, a.kv_len, a.D = dt, B, Hq, k.shape[1], Tq, k.shape[2], D
    a.scale = 0.0 if scale is None else float(scale)
    a.q, a.k, a.v, a.o, a.lse = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.flags = OUT_FP32 if out_fp32 else 0
    sc = ScoreDesc()
    sc.kind = SCORE_KINDS[score]
    sc.softcap = softcap
    if alibi_slopes is not None:
        sc.alibi_slopes = alibi_slopes.data_ptr()
    if rel_bias is not None:
        sc.rel_bias = rel_bias.data_ptr()
        sc.rel_max = rel_max
    _check(load_library().fa_fwd_noalloc(ctypes.byref(a), ctypes.byref(bm.struct), ctypes.byref(sc),
                                         _stream_ptr(stream)))
    return out, lse


def _score_desc(score, softcap, alibi_slopes, rel_bias, rel_max) -> ScoreDesc:
    sc = ScoreDesc()
    sc.kind = SCORE_KINDS[score]
    sc.softcap = softcap
    if alibi_slopes is not None:
        sc.alibi_slopes = alibi_slopes.data_ptr()
    if rel_bias is not None:
        sc.rel_bias = rel_bias.data_ptr()
        sc.rel_max = rel_max
    return sc


def decode_args(q: torch.Tensor, k: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, v: torch.Tensor = None,
                scale: Optional[float] = None, out_fp32: bool = False) -> FwdArgs:
    """The fa_fwd_args of a bf16 decoding call (shapes taken from q and k)."""
    B, Hq, Tq, D = q.shape
    a = FwdArgs()
    a.dtype, a.B, a.Hq, a.Hkv, a.q_len, a.kv_len, a.D = BF16, B, Hq, k.shape[1], Tq, k.shape[2], D
    a.scale = 0.0 if scale is None else float(scale)
    a.q, a.k, a.o, a.lse = q.data_ptr(), k.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.v = (v if v is not None else k).data_ptr()
    a.flags = OUT_FP32 if out_fp32 else 0
    return a


def decode_splits(q: torch.Tensor, k: torch.Tensor, bm: BlockMask) -> int:
    """The split count fa_fwd_decode picks for num_splits=0 on this device."""
    a = decode_args(q, k, q, q)
    return int(load_library().fa_decode_splits(ctypes.byref(a), ctypes.byref(bm.struct)))


def decode_partials(q: torch.Tensor, num_splits: int, stream=None) -> torch.Tensor:
    """fp32 scratch for fa_fwd_decode: [B, Hq, q_len, num_splits, D + 2]."""
    B, Hq, Tq, D = q.shape
    return _new((B, Hq, Tq, num_splits, D + 2), torch.float32, q.device, stream)


def fwd_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, bm: BlockMask, *, score: str = "none",
               softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
               rel_bias: Optional[torch.Tensor] = None, rel_max: int = 0, scale: Optional[float] = None,
               num_splits: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               partials: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None, stream=None,
               timeout_ms: int = 0, out_fp32: bool = False):
    """Split-KV decoding forward (fa_fwd_decode) for bf16 q of at most 128
    rows; returns (o, lse).  ``num_splits`` 0 lets the library choose;
    ``partials`` (see decode_partials) is allocated when not given."""
    if q.dtype != torch.bfloat16 or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("fwd_decode takes bf16 q, k, v")
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4):
            raise ValueError("q, k, v must be contiguous CUDA tensors [B, H, T, D]")
    B, Hq, Tq, D = q.shape
    if out is None:
        out = _new(q.shape, torch.float32 if out_fp32 else q.dtype, q.device, stream)
    if lse is None:
        lse = _new((B, Hq, Tq), torch.float32, q.device, stream)
    want = torch.float32 if out_fp32 else torch.bfloat16
    if out.dtype != want or not out.is_cuda or not out.is_contiguous() or tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out must be a contiguous CUDA {want} tensor of q's shape")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or tuple(lse.shape) != (B, Hq, Tq):
        raise ValueError("lse must be a contiguous CUDA float32 tensor [B, Hq, q_len]")
    a = decode_args(q, k, out, lse, v=v, scale=scale, out_fp32=out_fp32)
    a.timeout_ms = timeout_ms
    lib = load_library()
    if num_splits == 0:
        num_splits = int(lib.fa_decode_splits(ctypes.byref(a), ctypes.byref(bm.struct))) or 1
    if partials is None:
        partials = decode_partials(q, num_splits, stream)
    if partials.dtype != torch.float32 or not partials.is_cuda or not partials.is_contiguous():
        raise ValueError("partials must be a contiguous CUDA float32 tensor (see decode_partials)")
    sc = _score_desc(score, softcap, alibi_slopes, rel_bias, rel_max)
    ws, raw = _launch(q.device, stream, workspace)
    _check(lib.fa_fwd_decode(ctypes.byref(a), ctypes.byref(bm.struct), ctypes.byref(sc), num_splits,
                             ctypes.c_void_p(partials.data_ptr()), partials.numel() * partials.element_size(),
                             ws, raw))
    return out, lse


def bwd_rowstats(q: torch.Tensor, stream=None) -> torch.Tensor:
    """fp32 scratch for fa_bwd: fa_bwd_rowstats_bytes() bytes as a flat tensor."""
    B, Hq, Tq, _ = q.shape
    n = load_library().fa_bwd_rowstats_bytes(B, Hq, Tq) // 4
    return _new((n,), torch.float32, q.device, stream)


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
        dout: torch.Tensor, bm: BlockMask, *, score: str = "none", softcap: float = 0.0,
        alibi_slopes: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None, rel_max: int = 0,
        scale: Optional[float] = None, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
        dv: Optional[torch.Tensor] = None, rowstats: Optional[torch.Tensor] = None,
        workspace: Optional[Workspace] = None, stream=None, timeout_ms: int = 0):
    """Backward of fwd (fa_bwd) for bf16 q, k, v, the forward's bf16 o and
    its lse, and the upstream gradient dout; returns fp32 (dq, dk, dv).  The
    BlockMask's transposed lists are built on first use (BlockMask.cols)."""
    for t in (q, k, v, o, dout):
        if t.dtype is not torch.bfloat16 or not (t.is_cuda and t.is_contiguous() and t.dim() == 4):
            raise ValueError("q, k, v, o and dout must be contiguous CUDA bf16 tensors [B, H, T, D]")
    B, Hq, Tq, D = q.shape
    Hkv, Tkv = k.shape[1], k.shape[2]
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must have q's shape")
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must be [B, Hkv, kv_len, D] with q's B and D")
    dq = _new((B, Hq, Tq, D), torch.float32, q.device, stream) if dq is None else dq
    dk = _new((B, Hkv, Tkv, D), torch.float32, q.device, stream) if dk is None else dk
    dv = _new((B, Hkv, Tkv, D), torch.float32, q.device, stream) if dv is None else dv
    rowstats = bwd_rowstats(q, stream) if rowstats is None else rowstats
    for name, t, shape in (("lse", lse, (B, Hq, Tq)), ("dq", dq, (B, Hq, Tq, D)), ("dk", dk, (B, Hkv, Tkv, D)),
                           ("dv", dv, (B, Hkv, Tkv, D))):
        if t.dtype is not torch.float32 or not t.is_cuda or not t.is_contiguous() or t.shape != shape:
            raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of shape {shape}")
    need = load_library().fa_bwd_rowstats_bytes(B, Hq, Tq)
    if rowstats.dtype != torch.float32 or not rowstats.is_cuda or not rowstats.is_contiguous() \
            or rowstats.numel() * 4 < need:
        raise ValueError(f"rowstats must be a contiguous CUDA float32 tensor of at least {need} bytes")
    if bm.q_len != Tq or bm.kv_len != Tkv:
        raise ValueError(f"the BlockMask was built for ({bm.q_len}, {bm.kv_len}), not ({Tq}, {Tkv})")
    a = BwdArgs()
    a.B, a.Hq, a.Hkv, a.q_len, a.kv_len, a.D = B, Hq, Hkv, Tq, Tkv, D
    a.scale = 0.0 if scale is None else float(scale)
    a.q, a.k, a.v, a.o, a.dout = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr()
    a.lse, a.dq, a.dk, a.dv = lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    a.rowstats = rowstats.data_ptr()
    a.timeout_ms = timeout_ms
    sc = _score_desc(score, softcap, alibi_slopes, rel_bias, rel_max)
    bm._build_cols(stream, workspace)
    ws, raw = _launch(q.device, stream, workspace)
    _check(load_library().fa_bwd(ctypes.byref(a), ctypes.byref(bm.struct), ctypes.byref(bm._cols_struct),
                                 ctypes.byref(sc), ws, raw))
    return dq, dk, dv


def _paged_kv(k_cache, v_cache, page_table, kv_len, q_start, total_q, dev, scaled=False):
    """The packed fa_paged_kv of these tensors and the cache's shape.  The C ABI reads them through raw pointers:
    everything it cannot see is checked here."""
    shape, dtype = k_cache.shape, torch.float8_e4m3fn if scaled else torch.bfloat16
    if len(shape) != 4 or k_cache.dtype is not dtype or v_cache.dtype is not dtype \
            or v_cache.shape != shape or not k_cache.is_contiguous() or not v_cache.is_contiguous() \
            or k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError("k_cache and v_cache must be contiguous CUDA bf16 tensors [num_pages, Hkv, page_size, D] "
                         "on the rows' device (float8_e4m3fn where k_scale and v_scale are given)")
    i32, table, lens, starts = torch.int32, page_table.shape, kv_len.shape, q_start.shape
    if len(table) != 2 or len(lens) != 1 or len(starts) != 1 \
            or page_table.dtype is not i32 or kv_len.dtype is not i32 or q_start.dtype is not i32 \
            or page_table.get_device() != dev or kv_len.get_device() != dev or q_start.get_device() != dev \
            or not page_table.is_contiguous() or not kv_len.is_contiguous() or not q_start.is_contiguous():
        for name, t, dims in (("page_table", page_table, 2), ("kv_len", kv_len, 1), ("q_start", q_start, 1)):
            if t.dtype is not i32 or t.dim() != dims or t.get_device() != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} dimensions on the rows' device")
    B, max_pages = table
    if lens[0] != B or starts[0] != B + 1:
        raise ValueError(f"page_table has {B} rows: kv_len must hold {B} lengths and q_start {B + 1} offsets "
                         f"(got {kv_len.numel()}, {q_start.numel()})")
    num_pages, Hkv, page, D = shape
    return _packed(_PAGED_KV, "the paged cache", B, Hkv, D, num_pages, page, max_pages, total_q, k_cache.data_ptr(),
                   v_cache.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(), q_start.data_ptr()), Hkv, D


def _scales(k_scale, v_scale, k_cache, dev):
    """The packed fa_paged_scales; None for a cache without scales (bf16)."""
    if k_scale is None and v_scale is None:
        return None
    want, f32 = k_cache.shape[:2], torch.float32
    if k_scale is None or v_scale is None or k_scale.dtype is not f32 or v_scale.dtype is not f32 \
            or k_scale.shape != want or v_scale.shape != want or k_scale.get_device() != dev \
            or v_scale.get_device() != dev or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise ValueError(f"k_scale and v_scale come together: contiguous float32 tensors [num_pages, Hkv] = {tuple(want)} "
                         "on the cache's device")
    return _PAGED_SCALES.pack(k_scale.data_ptr(), v_scale.data_ptr())


def _rows(name, t, total, H, D, dev):
    """Token and head strides of bf16 rows [total, H, D] (H None: any)."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA bf16 tensor [tokens, heads, D] on the cache's device")
    n, h, d = t.shape
    if n != total or d != D or (H is not None and h != H):
        raise ValueError(f"{name} must be [{total}, {'heads' if H is None else H}, {D}] (got {tuple(t.shape)})")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # the stride of a dimension of one entry says nothing
    return ts if n > 1 else D, hs if h > 1 else D


def _packed(layout, what, *values):
    """The packed struct of a paged call; numbers that its fields do not hold are refused like the other arguments."""
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError):
        raise ValueError(f"{what}: a number is past the 32 bits of its field (got {values})") from None


def _call_on(dev, fn, *args):
    """A paged call with its tensors' device current."""
    if dev == _device_now():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


# Scratch of eager calls on a device's current stream, grown as needed: calls
# on one stream run one after another, and the lock keeps the launches of one
# call together where several threads share a stream.  A captured call gets
# scratch of its own, which its graph keeps.
_paged_scratch = {}
_PAGED_KEEP = 64 << 20         # larger ones go back to the allocator
_paged_lock = threading.Lock()


def kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor, *,
              k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
              cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, interleaved: bool = False,
              positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              workspace: Optional[Workspace] = None, stream=None):
    """Append a step's keys and values to the paged cache (fa_kv_append), rotating queries and keys on the way;
    returns the rotated queries.

    q [tokens, Hq, D], k and v [tokens, Hkv, D]: bf16 rows, any token and head strides that are multiples of 8 (slices
    of a fused projection); q may be None.  k_cache and v_cache [num_pages, Hkv, page_size, D]; page_table int32
    [B, max_pages]; kv_len int32 [B] counts the new tokens; sequence b's rows are q_start[b] .. q_start[b + 1] - 1,
    rows from q_start[B] on are left as they were.  cos and sin: fp32 [positions, rot_dim / 2], both or neither.
    q_out may be q.

    With k_scale and v_scale, float32 [num_pages, Hkv], the cache is held in 8 bits (fa_kv_append_scaled): k_cache and
    v_cache are float8_e4m3fn, and every page that receives tokens gets, per kv head, the power of two that its largest
    value needs, or keeps a larger one that its earlier tokens have."""
    dev = k.get_device()
    if dev < 0 or k.dim() != 3:
        raise ValueError("k must be a CUDA bf16 tensor [tokens, Hkv, D]")
    total = k.shape[0]
    scales = _scales(k_scale, v_scale, k_cache, dev)
    c, Hkv, D = _paged_kv(k_cache, v_cache, page_table, kv_len, q_start, total, dev, scales is not None)
    ks, vs = _rows("k", k, total, Hkv, D, dev), _rows("v", v, total, Hkv, D, dev)
    Hq, qp, op, qs, os_ = 0, 0, 0, (0, 0), (0, 0)
    if q is not None:
        qs = _rows("q", q, total, None, D, dev)
        Hq, qp = q.shape[1], q.data_ptr()
        if q_out is None:
            q_out = _new((total, Hq, D), torch.bfloat16, q.device, stream)
        os_ = qs if q_out is q else _rows("q_out", q_out, total, Hq, D, dev)
        op = q_out.data_ptr()
    rot, rope_len, cp, sp, pp = 0, 0, 0, 0, 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        for t in (cos, sin):
            if t.dtype is not torch.float32 or t.dim() != 2 or t.get_device() != dev or not t.is_contiguous():
                raise ValueError("cos and sin must be contiguous float32 tensors [positions, rot_dim / 2] on the "
                                 "cache's device")
        if sin.shape != cos.shape:
            raise ValueError("cos and sin must have one shape")
        rope_len, half = cos.shape
        rot, cp, sp = 2 * half, cos.data_ptr(), sin.data_ptr()
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.get_device() != dev or not positions.is_contiguous() \
                or positions.numel() != total:
            raise ValueError("positions must be a contiguous int32 tensor with one entry per row")
        pp = positions.data_ptr()
    a = _packed(_KV_APPEND, "kv_append", Hq, rot, rope_len, 1 if interleaved else 0, qp, k.data_ptr(), v.data_ptr(), op,
                *qs, *ks, *vs, *os_, cp, sp, pp)
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    ws = workspace or _workspace_of(dev, raw, _capture_of(dev, raw, stream is not None))
    lib = load_library()
    if scales is None:
        st = _call_on(dev, lib.fa_kv_append, c, a, ws.tensor.data_ptr(), raw)
    else:
        st = _call_on(dev, lib.fa_kv_append_scaled, c, scales, a, ws.tensor.data_ptr(), raw)
    if st != OK:
        _check(st)
    return q_out


def fwd_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
              kv_len: torch.Tensor, q_start: torch.Tensor, *, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, max_q_len: Optional[int] = None, mask: str = "causal",
              window: int = 0, sinks: int = 0, shared_len: int = 0, score: str = "none", softcap: float = 0.0,
              alibi_slopes: Optional[torch.Tensor] = None, rel_bias: Optional[torch.Tensor] = None, rel_max: int = 0,
              scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              scratch: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None, stream=None,
              timeout_ms: int = 0, out_fp32: bool = False):
    """Attention from a step's queries to the paged cache (fa_fwd_paged); returns (o, lse), o [tokens, Hq, D] and lse
    float32 [tokens, Hq].

    q [tokens, Hq, D] bf16, token and head strides multiples of 8; the cache and the batch as for kv_append.
    ``max_q_len`` bounds the new tokens of a sequence (default: all of q's rows; a tight bound lets single tokens take
    the decoding kernel: 64 x 512 keys 31 us, 41 without, 8 x 32768 keys 165 and 176).  mask: "full", "causal", "sliding_window" (``window``) or "sink_window" (``window`` and
    ``sinks``), by position.  ``shared_len``: length of a prefix all sequences share, read once through page_table[0].
    Rows behind the last sequence are left as they were; ``scratch`` is allocated when not given.

    With k_scale and v_scale, float32 [num_pages, Hkv], the cache is held in 8 bits (fa_fwd_paged_scaled): k_cache and
    v_cache are float8_e4m3fn codes, whose values are code x scale of the code's page and kv head."""
    dev = q.get_device()
    if dev < 0 or q.dim() != 3:
        raise ValueError("q must be a CUDA bf16 tensor [tokens, Hq, D]")
    total, Hq, _ = q.shape
    scales = _scales(k_scale, v_scale, k_cache, dev)
    c, _, D = _paged_kv(k_cache, v_cache, page_table, kv_len, q_start, total, dev, scales is not None)
    qs = _rows("q", q, total, None, D, dev)
    want = torch.float32 if out_fp32 else torch.bfloat16
    if out is None:
        out = _new((total, Hq, D), want, q.device, stream)
    elif out.dtype is not want or out.get_device() != dev or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError(f"out must be a contiguous {want} tensor of q's shape on q's device")
    if lse is None:
        lse = _new((total, Hq), torch.float32, q.device, stream)
    elif lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() \
            or tuple(lse.shape) != (total, Hq):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, Hq] on q's device")
    sp, bp = 0, 0
    if alibi_slopes is not None or rel_bias is not None:
        for name, t, need in (("alibi_slopes", alibi_slopes, Hq), ("rel_bias", rel_bias, Hq * (2 * rel_max + 1))):
            if t is not None and (t.dtype is not torch.float32 or t.get_device() != dev or not t.is_contiguous()
                                  or t.numel() < need):
                raise ValueError(f"{name} must be a contiguous float32 tensor of at least {need} entries on q's device")
        sp = 0 if alibi_slopes is None else alibi_slopes.data_ptr()
        bp = 0 if rel_bias is None else rel_bias.data_ptr()
    if mask not in MASK_KINDS or score not in SCORE_KINDS:
        raise ValueError(f"unknown mask {mask!r} or score {score!r}")
    if sinks and mask != "sink_window":
        raise ValueError("sinks applies to the sink_window mask")
    a = _packed(_PAGED_FWD, "fwd_paged", Hq, (total or 1) if max_q_len is None else max_q_len, shared_len,
                0.0 if scale is None else scale, q.data_ptr(), *qs, out.data_ptr(), lse.data_ptr(), timeout_ms,
                OUT_FP32 if out_fp32 else 0)
    m = _packed(_MASK, "the mask", MASK_KINDS[mask], window, sinks, 0, 0, 0, 0)
    sc = _packed(_SCORE, "the score", SCORE_KINDS[score], softcap, sp, bp, rel_max)
    lib = load_library()
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    capture = _capture_of(dev, raw, stream is not None)
    ws = workspace or _workspace_of(dev, raw, capture)
    # the calls on the cache (and its scales, in 8 bits)
    head, call = ((c,), lib.fa_fwd_paged) if scales is None else ((c, scales), lib.fa_fwd_paged_scaled)

    if scratch is not None:
        if scratch.get_device() != dev or not scratch.is_contiguous():
            raise ValueError("scratch must be a contiguous tensor on q's device")
        st = _call_on(dev, call, *head, a, m, sc, scratch.data_ptr(), scratch.numel() * scratch.element_size(),
                      ws.tensor.data_ptr(), raw)
    elif stream is not None or capture:
        # (no bytes: the arguments are wrong, and the call says how)
        scratch = _new(_call_on(dev, lib.fa_paged_scratch_bytes, c, a) or 16, torch.uint8, q.device, stream)
        st = _call_on(dev, call, *head, a, m, sc, scratch.data_ptr(), scratch.numel(), ws.tensor.data_ptr(), raw)
    else:
        with _paged_lock:
            kept = _paged_scratch.get((dev, raw))
            st = ERR_INVALID_ARG if kept is None else \
                _call_on(dev, call, *head, a, m, sc, kept.data_ptr(), kept.numel(), ws.tensor.data_ptr(), raw)
            if st == ERR_INVALID_ARG:              # none yet, or too small (or wrong arguments: the call says so again)
                kept = torch.empty(_call_on(dev, lib.fa_paged_scratch_bytes, c, a) or 16, dtype=torch.uint8,
                                   device=q.device)
                st = _call_on(dev, call, *head, a, m, sc, kept.data_ptr(), kept.numel(), ws.tensor.data_ptr(), raw)
                if st == OK and kept.numel() <= _PAGED_KEEP:
                    _paged_scratch[(dev, raw)] = kept
    if st != OK:
        _check(st)
    return out, lse


def paged_scratch(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                  kv_len: torch.Tensor, q_start: torch.Tensor, *, max_q_len: Optional[int] = None,
                  shared_len: int = 0) -> torch.Tensor:
    """Scratch for fwd_paged calls of these shapes (of a bf16 cache or one held in 8 bits), for callers that keep their
    own."""
    with torch.cuda.device(q.device):
        c, _, _ = _paged_kv(k_cache, v_cache, page_table, kv_len, q_start, q.shape[0], q.get_device(),
                            k_cache.dtype is torch.float8_e4m3fn)
        a = _packed(_PAGED_FWD, "paged_scratch", q.shape[1], max(q.shape[0], 1) if max_q_len is None else max_q_len,
                    shared_len, 0.0, 0, 0, 0, 0, 0, 0, 0)
        n = load_library().fa_paged_scratch_bytes(c, a)
        if n == 0:
            raise FAError(ERR_INVALID_ARG, load_library().fa_last_error().decode())
        return torch.empty(n, dtype=torch.uint8, device=q.device)


def paged_step(new_len: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, free_pages: torch.Tensor,
               free_count: torch.Tensor, *, page_size: int, total_q: int, keep_len: Optional[torch.Tensor] = None,
               shared_pages: int = 0, kv_len_out: Optional[torch.Tensor] = None,
               free_count_out: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None,
               slots: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               workspace: Optional[Workspace] = None, stream=None):
    """A step's pages, offsets and slots from its sequences' lengths, on the device (fa_paged_step); returns
    (q_start, slots, positions): int32 [B + 1], int64 [total_q] (page x page_size + place, -1 behind the last sequence)
    and int32 [total_q].

    Sequence b had kv_len[b] tokens in the cache, of which it keeps keep_len[b] (default: all), and brings new_len[b]
    new ones.  Its row of page_table [B, max_pages] gets the pages that it needs from the stack free_pages [num_pages],
    of which the first free_count[0] are free, or gives back those that it no longer needs; the first shared_pages
    entries stay.  kv_len and free_count are brought up to date in place, or into kv_len_out and free_count_out.  All are
    int32 on one device.  A step that cannot be made (contradicting lengths, too few free pages) becomes an empty one,
    and the workspace's check() says so."""
    dev = kv_len.get_device()
    if dev < 0 or kv_len.dim() != 1 or page_table.dim() != 2 or page_table.shape[0] != kv_len.shape[0]:
        raise ValueError("kv_len must be a CUDA int32 tensor [B] and page_table one of [B, max_pages]")
    B, max_pages = page_table.shape
    if total_q < 0 or total_q > 2147483647:
        raise ValueError(f"total_q must be 0 .. 2^31 - 1 (got {total_q})")
    if q_start is None:
        q_start = _new((B + 1,), torch.int32, kv_len.device, stream)
    if slots is None:
        slots = _new((total_q,), torch.int64, kv_len.device, stream)
    if positions is None:
        positions = _new((total_q,), torch.int32, kv_len.device, stream)
    kv_out = kv_len if kv_len_out is None else kv_len_out
    count_out = free_count if free_count_out is None else free_count_out
    for name, t, n in (("new_len", new_len, B), ("kv_len", kv_len, B), ("keep_len", keep_len, B),
                       ("page_table", page_table, B * max_pages), ("free_pages", free_pages, None),
                       ("free_count", free_count, 1), ("kv_len_out", kv_out, B), ("free_count_out", count_out, 1),
                       ("q_start", q_start, B + 1), ("positions", positions, total_q)):
        if t is not None and (t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous()
                              or (n is not None and t.numel() != n)):
            raise ValueError(f"{name} must be a contiguous int32 tensor{'' if n is None else f' of {n} entries'} on "
                             "kv_len's device")
    if slots.dtype is not torch.int64 or slots.get_device() != dev or not slots.is_contiguous() \
            or slots.numel() != total_q:
        raise ValueError(f"slots must be a contiguous int64 tensor of {total_q} entries on kv_len's device")
    a = _packed(_PAGED_STEP, "paged_step", B, free_pages.numel(), page_size, max_pages, shared_pages, total_q,
                new_len.data_ptr(), 0 if keep_len is None else keep_len.data_ptr(), kv_len.data_ptr(),
                page_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), kv_out.data_ptr(),
                count_out.data_ptr(), q_start.data_ptr(), slots.data_ptr(), positions.data_ptr())
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    ws = workspace or _workspace_of(dev, raw, _capture_of(dev, raw, stream is not None))
    st = _call_on(dev, load_library().fa_paged_step, a, ws.tensor.data_ptr(), raw)
    if st != OK:
        _check(st)
    return q_start, slots, positions


def version() -> str:
    return load_library().fa_version().decode()
