"""ctypes binding of libparallax.so (declared in include/parallax.h).

Argument marshalling only: these functions read tensor pointers, shapes and
the current torch stream, fill the C parameter structs and call the library.
Every step of the computation runs in the library's CUDA kernels.  Importing
this module loads the library and raises if it has not been built; there is
no fallback.
"""

from __future__ import annotations

import collections
import ctypes
import os
import struct
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libparallax.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m parallax_local_linear_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

PLX_F32, PLX_BF16 = 0, 1
STATUS = {0: "PLX_OK", 1: "PLX_ERR_INVALID_ARG", 2: "PLX_ERR_UNSUPPORTED", 3: "PLX_ERR_WORKSPACE",
          4: "PLX_ERR_CUDA", 5: "PLX_ERR_DEVICE_FAULT", 6: "PLX_ERR_TIMEOUT"}
DEVERR_BAD_PAGE, DEVERR_TIMEOUT, DEVERR_BAD_LENGTH, DEVERR_SINGULAR = 1, 2, 4, 8
DEVERR_NO_PAGES, DEVERR_BAD_POSITION = 16, 32
PAGE_SIZE = 64


class DecodeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("num_ctas", ctypes.c_int32)]


class PrefillParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("cta_pair", ctypes.c_int32)]


class PrefillPagedParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("total_q", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32)]


class PagePlanParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_rows", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32), ("num_free", ctypes.c_int32)]


class NormRopeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("max_pos", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("pos_batch_stride", ctypes.c_int64)]


class HeadRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("w", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3)]


class HeadGrads(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("dw", ctypes.c_void_p),
                ("dy_stride", ctypes.c_int64 * 3), ("dx_stride", ctypes.c_int64 * 3)]


class AppendParams(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2)]


_vp, _i32p = ctypes.c_void_p, ctypes.c_void_p
lib.parallax_abi_version.restype = ctypes.c_int32
lib.parallax_status_string.restype = ctypes.c_char_p
lib.parallax_status_string.argtypes = [ctypes.c_int]
lib.parallax_decode_num_ctas.restype = ctypes.c_int32
lib.parallax_decode_num_ctas.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_int32]
lib.parallax_decode_workspace_size.restype = ctypes.c_size_t
lib.parallax_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_int32]
lib.parallax_decode.restype = ctypes.c_int
lib.parallax_decode.argtypes = [_vp, _vp, _vp, _vp, _i32p, _i32p, _vp, _vp, ctypes.c_size_t,
                                ctypes.POINTER(DecodeParams), _vp]
lib.parallax_prefill.restype = ctypes.c_int
lib.parallax_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.POINTER(PrefillParams), _vp]
lib.parallax_prefill_paged.restype = ctypes.c_int
lib.parallax_prefill_paged.argtypes = [_vp, _vp, _vp, _vp, _i32p, _i32p, _i32p, _vp,
                                       ctypes.POINTER(PrefillPagedParams), _vp]
lib.parallax_prefill_train.restype = ctypes.c_int
lib.parallax_prefill_train.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(PrefillParams), _vp]
lib.parallax_prefill_backward_workspace_size.restype = ctypes.c_size_t
lib.parallax_prefill_backward_workspace_size.argtypes = [ctypes.POINTER(PrefillParams)]
lib.parallax_prefill_backward.restype = ctypes.c_int
lib.parallax_prefill_backward.argtypes = [_vp] * 13 + [ctypes.c_size_t, ctypes.POINTER(PrefillParams), _vp]
lib.parallax_decode_noalloc.restype = ctypes.c_int
lib.parallax_decode_projected.argtypes = [_vp, _vp, _vp, ctypes.c_int32, _vp, _vp, _i32p, _i32p, _vp, _vp, _vp,
                                          _vp, ctypes.c_size_t, ctypes.POINTER(DecodeParams), _vp]
lib.parallax_decode_projected.restype = ctypes.c_int
lib.parallax_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i32p, _i32p, _vp, ctypes.POINTER(DecodeParams), _vp]
NOALLOC_SCRATCH_BYTES = 8 << 20
lib.parallax_lla_decode_workspace_size.restype = ctypes.c_size_t
lib.parallax_lla_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_float, ctypes.c_int32]
lib.parallax_lla_decode.restype = ctypes.c_int
lib.parallax_lla_decode.argtypes = [_vp, _vp, _vp, _i32p, _i32p, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t,
                                    ctypes.POINTER(DecodeParams), _vp]
lib.parallax_decode_plan_create.restype = ctypes.c_int
lib.parallax_decode_plan_create.argtypes = [_vp, _vp, _vp, _vp, _i32p, _i32p, _vp, _vp, ctypes.c_size_t,
                                            ctypes.POINTER(DecodeParams), ctypes.POINTER(ctypes.c_void_p)]
lib.parallax_decode_plan_run.restype = ctypes.c_int
lib.parallax_decode_plan_run.argtypes = [_vp, _vp]
lib.parallax_decode_plan_run_io.restype = ctypes.c_int
lib.parallax_decode_plan_run_io.argtypes = [_vp, _vp, _vp, _vp, _vp]
lib.parallax_decode_plan_destroy.restype = None
lib.parallax_decode_plan_destroy.argtypes = [_vp]
lib.parallax_set_wait_limit_ns.restype = ctypes.c_int
lib.parallax_set_wait_limit_ns.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64)]
lib.parallax_last_cuda_error.restype = ctypes.c_int32
lib.parallax_last_cuda_error.argtypes = []
lib.parallax_cuda_error_string.restype = ctypes.c_char_p
lib.parallax_cuda_error_string.argtypes = [ctypes.c_int32]
lib.parallax_capture_id.restype = ctypes.c_uint64
lib.parallax_capture_id.argtypes = [_vp]
lib.parallax_last_device_error.restype = ctypes.c_int
lib.parallax_last_device_error.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]

lib.parallax_page_plan.restype = ctypes.c_int
lib.parallax_page_plan.argtypes = [_vp] * 12
lib.parallax_norm_rope.restype = ctypes.c_int
lib.parallax_norm_rope.argtypes = [_vp, ctypes.c_int32, _i32p, _vp, _vp, _vp, _vp]
lib.parallax_norm_rope_backward_workspace_size.restype = ctypes.c_size_t
lib.parallax_norm_rope_backward_workspace_size.argtypes = [_vp, ctypes.c_int32]
lib.parallax_norm_rope_backward.restype = ctypes.c_int
lib.parallax_norm_rope_backward.argtypes = [_vp, _vp, ctypes.c_int32, _i32p, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
lib.parallax_cache_append.restype = ctypes.c_int
lib.parallax_cache_append.argtypes = [_vp] * 7
lib.parallax_q4_block_bytes.restype = ctypes.c_size_t
lib.parallax_q4_block_bytes.argtypes = [ctypes.c_int32]
lib.parallax_cache_append_q4.restype = ctypes.c_int
lib.parallax_cache_append_q4.argtypes = [_vp] * 6
lib.parallax_cache_gather_q4.restype = ctypes.c_int
lib.parallax_cache_gather_q4.argtypes = [_vp] * 6
lib.parallax_decode_q4_workspace_size.restype = ctypes.c_size_t
lib.parallax_decode_q4_workspace_size.argtypes = [_vp, ctypes.c_int32]
lib.parallax_decode_q4.restype = ctypes.c_int
lib.parallax_decode_q4.argtypes = [_vp, _vp, _vp, _i32p, _i32p, _vp, _vp, ctypes.c_size_t, _vp, _vp]

SIZE_MAX = ctypes.c_size_t(-1).value


class ParallaxError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = f"{what}: {STATUS.get(status, status)}"
        if status == 4:   # PLX_ERR_CUDA: name the CUDA error behind it
            code = lib.parallax_last_cuda_error()
            if code:
                msg += f" ({lib.parallax_cuda_error_string(code).decode()}, cudaError {code})"
        super().__init__(msg)


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return PLX_BF16
    if dt == torch.float32:
        return PLX_F32
    raise TypeError(f"unsupported dtype {dt}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_cuda(name, t, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _check_sequences(batch, seq_lens, page_table):
    """seq_lens [B] int32 and page_table [B, max_pages] int32 on the device
    (either may be None): the kernels read one entry / row per sequence."""
    if seq_lens is not None and tuple(seq_lens.shape) != (batch,):
        raise ValueError(f"seq_lens must have shape ({batch},), got {tuple(seq_lens.shape)}")
    if page_table is not None:
        if page_table.dim() != 2 or page_table.shape[0] != batch:
            raise ValueError(f"page_table must be [{batch}, max_pages], got {tuple(page_table.shape)}")
        if seq_lens is None:
            raise ValueError("a paged cache needs seq_lens")
        _check_cuda("page_table", page_table, torch.int32)
    if seq_lens is not None:
        _check_cuda("seq_lens", seq_lens, torch.int32)


def _check_cache_layout(batch, num_q_heads, head_dim, k_cache, v_cache, seq_lens, page_table, kv_len):
    """Shape checks of a decode's cache and sequence tables (host-only, so
    they run before any device check): the library reads the caches through
    these shapes, so a mismatch would read outside them."""
    if k_cache.dim() != 4 or tuple(k_cache.shape) != tuple(v_cache.shape):
        raise ValueError(f"k_cache and v_cache must be 4-D and alike, got {tuple(k_cache.shape)} "
                         f"and {tuple(v_cache.shape)}")
    if k_cache.shape[-1] != head_dim:
        raise ValueError(f"the caches' head_dim {k_cache.shape[-1]} differs from the queries' {head_dim}")
    if k_cache.shape[1] < 1 or num_q_heads % k_cache.shape[1]:
        raise ValueError(f"{num_q_heads} query heads do not split into {k_cache.shape[1]} KV heads")
    if page_table is None:
        if k_cache.shape[0] != batch:
            raise ValueError(f"a contiguous cache holds one sequence per row: {k_cache.shape[0]} != {batch}")
        # The library addresses token t of (b, kv head) as row (b * Hkv + kvh) * kv_len + t,
        # so kv_len must be the cache's own row count; seq_lens limits each sequence.
        if kv_len is not None and int(kv_len) != k_cache.shape[2]:
            raise ValueError(f"kv_len {kv_len} must equal the contiguous cache's length {k_cache.shape[2]} "
                             "(use seq_lens for shorter sequences)")
    else:
        if k_cache.shape[2] != PAGE_SIZE:
            raise ValueError(f"paged caches hold {PAGE_SIZE}-token pages: got {tuple(k_cache.shape)}")
        if page_table.dim() == 2 and kv_len is not None and int(kv_len) > page_table.shape[1] * PAGE_SIZE:
            raise ValueError(f"kv_len {kv_len} exceeds the page table's {page_table.shape[1]} pages")
    if seq_lens is not None and tuple(seq_lens.shape) != (batch,):
        raise ValueError(f"seq_lens must have shape ({batch},), got {tuple(seq_lens.shape)}")
    if page_table is not None:
        if page_table.dim() != 2 or page_table.shape[0] != batch:
            raise ValueError(f"page_table must be [{batch}, max_pages], got {tuple(page_table.shape)}")
        if seq_lens is None:
            raise ValueError("a paged cache needs seq_lens")


def _check_decode_inputs(q, rho, k_cache, v_cache, seq_lens, page_table, kv_len):
    """Every check of a decode call's inputs: shapes first, then devices and dtypes."""
    if q.dim() != 3 or tuple(rho.shape) != tuple(q.shape):
        raise ValueError(f"q and rho must be [B, Hq, d] and alike, got {tuple(q.shape)} and {tuple(rho.shape)}")
    B, Hq, d = q.shape
    _check_cache_layout(B, Hq, d, k_cache, v_cache, seq_lens, page_table, kv_len)
    _check_cuda("q", q)
    for name, t in (("rho", rho), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, q.dtype)
    _check_sequences(B, seq_lens, page_table)


def _output(out, out_dtype, shape, default_dtype, device):
    """The call's output tensor and dtype.  A caller's ``out`` must have
    ``shape`` (the kernels write every element of it) and, when
    ``out_dtype`` is given, that dtype; otherwise its own dtype is the
    output dtype.  Without ``out`` a new tensor is allocated."""
    if out is None:
        dt = out_dtype or default_dtype
        return torch.empty(tuple(shape), dtype=dt, device=device), dt
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out.shape)}")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype} but out_dtype is {out_dtype}")
    _check_cuda("out", out)
    return out, out.dtype


_ws_lock = threading.Lock()
_workspaces = {}


def _kept_workspace(kind, index, partials, counters):
    """(tensor, bytes for counters) of a workspace that the binding keeps for calls of ``kind``:
    that many bytes for counters at one end (none where ``counters`` is 0), which are zero before
    every call, and the rest for partials, each the most that a call has needed, so that one
    call's partials never lie where another's counters do.

    There is one per device and stream, since calls on different streams may overlap, and
    another per capture and stream: graphs may be replayed at once, and what a capture records
    is not done yet.  A graph clears its counters when it starts; after that, as in direct
    calls, every call leaves them zero.  (Memory taken under torch.cuda.graph belongs to the
    graph.  Captures made in another way need a DecodePlan, or decode_q4's ``workspace``,
    that outlives them.)
    """
    stream = _raw_stream(index)
    capture = lib.parallax_capture_id(stream) if _capturing(index) else 0
    key = kind, index, stream, capture != 0
    kept = _workspaces.get(key)
    if kept is None or kept[1] != capture or partials > kept[2] or counters > kept[3]:
        with _ws_lock:
            most, room = kept[2:] if kept is not None and kept[1] == capture else (1 << 20, 1 << 14 if counters else 0)
            most, room = max(most, partials), max(room, counters)
            ws = torch.empty(room + most, dtype=torch.uint8, device=index)
            (ws[most:] if kind == "q4" else ws[:room]).zero_()
            kept = _workspaces[key] = ws, capture, most, room
    return kept[0], kept[3]


def _decode_workspace(index, nbytes, params):
    """(tensor, address, bytes) of a decode's workspace: its counters (4 bytes per unit, padded to
    256) end where the partials of every call start.  The caller keeps the tensor until it has
    launched (another thread may replace it)."""
    units = params.batch * (params.num_kv_heads if params.in_dtype == PLX_BF16 else params.num_q_heads)
    counters = (4 * units + 255) & ~255
    ws, room = _kept_workspace("decode", index, nbytes - counters, counters)
    return ws, ws.data_ptr() + room - counters, ws.numel() - room + counters


def decode_params(q, k_cache, *, page_table=None, kv_len=None, scale=None, out_dtype=None,
                  num_ctas=0, num_pages=None):
    B, Hq, d = q.shape
    paged = page_table is not None
    Hkv = k_cache.shape[1]
    if paged:
        if k_cache.shape[2] != PAGE_SIZE:
            raise ValueError(f"paged caches hold {PAGE_SIZE}-token pages: got {tuple(k_cache.shape)}")
        max_pages = page_table.shape[1]
        L = kv_len if kv_len is not None else max_pages * PAGE_SIZE
        n_pages = k_cache.shape[0] if num_pages is None else num_pages
    else:
        max_pages = 0
        L = k_cache.shape[2] if kv_len is None else kv_len
        n_pages = 0
    scale = (1.0 / d ** 0.5) if scale is None else float(scale)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    return DecodeParams(B, Hq, Hkv, d, L, PAGE_SIZE if paged else 0, n_pages, max_pages,
                        _dtype_code(q.dtype), _dtype_code(out_dtype), scale, int(num_ctas))


def decode_workspace_size(params: DecodeParams, num_sms: int = 0) -> int:
    n = lib.parallax_decode_workspace_size(ctypes.byref(params), int(num_sms))
    if n == SIZE_MAX:
        raise ParallaxError(1, "parallax_decode_workspace_size")
    return n


def decode_num_ctas(params: DecodeParams, num_sms: int = 0) -> int:
    return lib.parallax_decode_num_ctas(ctypes.byref(params), int(num_sms))


def decode(q, rho, k_cache, v_cache, scale=None, *, seq_lens=None, page_table=None, out=None,
           out_dtype=None, num_ctas=0, kv_len=None):
    """Parallax decode: out[b, h] = vbar - Sigma_KV^T rho[b, h] over sequence b.

    q, rho: [B, Hq, d] (bfloat16 or float32, the cache's dtype).
    Contiguous cache: k_cache, v_cache [B, Hkv, L, d]; ``seq_lens`` (int32
    [B], optional) limits each sequence.  Paged cache: pools [P, Hkv, 64, d]
    with ``page_table`` (int32 [B, max_pages]) and ``seq_lens`` (required).
    Returns out [B, Hq, d] in ``out_dtype`` (default: the input dtype).
    Calls on several streams, and in several graphs (torch.cuda.graph), may
    overlap.
    """
    _check_decode_inputs(q, rho, k_cache, v_cache, seq_lens, page_table, kv_len)
    out, out_dtype = _output(out, out_dtype, q.shape, q.dtype, q.device)
    p = decode_params(q, k_cache, page_table=page_table, kv_len=kv_len, scale=scale,
                      out_dtype=out_dtype, num_ctas=num_ctas)
    nbytes = decode_workspace_size(p)
    ws, ws_at, ws_bytes = _decode_workspace(q.get_device(), nbytes, p)
    st = lib.parallax_decode(_ptr(q), _ptr(rho), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                             _ptr(seq_lens), _ptr(out), ws_at, ws_bytes, ctypes.byref(p), _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_decode")
    return out


class DecodePlan:
    """A prepared decode over fixed buffers (parallax_decode_plan_*).

    Checks and prepares ``decode(q, rho, k_cache, v_cache, ..., out=out)``
    once; each ``run()`` is one kernel launch on the current stream that
    reads the buffers' current contents.  The plan keeps references to every
    tensor it was made from (so they stay allocated at the same address) and
    owns a zeroed workspace of its own.  Runs of one plan must not overlap on
    the GPU (they share that workspace).
    """

    def __init__(self, q, rho, k_cache, v_cache, scale=None, *, out, seq_lens=None, page_table=None, num_ctas=0,
                 kv_len=None):
        _check_decode_inputs(q, rho, k_cache, v_cache, seq_lens, page_table, kv_len)
        out, out_dtype = _output(out, None, q.shape, q.dtype, q.device)
        p = decode_params(q, k_cache, page_table=page_table, kv_len=kv_len, scale=scale, out_dtype=out_dtype,
                          num_ctas=num_ctas)
        nbytes = decode_workspace_size(p)
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=q.device)
        handle = ctypes.c_void_p()
        st = lib.parallax_decode_plan_create(_ptr(q), _ptr(rho), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                             _ptr(seq_lens), _ptr(out), _ptr(ws), ws.numel(), ctypes.byref(p),
                                             ctypes.byref(handle))
        if st != 0:
            raise ParallaxError(st, "parallax_decode_plan_create")
        self._handle = handle
        self._keep = (q, rho, k_cache, v_cache, seq_lens, page_table, ws)
        self.out = out
        self._device = q.device
        self._run = lib.parallax_decode_plan_run

    def run(self):
        st = self._run(self._handle, ctypes.c_void_p(torch.cuda.current_stream(self._device).cuda_stream))
        if st != 0:
            raise ParallaxError(st, "parallax_decode_plan_run")
        return self.out

    def run_io(self, host_q, host_rho, host_out):
        """One step from host memory on the current stream: ``host_q`` and
        ``host_rho`` in, the decode, the output into ``host_out`` (host
        tensors: contiguous, shaped and typed like q / out).  When all three
        are pinned the kernel reads and writes them across PCIe itself, and
        reads q and rho as it starts, possibly before the kernel queued
        ahead of it has finished: the host must have written them before
        the call.  Otherwise they go through copies into and out of the
        plan's buffers."""
        q, rho = self._keep[0], self._keep[1]
        for name, t, like in (("host_q", host_q, q), ("host_rho", host_rho, rho), ("host_out", host_out, self.out)):
            if t.is_cuda or not t.is_contiguous() or t.dtype != like.dtype or tuple(t.shape) != tuple(like.shape):
                raise ValueError(f"{name} must be a contiguous host tensor like {tuple(like.shape)} {like.dtype}")
        st = lib.parallax_decode_plan_run_io(self._handle, _ptr(host_q), _ptr(host_rho), _ptr(host_out),
                                             ctypes.c_void_p(torch.cuda.current_stream(self._device).cuda_stream))
        if st != 0:
            raise ParallaxError(st, "parallax_decode_plan_run_io")
        return host_out

    def __del__(self):
        h = getattr(self, "_handle", None)
        if h is not None and h.value:
            lib.parallax_decode_plan_destroy(h)
            self._handle = None


def decode_projected(x, w_q, w_rho, k_cache, v_cache, scale=None, *, seq_lens=None, page_table=None,
                     q_out=None, rho_out=None, out=None, out_dtype=None, num_ctas=0, kv_len=None):
    """Decode with q and rho projected from the new token's layer input in the
    same call: q[b, h] = bf16(W_Q[h] x[b]), rho[b, h] = bf16(W_R[h] x[b]),
    then ``decode``.

    x: [B, hidden] bf16; w_q, w_rho: [Hq * d, hidden] bf16 (d = the cache's
    head_dim); caches and options as in ``decode``.  Returns (out, q, rho):
    out [B, Hq, d] in ``out_dtype`` (default bf16) and the projections
    [B, Hq, d] bf16 (written into ``q_out`` / ``rho_out`` when given).
    """
    if x.dim() != 2 or w_q.dim() != 2 or w_q.shape != w_rho.shape or w_q.shape[1] != x.shape[1]:
        raise ValueError("x must be [B, hidden] and w_q, w_rho [Hq * d, hidden]")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("caches must be 4-D and alike")
    d = k_cache.shape[-1]
    if w_q.shape[0] % d:
        raise ValueError("w_q rows must be a multiple of head_dim")
    B, Hq = x.shape[0], w_q.shape[0] // d
    _check_cache_layout(B, Hq, d, k_cache, v_cache, seq_lens, page_table, kv_len)
    _check_cuda("x", x, torch.bfloat16)
    for name, t in (("w_q", w_q), ("w_rho", w_rho), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, torch.bfloat16)
    if q_out is None:
        q_out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=x.device)
    if rho_out is None:
        rho_out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=x.device)
    for name, t in (("q_out", q_out), ("rho_out", rho_out)):
        _check_cuda(name, t, torch.bfloat16)
        if t.shape != (B, Hq, d):
            raise ValueError(f"{name} must be [B, Hq, d] = {(B, Hq, d)}")
    _check_sequences(B, seq_lens, page_table)
    out, out_dtype = _output(out, out_dtype, (B, Hq, d), torch.bfloat16, x.device)
    p = decode_params(q_out, k_cache, page_table=page_table, kv_len=kv_len, scale=scale,
                      out_dtype=out_dtype, num_ctas=num_ctas)
    nbytes = decode_workspace_size(p)
    ws, ws_at, ws_bytes = _decode_workspace(x.get_device(), nbytes, p)
    st = lib.parallax_decode_projected(_ptr(x), _ptr(w_q), _ptr(w_rho), int(x.shape[1]), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(page_table), _ptr(seq_lens), _ptr(q_out),
                                       _ptr(rho_out), _ptr(out), ws_at, ws_bytes, ctypes.byref(p),
                                       _stream_ptr(x.device))
    if st != 0:
        raise ParallaxError(st, "parallax_decode_projected")
    return out, q_out, rho_out


def decode_noalloc(q, rho, k_cache, v_cache, scale=None, *, seq_lens=None, page_table=None, out, num_ctas=0,
                   kv_len=None):
    """Decode through parallax_decode_noalloc: no workspace, no allocation.

    For callers that cannot allocate device memory: ``out`` must be given,
    and the library's fixed device scratch (NOALLOC_SCRATCH_BYTES per GPU)
    holds the split partials.  Calls that overlap on the GPU race.
    """
    _check_decode_inputs(q, rho, k_cache, v_cache, seq_lens, page_table, kv_len)
    if out is None:
        raise ValueError("decode_noalloc needs out")
    out, out_dtype = _output(out, None, q.shape, q.dtype, q.device)
    p = decode_params(q, k_cache, page_table=page_table, kv_len=kv_len, scale=scale, out_dtype=out_dtype,
                      num_ctas=num_ctas)
    st = lib.parallax_decode_noalloc(_ptr(q), _ptr(rho), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                     _ptr(seq_lens), _ptr(out), ctypes.byref(p), _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_decode_noalloc")
    return out


def lla_decode(q, k_cache, v_cache, scale=None, ridge=0.0, *, seq_lens=None, page_table=None, out=None,
               out_dtype=None, rho_out=None, num_ctas=0, kv_len=None):
    """Local Linear Attention with the solved probe (decode).

    Per (sequence, query head): rho* solves (S_KK + ridge I) rho* = kbar - q
    and out = vbar - S_KV^T rho*.  q: [B, Hq, 128] bf16; caches as in
    ``decode`` (bf16).  Returns (out [B, Hq, 128] in ``out_dtype``, default
    bf16; rho* [B, Hq, 128] float32, written into ``rho_out`` when given).
    """
    _check_decode_inputs(q, q, k_cache, v_cache, seq_lens, page_table, kv_len)
    if q.dtype != torch.bfloat16:
        raise TypeError("lla_decode takes bfloat16 queries and caches")
    out, out_dtype = _output(out, out_dtype, q.shape, torch.bfloat16, q.device)
    if rho_out is None:
        rho_out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check_cuda("rho_out", rho_out, torch.float32)
    if tuple(rho_out.shape) != tuple(q.shape):
        raise ValueError(f"rho_out must have shape {tuple(q.shape)}")
    p = decode_params(q, k_cache, page_table=page_table, kv_len=kv_len, scale=scale, out_dtype=out_dtype,
                      num_ctas=num_ctas)
    nbytes = lib.parallax_lla_decode_workspace_size(ctypes.byref(p), float(ridge), 0)
    if nbytes == SIZE_MAX:
        raise ParallaxError(1, "parallax_lla_decode_workspace_size")
    ws, _ = _kept_workspace("lla", q.get_device(), nbytes, 0)   # (written before it is read)
    st = lib.parallax_lla_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seq_lens),
                                 float(ridge), _ptr(rho_out), _ptr(out), _ptr(ws), ws.numel(),
                                 ctypes.byref(p), _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_lla_decode")
    return out, rho_out


def prefill(q, rho, k, v, causal=True, scale=None, *, out=None, out_dtype=None, cta_pair=False):
    """Parallax prefill.  q, rho: [B, H, T, d] bf16; k, v: [B, Hkv, T, d] bf16.
    Row t attends to keys 0..t when causal, else to all T keys.  ``cta_pair``
    runs the two-SM kernel (tcgen05 cta_group::2) instead of one CTA per 128
    rows; the results are the same."""
    for name, t in (("q", q), ("rho", rho), ("k", k), ("v", v)):
        _check_cuda(name, t, torch.bfloat16)
    B, H, T, d = q.shape
    if rho.shape != q.shape or k.shape != v.shape or k.shape[0] != B or k.shape[2] != T or k.shape[3] != d:
        raise ValueError("shape mismatch")
    out, out_dtype = _output(out, out_dtype, q.shape, q.dtype, q.device)
    scale = (1.0 / d ** 0.5) if scale is None else float(scale)
    p = PrefillParams(B, H, k.shape[1], T, d, PLX_BF16, _dtype_code(out_dtype), scale, 1 if causal else 0,
                      1 if cta_pair else 0)
    st = lib.parallax_prefill(_ptr(q), _ptr(rho), _ptr(k), _ptr(v), _ptr(out), ctypes.byref(p),
                              _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_prefill")
    return out


def _prefill_params(q, k, causal, scale, out_dtype, cta_pair=False):
    B, H, T, d = q.shape
    scale = (1.0 / d ** 0.5) if scale is None else float(scale)
    return PrefillParams(B, H, k.shape[1], T, d, PLX_BF16, _dtype_code(out_dtype), scale, 1 if causal else 0,
                         1 if cta_pair else 0)


def _check_prefill_inputs(q, rho, k, v):
    for name, t in (("q", q), ("rho", rho), ("k", k), ("v", v)):
        _check_cuda(name, t, torch.bfloat16)
    B, H, T, d = q.shape
    if rho.shape != q.shape or k.shape != v.shape or k.shape[0] != B or k.shape[2] != T or k.shape[3] != d:
        raise ValueError("shape mismatch")


def prefill_train(q, rho, k, v, causal=True, scale=None, *, out_dtype=None, cta_pair=False):
    """Prefill forward for training: returns (out, vbar, stats).

    vbar: float32 [B, H, T, d], the softmax average of the values of each
    row; stats: float32 [B, H, T, 2], (x, abar) per row with weights
    w_i = 2^(scale * log2(e) * q.k_i - x) and abar = sum_i w_i rho.k_i."""
    _check_prefill_inputs(q, rho, k, v)
    out_dtype = out_dtype or q.dtype
    out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    vbar = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    stats = torch.empty(q.shape[:3] + (2,), dtype=torch.float32, device=q.device)
    p = _prefill_params(q, k, causal, scale, out_dtype, cta_pair)
    st = lib.parallax_prefill_train(_ptr(q), _ptr(rho), _ptr(k), _ptr(v), _ptr(out), _ptr(vbar), _ptr(stats),
                                    ctypes.byref(p), _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_prefill_train")
    return out, vbar, stats


def prefill_backward(q, rho, k, v, out, vbar, stats, dout, causal=True, scale=None, *, grad_dtype=None):
    """Gradients (dq, drho, dk, dv) of a prefill given dout = dL/dout.

    ``out``, ``vbar``, ``stats`` come from prefill_train on the same inputs
    (out in the dtype the loss saw).  Gradients are returned in
    ``grad_dtype`` (default: out's dtype); dk, dv are summed over the query
    heads that share a KV head."""
    _check_prefill_inputs(q, rho, k, v)
    _check_cuda("dout", dout, torch.bfloat16)
    _check_cuda("out", out, out.dtype)
    _check_cuda("vbar", vbar, torch.float32)
    _check_cuda("stats", stats, torch.float32)
    rows = tuple(q.shape[:3])
    for name, t, shape in (("dout", dout, q.shape), ("out", out, q.shape), ("vbar", vbar, q.shape),
                           ("stats", stats, rows + (2,))):
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    grad_dtype = grad_dtype or out.dtype
    if grad_dtype != out.dtype:
        raise ValueError("gradients are returned in out's dtype")
    p = _prefill_params(q, k, causal, scale, out.dtype)
    dq = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    drho = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=q.device)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=q.device)
    nbytes = lib.parallax_prefill_backward_workspace_size(ctypes.byref(p))
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    st = lib.parallax_prefill_backward(_ptr(q), _ptr(rho), _ptr(k), _ptr(v), _ptr(out), _ptr(vbar), _ptr(stats),
                                       _ptr(dout), _ptr(dq), _ptr(drho), _ptr(dk), _ptr(dv), _ptr(ws), nbytes,
                                       ctypes.byref(p), _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_prefill_backward")
    return dq, drho, dk, dv


class ParallaxPrefill(torch.autograd.Function):
    """torch autograd node over prefill_train / prefill_backward (bf16 in and out)."""

    @staticmethod
    def forward(ctx, q, rho, k, v, causal=True, scale=None):
        out, vbar, stats = prefill_train(q, rho, k, v, causal, scale)
        ctx.save_for_backward(q, rho, k, v, out, vbar, stats)
        ctx.causal, ctx.scale = causal, scale
        return out

    @staticmethod
    def backward(ctx, dout):
        q, rho, k, v, out, vbar, stats = ctx.saved_tensors
        grads = prefill_backward(q, rho, k, v, out, vbar, stats, dout.to(torch.bfloat16).contiguous(),
                                 ctx.causal, ctx.scale)
        return grads + (None, None)


def prefill_paged(q, rho, k_cache, v_cache, page_table, cu_seqlens_q, seq_lens, *, max_q_len, scale=None,
                  causal=True, out=None, out_dtype=None):
    """Chunked (append) prefill over the paged cache.

    q, rho: [total_q, H, d] bf16, sequence b's queries at rows
    cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1, which are the LAST positions of
    its seq_lens[b] keys.  k_cache, v_cache: pools [P, Hkv, 64, d] bf16;
    page_table: int32 [B, max_pages]; cu_seqlens_q: int32 [B+1]; seq_lens:
    int32 [B] (all on the device).  ``max_q_len`` bounds every chunk length
    (a host int, so the call needs no device read-back).  Returns out
    [total_q, H, d]; rows outside every sequence are left as allocated.
    """
    for name, t in (("q", q), ("rho", rho), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(name, t, torch.bfloat16)
    for name, t in (("page_table", page_table), ("cu_seqlens_q", cu_seqlens_q), ("seq_lens", seq_lens)):
        _check_cuda(name, t, torch.int32)
    total_q, H, d = q.shape
    P, Hkv, ps, dk = k_cache.shape
    B = seq_lens.shape[0]
    if (rho.shape != q.shape or v_cache.shape != k_cache.shape or dk != d or page_table.dim() != 2
            or page_table.shape[0] != B or cu_seqlens_q.shape != (B + 1,)):
        raise ValueError("shape mismatch")
    out, out_dtype = _output(out, out_dtype, q.shape, q.dtype, q.device)
    scale = (1.0 / d ** 0.5) if scale is None else float(scale)
    p = PrefillPagedParams(B, H, Hkv, d, total_q, int(max_q_len), ps, P, page_table.shape[1], PLX_BF16,
                           _dtype_code(out_dtype), scale, 1 if causal else 0)
    st = lib.parallax_prefill_paged(_ptr(q), _ptr(rho), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                    _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(out), ctypes.byref(p),
                                    _stream_ptr(q.device))
    if st != 0:
        raise ParallaxError(st, "parallax_prefill_paged")
    return out


# ---------------------------------------------------------------- the step around attention

# These calls are made between small kernels, where the host's time counts: parameter
# structs are packed in one step (the formats below are the Structures' layouts), and
# checks read plain integers.
_PAGE_PLAN = struct.Struct("@6i")
_NORM_ROPE = struct.Struct("@8if4xq")
_HEAD_ROWS = struct.Struct("@PPPi4x6q")
_HEAD_GRADS = struct.Struct("@PPP6q")
_APPEND = struct.Struct("@6i4q")
_DECODE = struct.Struct("@10ifi")
for _fmt, _cls in ((_PAGE_PLAN, PagePlanParams), (_NORM_ROPE, NormRopeParams), (_HEAD_ROWS, HeadRows),
                   (_HEAD_GRADS, HeadGrads), (_APPEND, AppendParams), (_DECODE, DecodeParams)):
    assert _fmt.size == ctypes.sizeof(_cls), _cls


def _on(index, name, t, dtype=None):
    """t is a CUDA tensor of device ``index`` and of ``dtype`` (None: any)."""
    if t.get_device() != index:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _cuda_index(name, t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _check_shape(name, t, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_contiguous(name, t):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(index, fn, *args):
    """fn(*args, stream) with device ``index`` current (the library launches on the
    current device), on that device's current stream."""
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        raise ParallaxError(st, fn.__name__)


def _workspace_size(index, status, fn, *args):
    """fn(*args), bytes, with device ``index`` current; ``status`` is raised for what fn refuses."""
    if _current_device() == index:
        nbytes = fn(*args)
    else:
        with torch.cuda.device(index):
            nbytes = fn(*args)
    if nbytes == SIZE_MAX:
        raise ParallaxError(status, fn.__name__)
    return nbytes


_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _capturing(index):
    """Whether device ``index``'s current stream is being captured."""
    if _current_device() == index:
        return _is_capturing()
    with torch.cuda.device(index):
        return _is_capturing()


def _raw(t):
    return None if t is None else t.data_ptr()


PagePlan = collections.namedtuple("PagePlan", "seq_lens cu_seqlens slot_map positions pages_used")


def page_plan(cached_lens, new_lens, page_table, free_pages, *, num_rows, num_pages, free_head=None):
    """The tables of one serving step, from the requests' lengths (parallax_page_plan).

    cached_lens, new_lens: int32 [B], the tokens that each request has in the
    cache and gets now.  page_table: int32 [B, max_pages], updated in place
    with the new pages, which are taken in order from free_pages (int32
    [num_free]) at ``free_head`` (a device int32 tensor of one element; None
    means 0).  ``num_rows`` is the number of packed new-token rows (a host
    int: the sum of new_lens, or more where a captured graph pads) and
    ``num_pages`` the pool's size.

    Returns PagePlan(seq_lens int32 [B], cu_seqlens int32 [B + 1], slot_map
    int64 [num_rows], positions int32 [num_rows], pages_used int32 [1]): what
    decode / decode_q4 / prefill_paged, cache_append and norm_rope take.  Rows
    past the last request have slot and position -1.  Requests that do not fit
    are reported through last_device_error and get seq_lens 0 and slots -1.
    """
    if cached_lens.dim() != 1 or page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("cached_lens and free_pages must be 1-D and page_table 2-D")
    (B,), width = cached_lens.shape, page_table.shape[1]
    _check_contiguous("cached_lens", cached_lens)
    _check_shape("new_lens", new_lens, (B,))
    _check_shape("page_table", page_table, (B, width))
    _check_contiguous("free_pages", free_pages)
    if free_head is not None and free_head.numel() != 1:
        raise ValueError("free_head must hold one element")
    index = _cuda_index("cached_lens", cached_lens)
    i32 = torch.int32
    _on(index, "cached_lens", cached_lens, i32)
    _on(index, "new_lens", new_lens, i32)
    _on(index, "page_table", page_table, i32)
    _on(index, "free_pages", free_pages, i32)
    if free_head is not None:
        _on(index, "free_head", free_head, i32)
    num_rows = int(num_rows)
    # one allocation, the slots (8-byte entries) first
    slots, seq_lens, cu, positions, used = cached_lens.new_empty(3 * num_rows + 2 * B + 2).split_with_sizes(
        (2 * num_rows, B, B + 1, num_rows, 1))
    slots = slots.view(torch.int64)
    _call(index, lib.parallax_page_plan, cached_lens.data_ptr(), new_lens.data_ptr(), page_table.data_ptr(),
          free_pages.data_ptr(), _raw(free_head), seq_lens.data_ptr(), cu.data_ptr(), slots.data_ptr(),
          positions.data_ptr(), used.data_ptr(),
          _PAGE_PLAN.pack(B, num_rows, PAGE_SIZE, num_pages, width, free_pages.shape[0]))
    return PagePlan(seq_lens, cu, slots, positions, used)


def _dense_strides(shape):
    """Element strides (batch entry, token, head) of contiguous [B, H, T, d] or packed [N, H, d] rows."""
    if len(shape) == 4:
        _, h, t, d = shape
        return h * t * d, d, t * d
    return 0, shape[1] * shape[2], shape[2]


def _head_strides(name, t):
    """The same of a tensor that is not contiguous (0 for a dimension of one entry,
    whatever torch says there)."""
    s, n = t.stride(), t.shape
    if s[-1] != 1 and t.numel() > 0:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if len(n) == 4:
        return s[0] if n[0] > 1 else 0, s[2] if n[2] > 1 else 0, s[1] if n[1] > 1 else 0
    return 0, s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0


def _norm_rope_call(q, rho, k, cos, sin, positions, weights, eps, norm, interleaved):
    """Checks and parameters that the two directions share: (sets, params, device index), a
    set being (name, x, shape, its contiguous strides, the input part of its plx_head_rows:
    address, weight's address, heads and strides)."""
    shape = q.shape
    batched = len(shape) == 4
    if not batched and len(shape) != 3:
        raise ValueError(f"q must be [B, H, T, d] or packed [N, H, d], got {tuple(shape)}")
    d = shape[-1]
    B, T = (shape[0], shape[2]) if batched else (1, shape[0])
    index, dtype = _cuda_index("q", q), q.dtype
    dense = _dense_strides(shape)
    tensors = [("q", q, shape, dense, weights[0])]
    if rho is not None:
        if rho.shape != shape:
            raise ValueError(f"rho must have q's shape {tuple(shape)}, got {tuple(rho.shape)}")
        _on(index, "rho", rho, dtype)
        tensors.append(("rho", rho, shape, dense, weights[1]))
    if k is not None:
        ks = k.shape
        if len(ks) != len(shape) or ks[-1] != d or ks[0] != shape[0] or (batched and ks[2] != T):
            raise ValueError(f"k's rows {tuple(ks)} do not match q's {tuple(shape)}")
        _on(index, "k", k, dtype)
        tensors.append(("k", k, ks, _dense_strides(ks), weights[2]))
    sets = []
    for name, x, n, dense, w in tensors:
        at = 0
        if w is not None:
            if not norm:
                raise ValueError(f"{name}_weight needs norm=True")
            _check_shape(name + "_weight", w, (d,))
            _on(index, name + "_weight", w, dtype)
            at = w.data_ptr()
        sets.append((name, x, n, dense,
                     (x.data_ptr(), at, n[1], dense if x.is_contiguous() else _head_strides(name, x))))
    rot, max_pos = 0, 0
    if cos is not None and sin is not None:
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [max_pos, rot_dim / 2] and alike")
        if not (cos.is_contiguous() and sin.is_contiguous()):
            raise ValueError("cos and sin must be contiguous")
        max_pos, rot = cos.shape
        rot *= 2
        _on(index, "cos", cos, torch.float32)
        _on(index, "sin", sin, torch.float32)
    elif cos is not None or sin is not None:
        raise ValueError("cos and sin come together")
    pos_stride = 0
    if positions is not None:
        ps = positions.shape
        if ps != (T,) and not (batched and ps == (B, T)):
            raise ValueError(f"positions must have shape {(T,)}{f' or {(B, T)}' if batched else ''}, got {tuple(ps)}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        _on(index, "positions", positions, torch.int32)
        pos_stride = T if len(ps) == 2 else 0
    elif rot and T > max_pos:
        raise ValueError(f"{T} tokens need as many rows of cos and sin, got {max_pos}")
    p = _NORM_ROPE.pack(B, T, d, rot, max_pos, 1 if interleaved else 0, 1 if norm else 0, _dtype_code(dtype), eps,
                        pos_stride)
    return sets, p, index


def norm_rope(q, rho, k, cos, sin, positions=None, *, q_weight=None, rho_weight=None, k_weight=None, eps=1e-6,
              norm=True, interleaved=False, out=None):
    """RMS norm of every query, probe and key head with the position rotation, in one pass.

    q, rho: [B, H, T, d], or packed [N, H, d]; k: the same with its own heads
    (rho and k may be None).  Any strides with a contiguous last dimension (16-byte
    aligned rows), so that slices of one fused projection need no copy.
    cos, sin: float32 [max_pos, rot_dim / 2] (None: no rotation), for pairs
    (f, f + rot_dim / 2), or (2f, 2f + 1) with ``interleaved``.  positions:
    int32 [T], [B, T] or packed [N] (None: row t has position t); rows at
    position -1 are skipped.  Weights [d] of q's dtype, or None for ones;
    norm=False only rotates.  ``out``: a tuple of tensors to write (an entry
    may be the input itself: in place).  Returns (q, rho, k), None where the
    input is.
    """
    sets, p, index = _norm_rope_call(q, rho, k, cos, sin, positions, (q_weight, rho_weight, k_weight), eps, norm,
                                     interleaved)
    done, rows = {"q": None, "rho": None, "k": None}, b""
    given = dict(zip(done, out)) if out is not None else None
    for name, x, shape, y_strides, (at, weight, heads, strides) in sets:
        if given is None:
            y = torch.empty_like(x, memory_format=torch.contiguous_format)
        else:
            y = given.get(name)
            if y is None or y.shape != shape:
                raise ValueError(f"out's {name} must have shape {tuple(shape)}")
            _on(index, "out's " + name, y, x.dtype)
            if not y.is_contiguous():
                y_strides = _head_strides("out's " + name, y)
        done[name] = y
        rows += _HEAD_ROWS.pack(at, y.data_ptr(), weight, heads, *strides, *y_strides)
    _call(index, lib.parallax_norm_rope, rows, len(sets), _raw(positions), _raw(cos), _raw(sin), p)
    return tuple(done.values())


def norm_rope_backward(dq, drho, dk, q, rho, k, cos, sin, positions=None, *, q_weight=None, rho_weight=None,
                       k_weight=None, eps=1e-6, norm=True, interleaved=False):
    """Gradients of norm_rope: (dq, drho, dk, dq_weight, drho_weight, dk_weight).

    dq, drho, dk: the gradients of norm_rope's results, shaped and typed like
    q, rho, k (the forward's inputs).  Weight gradients are float32 [d], summed
    over all rows; None without norm, and everything is None for a set that is.
    Without given weights, the gradients of weights of one are returned.
    """
    sets, p, index = _norm_rope_call(q, rho, k, cos, sin, positions, (q_weight, rho_weight, k_weight), eps, norm,
                                     interleaved)
    names = ("q", "rho", "k")
    incoming, dxs, dws = dict(zip(names, (dq, drho, dk))), dict.fromkeys(names), dict.fromkeys(names)
    rows = grads = b""
    if norm:
        size = len(sets), q.shape[-1]
        # (without a dtype the allocation takes a third less of the host)
        dw = q.new_empty(size, dtype=torch.float32) if cos is None else cos.new_empty(size)
        dws.update(zip([one[0] for one in sets], dw.unbind()))
    for name, x, shape, dense, (at, weight, heads, strides) in sets:
        dy = incoming[name]
        if dy is None or dy.shape != shape:
            raise ValueError(f"d{name} must have shape {tuple(shape)}")
        if dy.get_device() != index or dy.dtype is not x.dtype:
            _on(index, "d" + name, dy, x.dtype)
        dx = dxs[name] = torch.empty_like(x, memory_format=torch.contiguous_format)
        rows += _HEAD_ROWS.pack(at, 0, weight, heads, *strides, 0, 0, 0)
        grads += _HEAD_GRADS.pack(dy.data_ptr(), dx.data_ptr(), dws[name].data_ptr() if norm else 0,
                                  *(dense if dy.is_contiguous() else _head_strides("d" + name, dy)), *dense)
    ws, nbytes = None, 0
    if norm:
        nbytes = _workspace_size(index, 2, lib.parallax_norm_rope_backward_workspace_size, p, len(sets))
        ws = q.new_empty(nbytes // q.element_size())   # (a multiple of 4 bytes)
    _call(index, lib.parallax_norm_rope_backward, rows, grads, len(sets), _raw(positions), _raw(cos), _raw(sin),
          _raw(ws), nbytes, p)
    return tuple(dxs.values()) + tuple(dws.values())


class NormRope(torch.autograd.Function):
    """torch autograd node over norm_rope / norm_rope_backward:
    apply(q, rho, k, q_weight, rho_weight, k_weight, cos, sin, positions, eps, norm, interleaved)
    returns (q, rho, k).  cos and sin get no gradient."""

    @staticmethod
    def forward(ctx, q, rho, k, q_weight, rho_weight, k_weight, cos, sin, positions=None, eps=1e-6, norm=True,
                interleaved=False):
        # padding rows are not written: they are zero here
        out = None if positions is None else tuple(None if x is None else torch.zeros(x.shape, dtype=x.dtype,
                                                                                      device=x.device)
                                                   for x in (q, rho, k))
        out = norm_rope(q, rho, k, cos, sin, positions, q_weight=q_weight, rho_weight=rho_weight, k_weight=k_weight,
                        eps=eps, norm=norm, interleaved=interleaved, out=out)
        ctx.save_for_backward(q, rho, k, q_weight, rho_weight, k_weight, cos, sin, positions)
        ctx.options = dict(eps=eps, norm=norm, interleaved=interleaved)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, drho, dk):
        q, rho, k, qw, rw, kw, cos, sin, positions = ctx.saved_tensors
        grads = [None if x is None else (torch.zeros_like(x) if g is None else _dense_rows(g.to(x.dtype)))
                 for x, g in ((q, dq), (rho, drho), (k, dk))]
        dx = norm_rope_backward(*grads, q, rho, k, cos, sin, positions, q_weight=qw, rho_weight=rw, k_weight=kw,
                                **ctx.options)
        dw = tuple(None if w is None else g.to(w.dtype) for w, g in zip((qw, rw, kw), dx[3:]))
        return dx[:3] + dw + (None,) * 6


def _dense_rows(g):
    """g itself where the library can read its rows (broadcast and unaligned gradients are copied)."""
    unit = 16 // g.element_size()
    ok = g.stride(-1) == 1 and g.data_ptr() % 16 == 0 and all(s % unit == 0 for s in g.stride()[:-1])
    return g if ok else g.contiguous()


def _append_params(k, v, slot_map, num_pages, num_kv_heads, head_dim, dtype, index):
    """Checks of k, v [N, Hkv, d] and slot_map [N]; the packed parameters."""
    shape = k.shape
    if len(shape) != 3 or shape[1] != num_kv_heads or shape[2] != head_dim:
        raise ValueError(f"k must be [N, {num_kv_heads}, {head_dim}], got {tuple(shape)}")
    n = shape[0]
    if v.shape != shape:
        raise ValueError(f"v must have k's shape {tuple(shape)}, got {tuple(v.shape)}")
    ks, vs = k.stride(), v.stride()
    if n > 0 and (ks[2] != 1 or vs[2] != 1):
        raise ValueError("the last dimension of k and v must be contiguous")
    _check_shape("slot_map", slot_map, (n,))
    _on(index, "k", k, dtype)
    _on(index, "v", v, dtype)
    _on(index, "slot_map", slot_map, torch.int64)
    row, head = n > 1, num_kv_heads > 1    # (a dimension of one entry has any stride)
    return _APPEND.pack(n, num_kv_heads, head_dim, PAGE_SIZE, num_pages, _dtype_code(dtype), ks[0] * row,
                        ks[1] * head, vs[0] * row, vs[1] * head)


def cache_append(k, v, slot_map, k_cache, v_cache):
    """Writes a step's keys and values into the paged pools, in place.

    k, v: [N, Hkv, d] (row and head strides are free, rows 16-byte aligned), of
    the pools' dtype (bfloat16 or float32); slot_map: int64 [N], row r goes to
    row slot % 64 of page slot // 64 (page_plan's map; -1 skips); pools
    [P, Hkv, 64, d] as decode and prefill_paged read them.  Slots are distinct.
    """
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[2] != PAGE_SIZE:
        raise ValueError(f"pools must be [P, Hkv, {PAGE_SIZE}, d] and alike, got {tuple(k_cache.shape)} and "
                         f"{tuple(v_cache.shape)}")
    P, Hkv, _, d = k_cache.shape
    _check_shape("k_cache", k_cache, k_cache.shape)
    _check_shape("v_cache", v_cache, v_cache.shape)
    index = _cuda_index("k_cache", k_cache)
    _on(index, "v_cache", v_cache, k_cache.dtype)
    p = _append_params(k, v, slot_map, P, Hkv, d, k_cache.dtype, index)
    _call(index, lib.parallax_cache_append, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), p)


def q4_block_bytes(head_dim: int) -> int:
    """Bytes of one (page, KV head) block of the 4-bit cache."""
    n = lib.parallax_q4_block_bytes(int(head_dim))
    if n == 0:
        raise ParallaxError(2, "parallax_q4_block_bytes")
    return n


def _q4_head_dim(dtype, nbytes):
    """The head_dim that a 4-bit cache's block size says."""
    if dtype is not torch.uint8:
        raise TypeError(f"a 4-bit cache is a uint8 tensor, got {dtype}")
    for d in (64, 128):
        if nbytes == 72 * d:
            return d
    raise ValueError(f"a 4-bit cache's blocks have {q4_block_bytes(64)} or {q4_block_bytes(128)} bytes, got {nbytes}")


def q4_cache(num_pages, num_kv_heads, head_dim, device="cuda"):
    """An empty 4-bit pool [num_pages, num_kv_heads, q4_block_bytes(head_dim)] (uint8)."""
    return torch.zeros(num_pages, num_kv_heads, q4_block_bytes(head_dim), dtype=torch.uint8, device=device)


def _q4_pool(kv_cache):
    if kv_cache.dim() != 3:
        raise ValueError(f"a 4-bit pool is [P, Hkv, block bytes], got {tuple(kv_cache.shape)}")
    _check_contiguous("kv_cache", kv_cache)
    P, Hkv, nbytes = kv_cache.shape
    return P, Hkv, _q4_head_dim(kv_cache.dtype, nbytes)


def cache_append_q4(k, v, slot_map, kv_cache):
    """Quantises a step's keys and values to 4 bits into the pool, in place.

    k, v: [N, Hkv, d] bfloat16; slot_map as for cache_append; kv_cache: uint8
    [P, Hkv, q4_block_bytes(d)] (see q4_cache; parallax.h has the layout).
    Each 64 columns of a row share a scale and a minimum.
    """
    P, Hkv, d = _q4_pool(kv_cache)
    index = _cuda_index("kv_cache", kv_cache)
    p = _append_params(k, v, slot_map, P, Hkv, d, torch.bfloat16, index)
    _call(index, lib.parallax_cache_append_q4, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), kv_cache.data_ptr(), p)


def cache_gather_q4(kv_cache, slot_map, *, out_dtype=torch.bfloat16, out=None):
    """The keys and values at the slots, dequantised: (k, v), each [N, Hkv, d]
    of ``out_dtype`` (bfloat16 or float32).  Rows at slot -1 are left as
    allocated (``out``: the two tensors to write)."""
    P, Hkv, d = _q4_pool(kv_cache)
    index = _cuda_index("kv_cache", kv_cache)
    if out is None:
        if slot_map.dim() != 1:
            raise ValueError(f"slot_map must be 1-D, got {tuple(slot_map.shape)}")
        shape = (slot_map.shape[0], Hkv, d)
        k = torch.empty(shape, dtype=out_dtype, device=kv_cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
    p = _append_params(k, v, slot_map, P, Hkv, d, k.dtype, index)
    _call(index, lib.parallax_cache_gather_q4, kv_cache.data_ptr(), slot_map.data_ptr(), k.data_ptr(), v.data_ptr(), p)
    return k, v


def decode_q4_workspace(q, kv_cache, *, page_table=None, kv_len=None, num_ctas=0):
    """A zeroed workspace for decode_q4 calls of these shapes (pass it as
    ``workspace``), for a graph that otherwise clears the counters when it starts.
    Calls that share one must not overlap on the GPU."""
    B, Hkv = q.shape[0], kv_cache.shape[1]
    if kv_len is None:
        kv_len = PAGE_SIZE * (kv_cache.shape[2] if page_table is None else page_table.shape[1])
    paged = page_table is not None
    p = _DECODE.pack(B, q.shape[1], Hkv, q.shape[2], int(kv_len), PAGE_SIZE if paged else 0,
                     kv_cache.shape[0] if paged else 0, page_table.shape[1] if paged else 0, PLX_BF16, PLX_BF16, 1.0,
                     int(num_ctas))
    nbytes = _workspace_size(_cuda_index("q", q), 1, lib.parallax_decode_q4_workspace_size, p, 0)
    return torch.zeros(nbytes, dtype=torch.uint8, device=q.device)


def decode_q4(q, rho, kv_cache, scale=None, *, seq_lens=None, page_table=None, out=None, out_dtype=None, num_ctas=0,
              kv_len=None, workspace=None):
    """Parallax decode over the 4-bit cache.

    q, rho: [B, Hq, d] bfloat16.  Paged: kv_cache uint8 [P, Hkv, block bytes],
    page_table int32 [B, max_pages] and seq_lens int32 [B].  Contiguous:
    kv_cache [B, Hkv, ceil(kv_len / 64), block bytes] with ``kv_len`` (default:
    all of its pages' tokens) and optional seq_lens.  Returns out [B, Hq, d] in
    ``out_dtype`` (default bfloat16).  ``workspace``: see decode_q4_workspace
    (default: one that the binding keeps for the stream or the capture).
    """
    shape, blocks = q.shape, kv_cache.shape
    if len(shape) != 3 or rho.shape != shape:
        raise ValueError(f"q and rho must be [B, Hq, d] and alike, got {tuple(shape)} and {tuple(rho.shape)}")
    B, Hq, d = shape
    paged = page_table is not None
    if len(blocks) != (3 if paged else 4):
        raise ValueError("a paged 4-bit cache is [P, Hkv, block bytes] and a contiguous one "
                         f"[B, Hkv, pages, block bytes], got {tuple(blocks)}")
    cache_dim = _q4_head_dim(kv_cache.dtype, blocks[-1])
    if cache_dim != d:
        raise ValueError(f"the cache's head_dim {cache_dim} differs from the queries' {d}")
    Hkv, num_pages, width = blocks[1], 0, 0
    if Hkv < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads do not split into {Hkv} KV heads")
    if paged:
        num_pages, width = blocks[0], page_table.shape[-1]
        kv_len = width * PAGE_SIZE if kv_len is None else int(kv_len)
        if kv_len > width * PAGE_SIZE:
            raise ValueError(f"kv_len {kv_len} exceeds the page table's {width} pages")
        if seq_lens is None:
            raise ValueError("a paged cache needs seq_lens")
        _check_shape("page_table", page_table, (B, width))
    else:
        if blocks[0] != B:
            raise ValueError(f"a contiguous cache holds one sequence per row: {blocks[0]} != {B}")
        pages = blocks[2]
        kv_len = pages * PAGE_SIZE if kv_len is None else int(kv_len)
        if (kv_len + PAGE_SIZE - 1) // PAGE_SIZE != pages:
            raise ValueError(f"kv_len {kv_len} does not fill the cache's {pages} pages of {PAGE_SIZE} tokens "
                             "(use seq_lens for shorter sequences)")
    if seq_lens is not None:
        _check_shape("seq_lens", seq_lens, (B,))
    _check_contiguous("q", q)
    _check_contiguous("rho", rho)
    _check_contiguous("kv_cache", kv_cache)
    index = _cuda_index("q", q)
    _on(index, "q", q, torch.bfloat16)
    _on(index, "rho", rho, torch.bfloat16)
    _on(index, "kv_cache", kv_cache)
    if page_table is not None:
        _on(index, "page_table", page_table, torch.int32)
    if seq_lens is not None:
        _on(index, "seq_lens", seq_lens, torch.int32)
    if out is None and (out_dtype is None or out_dtype is torch.bfloat16):
        out, out_dtype = torch.empty_like(q), torch.bfloat16
    else:
        out, out_dtype = _output(out, out_dtype, q.shape, torch.bfloat16, q.device)
        _on(index, "out", out)
    p = _DECODE.pack(B, Hq, Hkv, d, kv_len, PAGE_SIZE if paged else 0, num_pages, width, PLX_BF16,
                     _dtype_code(out_dtype), (1.0 / d ** 0.5) if scale is None else float(scale), int(num_ctas))
    if workspace is not None:
        _on(index, "workspace", workspace, torch.uint8)
        _check_shape("workspace", workspace, (workspace.numel(),))
    else:
        nbytes = _workspace_size(index, 1, lib.parallax_decode_q4_workspace_size, p, 0)
        counters = (4 * B * Hkv + 255) & ~255   # at the end
        workspace, _ = _kept_workspace("q4", index, nbytes - counters, counters)
    _call(index, lib.parallax_decode_q4, q.data_ptr(), rho.data_ptr(), kv_cache.data_ptr(), _raw(page_table),
          _raw(seq_lens), out.data_ptr(), workspace.data_ptr(), workspace.numel(), p)
    return out


def last_device_error(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device error word."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    code = ctypes.c_int32(0)
    st = lib.parallax_last_device_error(_stream_ptr(device), ctypes.byref(code))
    if st != 0:
        raise ParallaxError(st, "parallax_last_device_error")
    return code.value


def set_wait_limit_ns(limit_ns: int) -> int:
    """Sets the pipeline wait limit of the current device's kernels (ns) and
    returns the previous one (see parallax_set_wait_limit_ns)."""
    prev = ctypes.c_uint64(0)
    st = lib.parallax_set_wait_limit_ns(int(limit_ns), ctypes.byref(prev))
    if st != 0:
        raise ParallaxError(st, "parallax_set_wait_limit_ns")
    return prev.value
