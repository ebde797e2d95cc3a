"""Thin ctypes binding over ``libattn_b200.so`` (C ABI in ``include/attn.h``).

Argument marshalling only: tensors are checked for dtype/device/contiguity, their data pointers and
the current CUDA stream are passed to the C entry points, and a non-zero status becomes an
``AttnError``. PyTorch supplies device memory and streams; every step of the attention itself runs
in the library's kernels. There is no fallback: if the library is missing the call fails.

``stream`` (a torch stream or a handle; default the current stream) is where a call runs. Its inputs
have to be ready there and to stay until it is done; what the call allocates itself, results and
workspaces, is that stream's memory and may be dropped at any time.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libattn_b200.so"
library_path = os.path.join(_PKG, LIB_NAME)

ATTN_OK = 0
STATUS_NAMES = {
    0: "ATTN_OK", -1: "ATTN_ERR_NULL", -2: "ATTN_ERR_SHAPE", -3: "ATTN_ERR_GQA", -4: "ATTN_ERR_HEADDIM",
    -5: "ATTN_ERR_ALIGN", -6: "ATTN_ERR_CAUSAL_SQ_GT_SKV", -7: "ATTN_ERR_ARCH", -8: "ATTN_ERR_WORKSPACE",
    -9: "ATTN_ERR_LAUNCH", -10: "ATTN_ERR_DEVICE_TIMEOUT", -11: "ATTN_ERR_SCALE", -12: "ATTN_ERR_CUDA",
    -13: "ATTN_ERR_SCRATCH_LIMIT", -14: "ATTN_ERR_ROTATION", -15: "ATTN_ERR_EPS",
}
EXPORTED = ("attn_fwd", "attn_fwd_ex", "attn_fwd_host", "attn_fwd_strided", "attn_decode_ctas", "attn_status_string", "attn_version",
            "attn_device_status", "attn_decode_noalloc", "attn_decode_paged", "attn_prefill_paged", "attn_bwd", "attn_decode_fp8", "attn_prefill_fp8",
            "attn_decode_paged_fp8", "attn_lse_merge", "attn_qk_norm_rope", "attn_qk_norm_rope_bwd", "attn_append_paged",
            "attn_append_paged_fp8", "attn_decode_prefix", "attn_decode_prefix_workspace")

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load_library(path: str | None = None):
    """Load the library once. Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or library_path
        if not os.path.exists(p):
            raise RuntimeError(f"{LIB_NAME} is not built (expected at {p}); "
                               "run `python -m causal_attention_attn_b200.build`")
        lib = ctypes.CDLL(p)
        i, f, vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        lib.attn_fwd.restype = i
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.attn_fwd_ex.restype = i
        lib.attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
        lib.attn_fwd_host.restype = i
        lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        ll3 = ctypes.POINTER(ctypes.c_longlong)
        lib.attn_fwd_strided.restype = i
        lib.attn_fwd_strided.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ll3, ll3, ll3, ll3, f, i, vp]
        lib.attn_decode_ctas.restype = i
        lib.attn_decode_ctas.argtypes = [i, i, i, i, i]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_status_string.argtypes = [i]
        lib.attn_version.restype = i
        lib.attn_version.argtypes = []
        lib.attn_device_status.restype = i
        lib.attn_device_status.argtypes = [vp]
        lib.attn_decode_noalloc.restype = i
        lib.attn_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
        lib.attn_decode_paged.restype = i
        lib.attn_bwd.restype = i
        lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
        lib.attn_prefill_paged.restype = i
        lib.attn_prefill_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, vp]
        lib.attn_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        lib.attn_prefill_fp8.restype = i
        lib.attn_prefill_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.attn_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
        lib.attn_lse_merge.restype = i
        lib.attn_lse_merge.argtypes = [vp, vp, vp, vp, vp, ctypes.c_longlong, i, vp]
        lib.attn_qk_norm_rope.restype = i
        lib.attn_qk_norm_rope.argtypes = [vp] * 9 + [i] * 5 + [ll3] * 4 + [i, i, i, f, vp]
        lib.attn_qk_norm_rope_bwd.restype = i
        lib.attn_qk_norm_rope_bwd.argtypes = [vp] * 14 + [i] * 5 + [ll3] * 6 + [i, i, i, f, vp]
        lib.attn_append_paged.restype = i
        lib.attn_append_paged.argtypes = [vp] * 14 + [i] * 4 + [ll3] * 4 + [i] * 6 + [f, vp]
        lib.attn_append_paged_fp8.restype = i
        lib.attn_append_paged_fp8.argtypes = [vp] * 16 + [i] * 4 + [ll3] * 4 + [i] * 6 + [f, vp]
        lib.attn_decode_prefix.restype = i
        lib.attn_decode_prefix.argtypes = [vp] * 10 + [ctypes.c_longlong] + [i] * 9 + [f, vp]
        lib.attn_decode_prefix_workspace.restype = ctypes.c_longlong
        lib.attn_decode_prefix_workspace.argtypes = [i] * 5
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def _check(status: int):
    if status != ATTN_OK:
        raise AttnError(status, status_string(status))


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _side(stream, dev: int):
    """The stream that a call on `stream` allocates for, or None when that is the current one."""
    if stream is None:
        return None
    handle = _stream_handle(stream)
    if handle == torch._C._cuda_getCurrentRawStream(dev):
        return None
    if handle in (0, 1):  # both name the legacy default stream
        return torch.cuda.default_stream(dev)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device=dev)


def _made(side, *slots):
    """The tensors of a call, each slot (the caller's or None; what makes one; of what). The caching
    allocator orders a block's next use behind the stream that it was allocated on, so with a `side` stream
    what is made is that stream's: what had the block before is behind the call, and what gets it when the
    result is dropped, behind the call too. The current stream, where a result is usually read next, is
    recorded beside it."""
    if side is None:
        return [make(of) if given is None else given for given, make, of in slots]
    current = torch.cuda.current_stream(side.device)
    with torch.cuda.stream(side):
        made = [make(of) if given is None else given for given, make, of in slots]
    for t, slot in zip(made, slots):
        if slot[0] is None:
            t.record_stream(current)
    return made


def _lse_of(q):
    return torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)


def _check_tensor(name, t, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_rows(name, t, dtype):
    """A [batch, head, row, dim] tensor in any layout whose last (dim) axis is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dims, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last (head-dim) axis")


def _strides3(t):
    """(batch, head, row) element strides of a [B, H, S, D] view; an axis of extent 1 gets D
    (its stride is never used, and the library wants a multiple of 8)."""
    D = int(t.shape[-1])
    return tuple(int(t.stride(i)) if t.shape[i] > 1 else D for i in range(3))


def attn_fwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, Hq: int, Hkv: int,
                 Sq: int, Skv: int, D: int, scale: float, causal: bool, stream: int = 0,
                 decode_ctas: int = 0) -> int:
    """Call the C entry point with raw pointers; returns the status code (no exception)."""
    lib = load_library()
    if decode_ctas:
        return lib.attn_fwd_ex(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, Hq, Hkv, Sq, Skv, D, float(scale),
                               int(causal), int(decode_ctas), stream)
    return lib.attn_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, Hq, Hkv, Sq, Skv, D, float(scale), int(causal),
                        stream)


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None, causal: bool = True,
             out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
             decode_ctas: int = 0):
    """Fused causal attention forward on the GPU.

    q: [B, Hq, Sq, D], k/v: [B, Hkv, Skv, D], bf16, on one CUDA device, each either contiguous or any
    view with a contiguous last axis (e.g. a token-major [B, S, H, D] tensor passed as
    ``x.transpose(1, 2)``); views go through ``attn_fwd_strided``. ``out`` (shape of q) may be such a
    view too. Returns (o [B, Hq, Sq, D] bf16, lse [B, Hq, Sq] fp32, contiguous). ``scale``
    defaults to 1/sqrt(D).
    """
    _check_rows("q", q, torch.bfloat16)
    _check_rows("k", k, torch.bfloat16)
    _check_rows("v", v, torch.bfloat16)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if scale is None:
        scale = D ** -0.5
    if out is not None:
        _check_rows("out", out, torch.bfloat16)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, 3)
        if tuple(lse.shape) != (B, Hq, Sq):
            raise ValueError("lse must be [B, Hq, Sq]")
    out, lse = _made(_side(stream, q.get_device()), (out, _new_rows, q), (lse, _lse_of, q))
    strided = not all(t.is_contiguous() for t in (q, k, v, out))
    with torch.cuda.device(q.device):
        if strided:
            arr = [(ctypes.c_longlong * 3)(*_strides3(t)) for t in (q, k, v, out)]
            rc = load_library().attn_fwd_strided(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                 lse.data_ptr(), B, Hq, Hkv, Sq, Skv, D, *arr, float(scale),
                                                 int(causal), _stream_handle(stream))
        else:
            rc = attn_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv,
                              Sq, Skv, D, scale, causal, _stream_handle(stream), decode_ctas)
    _check(rc)
    return out, lse


def attn_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
                  causal: bool = True, device="cuda", stream=None, out_host=None, lse_host=None, dev_bufs=None):
    """End-to-end call on HOST tensors through ``attn_fwd_host``: the library copies q, k, v in,
    runs the attention and copies o and lse out, slice by slice, with the copies of one slice
    overlapping the attention of the next (so pinned inputs and outputs matter: pageable memory
    works but does not overlap).

    ``dev_bufs`` optionally supplies the device staging tensors (q, k, v, o, lse) so that a loop of
    calls does not allocate. Returns host (o, lse); the call synchronises on the stream before
    returning.
    """
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu" or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be a bf16 host tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [batch, head, row, dim] tensor")
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Skv, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"k {tuple(k.shape)} / v {tuple(v.shape)} do not match q {tuple(q.shape)}")
    if scale is None:
        scale = D ** -0.5
    stream = stream or torch.cuda.current_stream(device)
    if dev_bufs is None:
        dev = torch.device(device).index
        slots = [(None, functools.partial(torch.empty, dtype=torch.bfloat16, device=device), t.shape) for t in (q, k, v, q)]
        slots.append((None, functools.partial(torch.empty, dtype=torch.float32, device=device), q.shape[:3]))
        dev_bufs = _made(_side(stream, torch.cuda.current_device() if dev is None else dev), *slots)
    qd, kd, vd, od, ld = dev_bufs
    if out_host is None:
        out_host = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty((B, Hq, Sq), dtype=torch.float32, pin_memory=True)
    for name, t in (("out_host", out_host), ("lse_host", lse_host)):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    rc = load_library().attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out_host.data_ptr(),
                                      lse_host.data_ptr(), qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), od.data_ptr(),
                                      ld.data_ptr(), B, Hq, Hkv, Sq, Skv, D, float(scale), int(bool(causal)),
                                      _stream_handle(stream))
    _check(rc)
    stream.synchronize()
    return out_host, lse_host


def attn_decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Single-token decode through ``attn_decode_noalloc``: the library allocates nothing (its
    scratch is a fixed device array). For callers that must not have the library call cudaMalloc.
    ``out`` and ``lse`` should be passed by such callers; when omitted they are created here with
    torch. q: [B, Hq, 1, D]; k/v: [B, Hkv, Skv, D]. Returns (o, lse)."""
    _check_tensor("q", q, torch.bfloat16, 4)
    _check_tensor("k", k, torch.bfloat16, 4)
    _check_tensor("v", v, torch.bfloat16, 4)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if Sq != 1 or tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D:
        raise ValueError(f"expected q [B,Hq,1,D] and k, v [B,Hkv,Skv,D]; got {tuple(q.shape)}, {tuple(k.shape)}")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_decode_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                lse.data_ptr(), B, Hq, Hkv, Skv, D, float(scale),
                                                _stream_handle(stream))
    _check(rc)
    return out, lse


def attn_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, max_seq_len: int, scale: float | None = None,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
                      decode_ctas: int = 0):
    """Single-token decode over a paged, variable-length KV cache through ``attn_decode_paged``.
    q: [B, Hq, 1, 128] bf16; k_pages, v_pages: [num_pages, Hkv, page_size, 128] bf16;
    block_table: int32 [B, pages_per_seq]; seq_lens: int32 [B] (all on the GPU); max_seq_len: a
    host-side bound of the lengths. Returns (o [B, Hq, 1, 128], lse [B, Hq, 1])."""
    _check_tensor("q", q, torch.bfloat16, 4)
    _check_tensor("k_pages", k_pages, torch.bfloat16, 4)
    _check_tensor("v_pages", v_pages, torch.bfloat16, 4)
    _check_tensor("block_table", block_table, torch.int32, 2)
    _check_tensor("seq_lens", seq_lens, torch.int32, 1)
    B, Hq, Sq, D = q.shape
    num_pages, Hkv, page_size, Dk = k_pages.shape
    if Sq != 1 or tuple(v_pages.shape) != tuple(k_pages.shape) or Dk != D:
        raise ValueError(f"expected q [B,Hq,1,D] and k, v pages [P,Hkv,page,D]; got {tuple(q.shape)}, "
                         f"{tuple(k_pages.shape)}")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row / entry per batch element")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                              block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                                              lse.data_ptr(), B, Hq, Hkv, num_pages, page_size,
                                              int(block_table.shape[1]), int(max_seq_len), float(scale),
                                              int(decode_ctas), _stream_handle(stream))
    _check(rc)
    return out, lse


def attn_prefill_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, max_seq_len: int, scale: float | None = None, causal: bool = True,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Chunked prefill over a paged, variable-length KV cache through ``attn_prefill_paged``:
    sequence b's Sq new queries attend to its first seq_lens[b] cached keys, the causal mask aligned
    to the last Sq of them. q: [B, Hq, Sq, 128] bf16; k_pages, v_pages: [num_pages, Hkv, page_size,
    128] bf16; block_table int32 [B, pages_per_seq]; seq_lens int32 [B] (all on the GPU).
    Returns (o [B, Hq, Sq, 128], lse [B, Hq, Sq])."""
    _check_tensor("q", q, torch.bfloat16, 4)
    _check_tensor("k_pages", k_pages, torch.bfloat16, 4)
    _check_tensor("v_pages", v_pages, torch.bfloat16, 4)
    _check_tensor("block_table", block_table, torch.int32, 2)
    _check_tensor("seq_lens", seq_lens, torch.int32, 1)
    B, Hq, Sq, D = q.shape
    num_pages, Hkv, page_size, Dk = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape) or Dk != D:
        raise ValueError(f"expected q [B,Hq,Sq,D] and k, v pages [P,Hkv,page,D]; got {tuple(q.shape)}, "
                         f"{tuple(k_pages.shape)}")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row / entry per batch element")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_prefill_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                               block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                                               lse.data_ptr(), B, Hq, Hkv, Sq, num_pages, page_size,
                                               int(block_table.shape[1]), int(max_seq_len), float(scale),
                                               int(bool(causal)), _stream_handle(stream))
    _check(rc)
    return out, lse


def _as_codes(name, t):
    """e4m3 codes: a uint8 tensor, or a float8_e4m3fn tensor viewed as its bytes."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    _check_tensor(name, t, torch.uint8, 4)
    return t


def attn_decode_fp8(q: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, stream=None, decode_ctas: int = 0):
    """Single-token decode over an e4m3 K/V cache through ``attn_decode_fp8``.
    q: [B, Hq, 1, 128] bf16; k8, v8: [B, Hkv, Skv, 128] e4m3 codes (uint8 or float8_e4m3fn);
    k_scale, v_scale: fp32 [Hkv, 128] (value = code * coefficient). Returns (o, lse)."""
    _check_tensor("q", q, torch.bfloat16, 4)
    k8, v8 = _as_codes("k8", k8), _as_codes("v8", v8)
    _check_tensor("k_scale", k_scale, torch.float32, 2)
    _check_tensor("v_scale", v_scale, torch.float32, 2)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k8.shape
    if Sq != 1 or tuple(v8.shape) != tuple(k8.shape) or Bk != B or Dk != D \
            or tuple(k_scale.shape) != (Hkv, D) or tuple(v_scale.shape) != (Hkv, D):
        raise ValueError("expected q [B,Hq,1,D], k8, v8 [B,Hkv,Skv,D] and scales [Hkv,D]")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_decode_fp8(q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
                                            v_scale.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Skv, D,
                                            float(scale), int(decode_ctas), _stream_handle(stream))
    _check(rc)
    return out, lse


def attn_prefill_fp8(q: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, scale: float | None = None, causal: bool = True,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention of Sq queries over an e4m3 K/V cache through ``attn_prefill_fp8`` (the causal mask
    aligned to the last Sq keys). q: [B, Hq, Sq, 128] bf16; k8, v8: [B, Hkv, Skv, 128] e4m3 codes
    (uint8 or float8_e4m3fn); k_scale, v_scale: fp32 [Hkv, 128]. Returns (o, lse)."""
    _check_tensor("q", q, torch.bfloat16, 4)
    k8, v8 = _as_codes("k8", k8), _as_codes("v8", v8)
    _check_tensor("k_scale", k_scale, torch.float32, 2)
    _check_tensor("v_scale", v_scale, torch.float32, 2)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k8.shape
    if tuple(v8.shape) != tuple(k8.shape) or Bk != B or Dk != D \
            or tuple(k_scale.shape) != (Hkv, D) or tuple(v_scale.shape) != (Hkv, D):
        raise ValueError("expected q [B,Hq,Sq,D], k8, v8 [B,Hkv,Skv,D] and scales [Hkv,D]")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_prefill_fp8(q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
                                             v_scale.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Skv,
                                             D, float(scale), int(bool(causal)), _stream_handle(stream))
    _check(rc)
    return out, lse


def attn_decode_paged_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                          v_scale: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                          scale: float | None = None, out: torch.Tensor | None = None,
                          lse: torch.Tensor | None = None, stream=None, decode_ctas: int = 0):
    """attn_decode_paged over e4m3 pages: k_pages, v_pages [num_pages, Hkv, page_size, 128] e4m3
    codes; k_scale, v_scale fp32 [Hkv, 128]; the rest as :func:`attn_decode_paged`."""
    _check_tensor("q", q, torch.bfloat16, 4)
    k_pages, v_pages = _as_codes("k_pages", k_pages), _as_codes("v_pages", v_pages)
    _check_tensor("k_scale", k_scale, torch.float32, 2)
    _check_tensor("v_scale", v_scale, torch.float32, 2)
    _check_tensor("block_table", block_table, torch.int32, 2)
    _check_tensor("seq_lens", seq_lens, torch.int32, 1)
    B, Hq, Sq, D = q.shape
    num_pages, Hkv, page_size, Dk = k_pages.shape
    if Sq != 1 or tuple(v_pages.shape) != tuple(k_pages.shape) or Dk != D \
            or tuple(k_scale.shape) != (Hkv, D) or tuple(v_scale.shape) != (Hkv, D):
        raise ValueError("expected q [B,Hq,1,D], pages [P,Hkv,page,D] and scales [Hkv,D]")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row / entry per batch element")
    if scale is None:
        scale = D ** -0.5
    out, lse = _made(_side(stream, q.get_device()), (out, torch.empty_like, q), (lse, _lse_of, q))
    _check_tensor("out", out, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    with torch.cuda.device(q.device):
        rc = load_library().attn_decode_paged_fp8(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                                  k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                                  seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv,
                                                  num_pages, page_size, int(block_table.shape[1]), int(max_seq_len),
                                                  float(scale), int(decode_ctas), _stream_handle(stream))
    _check(rc)
    return out, lse


def attn_lse_merge(o_acc: torch.Tensor, lse_acc: torch.Tensor, o_part: torch.Tensor, lse_part: torch.Tensor,
                   out: torch.Tensor | None = None, stream=None):
    """Merge one attention result over a block of keys (o_part bf16 [..., D], lse_part fp32 [...])
    into a running result (o_acc fp32, lse_acc fp32, same shapes; updated in place) through
    ``attn_lse_merge``. ``out`` (bf16, shape of o_part) optionally receives the merged O."""
    _check_tensor("o_part", o_part, torch.bfloat16, o_part.dim())
    _check_tensor("o_acc", o_acc, torch.float32, o_part.dim())
    _check_tensor("lse_part", lse_part, torch.float32, o_part.dim() - 1)
    _check_tensor("lse_acc", lse_acc, torch.float32, o_part.dim() - 1)
    if o_acc.shape != o_part.shape or lse_acc.shape != lse_part.shape or tuple(lse_part.shape) != tuple(o_part.shape[:-1]):
        raise ValueError("o_acc, o_part [..., D] and lse_acc, lse_part [...] must agree")
    if out is not None:
        _check_tensor("out", out, torch.bfloat16, o_part.dim())
        if out.shape != o_part.shape:
            raise ValueError("out must have the shape of o_part")
    D = int(o_part.shape[-1])
    rows = o_part.numel() // D if D else 0
    with torch.cuda.device(o_part.device):
        rc = load_library().attn_lse_merge(o_acc.data_ptr(), lse_acc.data_ptr(), o_part.data_ptr(), lse_part.data_ptr(),
                                           out.data_ptr() if out is not None else None, rows, D,
                                           _stream_handle(stream))
    _check(rc)
    return o_acc, lse_acc


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
             dout: torch.Tensor, scale: float | None = None, causal: bool = True, dq: torch.Tensor | None = None,
             dk: torch.Tensor | None = None, dv: torch.Tensor | None = None, stream=None):
    """Backward pass through ``attn_bwd``: gradients for q, k, v given dout = dL/do, the forward's
    inputs and its outputs o and lse. Head dim 128. Returns (dq, dk, dv), bf16."""
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_tensor(name, t, torch.bfloat16, 4)
    _check_tensor("lse", lse, torch.float32, 3)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or Dk != D or tuple(o.shape) != tuple(q.shape) \
            or tuple(dout.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Sq):
        raise ValueError("shapes of q, k, v, o, lse, dout disagree")
    if scale is None:
        scale = D ** -0.5
    dq, dk, dv = _made(_side(stream, q.get_device()), (dq, torch.empty_like, q), (dk, torch.empty_like, k),
                       (dv, torch.empty_like, v))
    with torch.cuda.device(q.device):
        rc = load_library().attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                                     lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Sq, Skv, D,
                                     float(scale), int(bool(causal)), _stream_handle(stream))
    _check(rc)
    return dq, dk, dv


_NORM_ROPE_BWD_BLOCKS = 592  # ATTN_QK_NORM_ROPE_BWD_WORKSPACE(D) holds two rows of D floats for each

# The calls below come once per layer and token, so the host's time counts: each tensor is checked
# with as few torch calls as the checks need, and only a tensor that fails them is looked at again to
# say what is wrong.


@functools.lru_cache(maxsize=1024)
def _stride_array(b: int, h: int, s: int):
    """The {batch, head, row} array the library reads strides from (read only, so calls share it)."""
    return (ctypes.c_longlong * 3)(b, h, s)


def _device_of(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


def _flat(name, t, dtype, ndim, dev):
    """The shape of a contiguous tensor of this type and rank on device `dev`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev >= 0 and t.is_contiguous():
        shape = t.shape
        if len(shape) == ndim:
            return shape
    _check_tensor(name, t, dtype, ndim)
    raise ValueError(f"{name} must live on cuda:{dev}, got {t.device}")


def _rows(name, t, dev, like=None):
    """The shape and the stride array of a bf16 [batch, head, row, dim] view with a contiguous dim on
    device `dev`; with `like`, of that shape."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == dev >= 0:
        strides = t.stride()
        if len(strides) == 4 and strides[3] == 1:
            B, H, S, D = shape = t.shape
            if like is not None and shape != like:
                raise ValueError(f"{name} must have the shape {tuple(like)}, got {tuple(shape)}")
            # An axis of extent 1 gets D: its stride is never used, and the library wants a multiple of 8.
            return shape, _stride_array(strides[0] if B > 1 else D, strides[1] if H > 1 else D, strides[2] if S > 1 else D)
    _check_rows(name, t, torch.bfloat16)
    if t.shape[-1] == 1:
        raise ValueError(f"{name} has a head dim of 1")
    raise ValueError(f"{name} must live on cuda:{dev}, got {t.device}")


def _call(fn, dev, stream, *args):
    """The library call `fn` with device `dev` current and its stream (the current one unless given) last."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_handle(stream)
    if torch.cuda.current_device() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, status_string(rc))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rotation(cos, sin, D, dev):
    """(rot_dim, max_pos) of the angle tables cos, sin [max_pos, rot_dim / 2]; (0, 0) without them."""
    if cos is None and sin is None:
        return 0, 0
    max_pos, half = shape = _flat("cos", cos, torch.float32, 2, dev)
    if _flat("sin", sin, torch.float32, 2, dev) != shape:
        raise ValueError(f"cos {tuple(cos.shape)} and sin {tuple(sin.shape)} must agree")
    if 2 * half > D:
        raise ValueError(f"the tables rotate {2 * half} channels of a head of {D}")
    return 2 * half, max_pos


def _weight(name, w, D, dev):
    if w is None:
        return None
    if _flat(name, w, torch.bfloat16, 1, dev)[0] != D:
        raise ValueError(f"{name} must be [{D}], got {tuple(w.shape)}")
    return w.data_ptr()


def _positions(positions, B, S, dev):
    if positions is None:
        return None
    if _flat("positions", positions, torch.int32, 2, dev) != (B, S):
        raise ValueError(f"positions must be [{B}, {S}], got {tuple(positions.shape)}")
    return positions.data_ptr()


def _new_rows(like):
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _weight_grad_of(weight):
    return torch.empty_like(weight, dtype=torch.float32)


def _bwd_workspace_of(weight):
    return torch.empty(_NORM_ROPE_BWD_BLOCKS * 2 * weight.shape[0], dtype=torch.float32, device=weight.device)


def _prefix_workspace_of(sizes):
    return decode_prefix_workspace(*sizes)


def attn_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, cos: torch.Tensor | None, sin: torch.Tensor | None,
                      q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                      positions: torch.Tensor | None = None, interleaved: bool = False, eps: float = 1e-6,
                      q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm and rotation of queries and keys through ``attn_qk_norm_rope``: each head of each token is
    RMS-normalised with a weight per channel (without weights: not) and its first 2 * cos.shape[1]
    channels are rotated by the token's position.

    q [B, Hq, S, D], k [B, Hkv, S, D] bf16, any view with a contiguous last axis (head slices of a fused
    token-major projection, say); cos, sin fp32 [max_pos, rot_dim / 2], or None for both: no rotation;
    q_weight, k_weight bf16 [D], both or neither; positions int32 [B, S] (default: the row index).
    Returns (q_out, k_out), heads-major contiguous unless given; an output may be its input."""
    dev = _device_of("q", q)
    qshape, qs = _rows("q", q, dev)
    kshape, ks = _rows("k", k, dev)
    B, Hq, S, D = qshape
    Bk, Hkv, Sk, Dk = kshape
    if Bk != B or Sk != S or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    rot_dim, max_pos = _rotation(cos, sin, D, dev)
    qw, kw, pos = _weight("q_weight", q_weight, D, dev), _weight("k_weight", k_weight, D, dev), _positions(positions, B, S, dev)
    if q_out is None or k_out is None:
        q_out, k_out = _made(_side(stream, dev), (q_out, _new_rows, q), (k_out, _new_rows, k))
    _, qos = _rows("q_out", q_out, dev, qshape)
    _, kos = _rows("k_out", k_out, dev, kshape)
    _call(load_library().attn_qk_norm_rope, dev, stream, q.data_ptr(), k.data_ptr(), qw, kw, _ptr(cos), _ptr(sin), pos,
          q_out.data_ptr(), k_out.data_ptr(), B, Hq, Hkv, S, D, qs, ks, qos, kos, rot_dim, max_pos, 1 if interleaved else 0, eps)
    return q_out, k_out


def attn_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, cos: torch.Tensor | None, sin: torch.Tensor | None,
                          dq_out: torch.Tensor, dk_out: torch.Tensor, q_weight: torch.Tensor | None = None,
                          k_weight: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                          interleaved: bool = False, eps: float = 1e-6, dq: torch.Tensor | None = None,
                          dk: torch.Tensor | None = None, stream=None):
    """Gradient of ``attn_qk_norm_rope`` through ``attn_qk_norm_rope_bwd``: dq_out, dk_out are the
    gradients of its outputs (``attn_bwd``'s dq and dk), q, k and the rest its inputs. dq, dk may be
    views (slices of a fused projection's gradient). Returns (dq, dk, dq_weight, dk_weight), the last
    two fp32 [D], or None without weights."""
    dev = _device_of("q", q)
    qshape, qs = _rows("q", q, dev)
    kshape, ks = _rows("k", k, dev)
    B, Hq, S, D = qshape
    Bk, Hkv, Sk, Dk = kshape
    if Bk != B or Sk != S or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    _, dqos = _rows("dq_out", dq_out, dev, qshape)
    _, dkos = _rows("dk_out", dk_out, dev, kshape)
    rot_dim, max_pos = _rotation(cos, sin, D, dev)
    qw, kw, pos = _weight("q_weight", q_weight, D, dev), _weight("k_weight", k_weight, D, dev), _positions(positions, B, S, dev)
    side = _side(stream, dev)
    if dq is None or dk is None:
        dq, dk = _made(side, (dq, _new_rows, q), (dk, _new_rows, k))
    _, dqs = _rows("dq", dq, dev, qshape)
    _, dks = _rows("dk", dk, dev, kshape)
    dwq = dwk = ws = None
    if qw is not None and kw is not None:  # (one alone: the library refuses it)
        dwq, dwk, ws = _made(side, (None, _weight_grad_of, q_weight), (None, _weight_grad_of, k_weight),
                             (None, _bwd_workspace_of, q_weight))
    _call(load_library().attn_qk_norm_rope_bwd, dev, stream, q.data_ptr(), k.data_ptr(), qw, kw, _ptr(cos), _ptr(sin), pos,
          dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk), _ptr(ws), B, Hq, Hkv, S,
          D, qs, ks, dqos, dkos, dqs, dks, rot_dim, max_pos, 1 if interleaved else 0, eps)
    return dq, dk, dwq, dwk


def _append(k, v, cos, sin, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, q, q_out, q_weight, k_weight,
            positions, new_lens, interleaved, eps, stream):
    fp8 = k_scale is not None
    dev = _device_of("k", k)
    shape, ks = _rows("k", k, dev)
    _, vs = _rows("v", v, dev, shape)
    if fp8:
        k_pages, v_pages = _as_codes("k_pages", k_pages), _as_codes("v_pages", v_pages)
    cache = torch.uint8 if fp8 else torch.bfloat16
    B, Hkv, Sq, D = shape
    num_pages, Hp, page_size, Dp = pages = _flat("k_pages", k_pages, cache, 4, dev)
    if _flat("v_pages", v_pages, cache, 4, dev) != pages or Hp != Hkv or D != 128 or Dp != D:
        raise ValueError(f"expected k, v [B,Hkv,Sq,128] and pages [P,Hkv,page,128]; got {tuple(k.shape)}, "
                         f"{tuple(v.shape)}, {tuple(k_pages.shape)}, {tuple(v_pages.shape)}")
    rows, per_seq = _flat("block_table", block_table, torch.int32, 2, dev)
    if rows != B or _flat("seq_lens", seq_lens, torch.int32, 1, dev)[0] != B:
        raise ValueError("block_table and seq_lens need one row / entry per batch element")
    if new_lens is not None and _flat("new_lens", new_lens, torch.int32, 1, dev)[0] != B:
        raise ValueError("new_lens needs one entry per batch element")
    if fp8:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if _flat(name, t, torch.float32, 2, dev) != (Hkv, D):
                raise ValueError(f"{name} must be [{Hkv}, {D}], got {tuple(t.shape)}")
    rot_dim, max_pos = _rotation(cos, sin, D, dev)
    qw, kw, pos = _weight("q_weight", q_weight, D, dev), _weight("k_weight", k_weight, D, dev), _positions(positions, B, Sq, dev)
    Hq, qs, qos = 0, None, None
    if q is not None:
        qshape, qs = _rows("q", q, dev)
        Bq, Hq, S, Dq = qshape
        if Bq != B or S != Sq or Dq != D:
            raise ValueError(f"q must be [{B}, Hq, {Sq}, {D}], got {tuple(q.shape)}")
        if q_out is None:
            q_out, = _made(_side(stream, dev), (None, _new_rows, q))
        _, qos = _rows("q_out", q_out, dev, qshape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    lib = load_library()
    scales = (k_scale.data_ptr(), v_scale.data_ptr()) if fp8 else ()
    _call(lib.attn_append_paged_fp8 if fp8 else lib.attn_append_paged, dev, stream, _ptr(q), k.data_ptr(), v.data_ptr(), qw,
          kw, _ptr(cos), _ptr(sin), pos, seq_lens.data_ptr(), _ptr(new_lens), block_table.data_ptr(), _ptr(q_out),
          k_pages.data_ptr(), v_pages.data_ptr(), *scales, B, Hq, Hkv, Sq, qs, ks, vs, qos, num_pages, page_size, per_seq,
          rot_dim, max_pos, 1 if interleaved else 0, eps)
    return q_out


def attn_append_paged(k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor | None, sin: torch.Tensor | None,
                      k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                      q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                      positions: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                      interleaved: bool = False, eps: float = 1e-6, stream=None):
    """Append new tokens to a paged cache through ``attn_append_paged``, keys normalised and rotated on
    the way, and the queries too when given.

    k, v [B, Hkv, Sq, 128] and q [B, Hq, Sq, 128] bf16, any view with a contiguous last axis; k_pages,
    v_pages [num_pages, Hkv, page_size, 128] bf16, updated in place; block_table int32 [B,
    pages_per_seq]; seq_lens int32 [B], counting the new tokens (what ``attn_decode_paged`` or
    ``attn_prefill_paged`` takes next); new_lens int32 [B]: only the last new_lens[b] of the Sq rows are
    tokens. The weights, tables and positions (default: the token's place in its sequence) as
    ``attn_qk_norm_rope``. Returns q_out (None without q)."""
    return _append(k, v, cos, sin, k_pages, v_pages, None, None, block_table, seq_lens, q, q_out, q_weight, k_weight,
                   positions, new_lens, interleaved, eps, stream)


def attn_append_paged_fp8(k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor | None, sin: torch.Tensor | None,
                          k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                          block_table: torch.Tensor, seq_lens: torch.Tensor, q: torch.Tensor | None = None,
                          q_out: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                          k_weight: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                          new_lens: torch.Tensor | None = None, interleaved: bool = False, eps: float = 1e-6,
                          stream=None):
    """``attn_append_paged`` to an e4m3 cache: pages hold codes (uint8 or float8_e4m3fn), k_scale, v_scale the cache's fp32
    [Hkv, 128] coefficients; an element x is stored as the code nearest to x / coefficient."""
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    return _append(k, v, cos, sin, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, q, q_out, q_weight,
                   k_weight, positions, new_lens, interleaved, eps, stream)


def decode_prefix_workspace(B: int, Hq: int, Hkv: int, max_prefix_len: int, max_seq_len: int,
                            device="cuda") -> torch.Tensor:
    """A workspace for ``attn_decode_prefix`` calls of these sizes (or smaller ones), to be kept for as
    long as calls, or graphs that captured them, use it. Calls that overlap need one each."""
    device = torch.device(device)
    with torch.cuda.device(device):
        n = load_library().attn_decode_prefix_workspace(B, Hq, Hkv, max_prefix_len, max_seq_len)
        if n < 0:
            _check(int(n))
        return torch.empty((n,), dtype=torch.uint8, device=device)


def attn_decode_prefix(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, prefix_table: torch.Tensor,
                       prefix_len: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                       max_prefix_len: int, max_seq_len: int, scale: float | None = None,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """Single-token decode of a batch that shares a prefix through ``attn_decode_prefix``: every sequence
    attends to the prefix's keys (read once for the batch) and to its own.

    q [B, Hq, 1, 128] bf16; k_pages, v_pages [num_pages, Hkv, page_size, 128] bf16; prefix_table int32
    [prefix_pages] and prefix_len int32 [1]; block_table int32 [B, pages_per_seq] and seq_lens int32 [B]:
    the keys behind the prefix (all on the GPU); max_prefix_len, max_seq_len: host-side bounds of the
    lengths. ``workspace`` from ``decode_prefix_workspace`` keeps a loop of calls from allocating.
    Returns (o [B, Hq, 1, 128], lse [B, Hq, 1])."""
    dev = _device_of("q", q)
    B, Hq, Sq, D = qshape = _flat("q", q, torch.bfloat16, 4, dev)
    num_pages, Hkv, page_size, Dk = pages = _flat("k_pages", k_pages, torch.bfloat16, 4, dev)
    if Sq != 1 or _flat("v_pages", v_pages, torch.bfloat16, 4, dev) != pages or Dk != D or D != 128:
        raise ValueError(f"expected q [B,Hq,1,128] and k, v pages [P,Hkv,page,128]; got {tuple(q.shape)}, "
                         f"{tuple(k_pages.shape)}, {tuple(v_pages.shape)}")
    prefix_pages, = _flat("prefix_table", prefix_table, torch.int32, 1, dev)
    rows, per_seq = _flat("block_table", block_table, torch.int32, 2, dev)
    if rows != B or _flat("seq_lens", seq_lens, torch.int32, 1, dev)[0] != B \
            or _flat("prefix_len", prefix_len, torch.int32, 1, dev)[0] != 1:
        raise ValueError("block_table and seq_lens need one row / entry per batch element, prefix_len one entry")
    if scale is None:
        scale = D ** -0.5
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _made(_side(stream, dev), (out, torch.empty_like, q), (lse, _lse_of, q),
                                    (workspace, _prefix_workspace_of, (B, Hq, Hkv, max_prefix_len, max_seq_len, q.device)))
    if _flat("out", out, torch.bfloat16, 4, dev) != qshape or _flat("lse", lse, torch.float32, 3, dev) != (B, Hq, 1):
        raise ValueError(f"out must be {tuple(qshape)} and lse {(B, Hq, 1)}")
    ws_bytes, = _flat("workspace", workspace, torch.uint8, 1, dev)
    _call(load_library().attn_decode_prefix, dev, stream, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
          prefix_table.data_ptr(), prefix_len.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
          lse.data_ptr(), workspace.data_ptr(), ws_bytes, B, Hq, Hkv, num_pages, page_size, prefix_pages, max_prefix_len,
          per_seq, max_seq_len, scale)
    return out, lse


def decode_ctas(B: int, Hq: int, Hkv: int, Skv: int, D: int) -> int:
    """Number of CTAs attn_fwd launches for a decode of this shape on the current device."""
    rc = load_library().attn_decode_ctas(B, Hq, Hkv, Skv, D)
    if rc < 0:
        _check(rc)
    return rc


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word: 0 or ATTN_ERR_DEVICE_TIMEOUT."""
    return load_library().attn_device_status(_stream_handle(stream))


def version() -> int:
    return load_library().attn_version()
