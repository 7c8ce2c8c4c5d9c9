"""ctypes binding of librswa.so: argument marshalling only.

Each function takes torch CUDA tensors, checks dtype/device/shape/contiguity,
and passes ``data_ptr()`` values and the CUDA stream handle to the C entry
point of the same name (declared in ``include/rswa.h``). Every step of the
computation runs in the library's kernels; there is no CPU or PyTorch
fallback: if the library is missing, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
import threading
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# RSWA_LIBRARY selects another build of the same library (for example one
# compiled with different pipeline-depth constants); default: the in-tree build.
LIB_PATH = os.environ.get("RSWA_LIBRARY") or os.path.join(_PKG, "librswa.so")
_DEFAULT_LIB = os.path.join(_PKG, "librswa.so")

OP_DECODE = 1
OP_SRSWA_DECODE = 2
OP_ROUTE = 3
OP_PREFILL = 4
OP_SRSWA_ROUTED = 5
OP_DECODE_SCORED = 6

STATUS_NAMES = {0: "RSWA_OK", 1: "RSWA_ERR_INVALID", 2: "RSWA_ERR_UNSUPPORTED", 3: "RSWA_ERR_CUDA",
                5: "RSWA_ERR_DEVICE_CHECK"}
DEVICE_BAD_PREFIX_LEN = 0x1
DEVICE_BAD_RING_STATE = 0x2
DEVICE_BAD_BLOCK_IDX = 0x4
DEVICE_WAIT_TIMEOUT = 0x8
DEVICE_PIPELINE = 0x10
DEVICE_BAD_RANGE = 0x20
DEVICE_BAD_POS = 0x40
DEVICE_BAD_SHARE = 0x80
TEST_SHARED_PART = 0x40000000

EXPORTED = ("rswa_last_error", "rswa_version", "rswa_workspace_bytes", "rswa_check_status", "rswa_append",
            "rswa_decode", "srswa_index_pool", "srswa_route", "srswa_decode", "rswa_decode_noalloc", "rswa_prefill",
            "rswa_quantize_prefix", "rswa_decode_fp8", "srswa_decode_fp8", "srswa_route_tokens", "srswa_prefill",
            "rswa_decode_append", "srswa_decode_append", "rswa_rope_page2d", "rswa_append_rope", "rswa_append_fp8",
            "rswa_decode_fp8kv", "srswa_decode_fp8kv", "rswa_test_arm_wait_timeout", "srswa_decode_routed",
            "srswa_step", "srswa_prefill_workspace_bytes", "rswa_decode_append_rope", "srswa_step_rope", "rswa_rope_1d",
            "rswa_decode_scored", "rswa_prefill_scored", "rswa_decode_shared", "rswa_decode_shared_workspace_bytes")


class RswaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("ring", ctypes.c_int32), ("prefix_cap", ctypes.c_int64)]

    def __repr__(self):
        return (f"Dims(batch={self.batch}, heads={self.heads}, head_dim={self.head_dim}, ring={self.ring}, "
                f"prefix_cap={self.prefix_cap})")


class Rope(ctypes.Structure):
    """rswa_rope: the page2d encoding of a fused decode step (device position arrays)."""
    _fields_ = [("tok_pos", ctypes.c_void_p), ("page", ctypes.c_void_p), ("base", ctypes.c_double),
                ("page_mod", ctypes.c_int32)]


class Score(ctypes.Structure):
    """rswa_score: the cap, distance bias and document ranges of scored attention (device arrays)."""
    _fields_ = [("softcap", ctypes.c_float), ("slope", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("range", ctypes.c_void_p)]


class Rope1d(ctypes.Structure):
    """rswa_rope1d: shapes and strides of a one-position rotary encoding."""
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads_q", "heads_k", "tokens", "head_dim", "rot_dim", "layout",
                                              "dtype", "inverse")] + \
        [("mscale", ctypes.c_float)] + \
        [(n, ctypes.c_int64 * 3) for n in ("q_stride", "q_out_stride", "k_stride", "k_out_stride")]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load librswa.so (building it first if the sources are newer). Raises if unavailable."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if path is None and p == _DEFAULT_LIB:
            from . import build as _build
            try:
                if not _build.up_to_date():
                    _build.build_lib()
            except RuntimeError:
                if not os.path.exists(p):
                    raise
        if not os.path.exists(p):
            raise RuntimeError(f"librswa.so not found at {p}; run python -m long_context_decode_swa_b200.build")
        lib = ctypes.CDLL(p)
        P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        DP = ctypes.POINTER(Dims)
        RP = ctypes.POINTER(Rope)
        sig = {
            "rswa_last_error": ([], ctypes.c_char_p),
            "rswa_version": ([], I32),
            "rswa_workspace_bytes": ([DP, I32], SZ),
            "rswa_check_status": ([P, SZ, P, P], ctypes.c_int),
            "rswa_test_arm_wait_timeout": ([I32, I64], ctypes.c_int),
            "srswa_decode_routed": ([DP, P, P, P, F32, I32, P, P, P, P, P, P, P, F32, P, P, P, P, P, P, SZ, P],
                                    ctypes.c_int),
            "srswa_step": ([DP, P, P, P, P, P, F32, I32, P, P, P, P, P, P, P, P, F32, P, P, P, P, P, P, SZ, P],
                           ctypes.c_int),
            "srswa_prefill_workspace_bytes": ([DP, I32], SZ),
            "rswa_decode_append_rope": ([DP, RP, P, P, P, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_step_rope": ([DP, RP, P, P, P, P, P, F32, I32, P, P, P, P, P, P, P, P, F32, P, P, P, P, P, P, SZ,
                                 P], ctypes.c_int),
            "rswa_append": ([DP, P, P, P, P, P, P, P, P, P], ctypes.c_int),
            "rswa_decode": ([DP, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_index_pool": ([DP, P, P, P, P], ctypes.c_int),
            "srswa_route": ([DP, P, P, P, F32, I32, P, P, P, P, P, SZ, P], ctypes.c_int),
            "srswa_decode": ([DP, P, P, P, P, P, P, I32, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "rswa_decode_noalloc": ([DP, P, P, P, P, P, P, P, P, F32, P, P, P, P], ctypes.c_int),
            "rswa_prefill": ([DP, I32, P, P, P, P, P, P, P, P, P, P, F32, P, P, I32, P, SZ, P], ctypes.c_int),
            "rswa_quantize_prefix": ([DP, P, P, P, P, P, P, P, P, P], ctypes.c_int),
            "rswa_decode_fp8": ([DP, P, P, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_decode_fp8": ([DP, P, P, P, P, P, P, P, P, I32, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_route_tokens": ([DP, I32, P, P, P, F32, I32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_prefill": ([DP, I32, P, P, P, P, P, P, P, P, I32, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "rswa_decode_append": ([DP, P, P, P, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_decode_append": ([DP, P, P, P, P, P, P, P, P, I32, P, P, P, P, P, F32, P, P, P, SZ, P],
                                    ctypes.c_int),
            "rswa_rope_page2d": ([I64, I32, I32, P, P, P, P, P, P, ctypes.c_double, I32, P], ctypes.c_int),
            "rswa_append_rope": ([DP, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_double, I32, P, P], ctypes.c_int),
            "rswa_append_fp8": ([DP, P, P, P, P, P, P, P, P, P, P, P], ctypes.c_int),
            "rswa_decode_fp8kv": ([DP, P, P, P, P, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P], ctypes.c_int),
            "srswa_decode_fp8kv": ([DP, P, P, P, P, P, P, P, P, I32, P, P, P, P, P, P, F32, P, P, P, SZ, P],
                                   ctypes.c_int),
        }
        sig["rswa_rope_1d"] = ([ctypes.POINTER(Rope1d), P, P, P, P, P, P, P], ctypes.c_int)
        sig["rswa_decode_scored"] = ([DP, ctypes.POINTER(Score), P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P],
                                     ctypes.c_int)
        sig["rswa_prefill_scored"] = ([DP, ctypes.POINTER(Score), I32, P, P, P, P, P, P, P, P, P, P, F32, P, P, I32, P,
                                       SZ, P], ctypes.c_int)
        sig["rswa_decode_shared_workspace_bytes"] = ([DP, I32], SZ)
        sig["rswa_decode_shared"] = ([DP, I32, I64, P, P, P, P, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P],
                                     ctypes.c_int)
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _check(fn: str, code: int):
    if code != 0:
        raise RswaError(fn, code, load().rswa_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _want(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


_native = None


def _extension(path: str):
    """The extension module `_tensors` in the file `path`."""
    spec = importlib.util.spec_from_file_location(f"{__package__}._tensors", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _tensors():
    """The tensor checks of the newer calls: addresses(index, spec, ..) gives the data pointers of the specs'
    tensors, each (tensor, name, dtype, shape): contiguous, of that dtype and shape, on CUDA device `index`; a
    fifth element lets a tensor be None. strided() gives (pointer, strides) of any layout, and refuses tensors
    that require a gradient while autograd records one. Native
    (csrc/tensors.cpp, built here if it is missing), or in Python (tensors.py) where it cannot be built."""
    global _native
    if _native is None:
        from . import build as _build
        try:
            native = _extension(_build.build_ext())
        except (RuntimeError, ImportError, OSError) as e:
            from . import tensors as native
            _native = native
            warnings.warn(f"the tensor checks run in Python, 5 to 7 us a call more: {e}", RuntimeWarning, stacklevel=3)
        _native = native
    return _native


@functools.lru_cache(maxsize=1024)
def _dims(batch: int, heads: int, head_dim: int, ring: int, prefix_cap: int) -> Dims:
    """A shared Dims of these values (read-only)."""
    return Dims(batch, heads, head_dim, ring, prefix_cap)


def _device_of(t, name: str) -> int:
    """The CUDA device index of a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.get_device()


# The raw handle of a device's current stream, without building a torch.cuda.Stream (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
# The current device without torch.cuda.current_device's check that CUDA is initialised (a CUDA tensor exists here).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_fns: dict = {}


def _call(name: str, index: int, stream, *args):
    """The C call on `stream` (default: the current stream of the tensors' device), with that device current."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(load(), name)
    if stream is None:
        raw = _raw_stream(index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _current_device() == index:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(*args, raw)
    if code != 0:
        _check(name, code)


def dims_of(pk: torch.Tensor, ring_k: torch.Tensor) -> Dims:
    B, H, cap, D = pk.shape
    return Dims(B, H, D, ring_k.shape[2], cap)


def workspace_bytes(dims: Dims, op: int) -> int:
    n = load().rswa_workspace_bytes(ctypes.byref(dims), op)
    if n == 0:
        raise RswaError("rswa_workspace_bytes", 1, load().rswa_last_error().decode())
    return int(n)


def new_workspace(dims: Dims, op: int, device=None) -> torch.Tensor:
    """A zero-filled workspace tensor (uint8) sized for `op` (see rswa_workspace_bytes)."""
    return torch.zeros(workspace_bytes(dims, op), dtype=torch.uint8, device=device or "cuda")


def route_workspace(batch: int, prefix_cap: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for srswa_route over `batch` sequences of capacity `prefix_cap`."""
    return new_workspace(Dims(batch, 1, 128, 1, prefix_cap), OP_ROUTE, device)


def test_arm_wait_timeout(drop_tile: int, wait_limit_ns: int) -> None:
    """Test hook: the next decode-family call of this thread drops CTA 0's tile `drop_tile`
    (its bounded wait then runs out) and waits at most `wait_limit_ns` (see rswa.h)."""
    _check("rswa_test_arm_wait_timeout", load().rswa_test_arm_wait_timeout(int(drop_tile), int(wait_limit_ns)))


def check_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise, read and clear the device status word; returns it (0 = clean)."""
    st = ctypes.c_int32(0)
    code = load().rswa_check_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                    ctypes.byref(st), _stream(stream))
    if code not in (0, 5):
        _check("rswa_check_status", code)
    return int(st.value)


def rswa_append(ring_k, ring_v, k_new, v_new, wp, fill, slot_out=None, status=None, stream=None):
    B, H, n, D = ring_k.shape
    _want(ring_k, "ring_k", torch.bfloat16)
    _want(ring_v, "ring_v", torch.bfloat16, ring_k.shape)
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    if status is not None:
        _want(status, "status", status.dtype)
    dims = Dims(B, H, D, n, 0)
    _check("rswa_append", load().rswa_append(ctypes.byref(dims), _ptr(ring_k), _ptr(ring_v), _ptr(k_new), _ptr(v_new),
                                             _ptr(wp), _ptr(fill), _ptr(slot_out), _ptr(status), _stream(stream)))


def rswa_rope_page2d(q, tok_pos, page, q_out=None, k=None, k_out=None, base: float = 10000.0, page_mod: int = 2,
                     stream=None):
    """page2d rotary encoding of q (and k) bf16 [..., H, D], one token per leading index with
    positions tok_pos / page (int32, shaped like the leading dims). q_out / k_out default to
    in place. Returns (q_out, k_out)."""
    if q.dim() < 2:
        raise ValueError("q: expected [..., H, D]")
    H, D = q.shape[-2:]
    lead = tuple(q.shape[:-2])
    _want(q, "q", torch.bfloat16)
    q_out = q if q_out is None else _want(q_out, "q_out", torch.bfloat16, q.shape)
    if k is not None:
        _want(k, "k", torch.bfloat16, q.shape)
        k_out = k if k_out is None else _want(k_out, "k_out", torch.bfloat16, q.shape)
    elif k_out is not None:
        raise ValueError("k_out given without k")
    _want(tok_pos, "tok_pos", torch.int32, lead)
    _want(page, "page", torch.int32, lead)
    rows = q.numel() // (H * D) if q.numel() else 0
    _check("rswa_rope_page2d", load().rswa_rope_page2d(rows, H, D, _ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out),
                                                       _ptr(tok_pos), _ptr(page), float(base), int(page_mod),
                                                       _stream(stream)))
    return q_out, k_out


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


@functools.lru_cache(maxsize=256)
def _rope_desc(dtype, layout, mscale, inverse, pairs, shape, heads_k, *strides):
    """The descriptor of a call's shapes and strides (read-only)."""
    if layout not in _ROPE_LAYOUTS:
        raise ValueError(f"layout: expected 'half' or 'interleaved', got {layout!r}")
    d = Rope1d(shape[0], shape[1], heads_k, shape[2] if len(shape) == 4 else 1, shape[-1], 2 * pairs,
               _ROPE_LAYOUTS[layout], _ROPE_DTYPES[dtype], 1 if inverse else 0, mscale)
    for st, name in zip(strides, ("q", "q_out", "k", "k_out")):
        if st[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{name}: the last axis must be dense")
        getattr(d, name + "_stride")[:] = (st[0], st[1], st[2] if len(st) == 4 else 0)
    return d


def _same_rows(shape, a, b) -> bool:
    """Whether strides a and b lay the rows of `shape` out alike (an axis of one entry has no say)."""
    return 0 in shape or all(n == 1 or x == y for n, x, y in zip(shape, a, b))


def rswa_rope_1d(q, pos, inv_freq, q_out=None, k=None, k_out=None, layout: str = "half", mscale: float = 1.0,
                 inverse: bool = False, stream=None):
    """Rotary encoding of q (and k), bf16 or f32 [B][H][T][D] at int32 positions pos [B][T], or [B][H][D]
    with pos [B] (one token per sequence). q and k may differ in their number of heads, and every
    tensor may be a strided view with a dense last axis. inv_freq: f64 pair frequencies on the host
    (a CPU tensor; see rope_freqs); its length is half the rotated dims, the rest of a head passes
    through. layout: "half" or "interleaved" pairs. inverse=True applies the transpose, which turns
    gradients back. Outputs default to in place. Returns (q_out, k_out). The call records nothing for autograd and
    refuses tensors that require a gradient while one is recorded: call it from an autograd.Function (forward, and
    with inverse=True backward) or under torch.no_grad()."""
    dev = _device_of(q, "q")
    shape, dtype = tuple(q.shape), q.dtype
    if len(shape) not in (3, 4):
        raise ValueError("q: expected [B, H, T, D] or [B, H, D]")
    if dtype not in _ROPE_DTYPES:
        raise TypeError(f"q: expected torch.bfloat16 or torch.float32, got {dtype}")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.is_cuda or inv_freq.dtype is not torch.float64 or \
            inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq: expected a contiguous 1-D float64 tensor on the CPU")
    if q_out is None:
        q_out = q
    native = _tensors()
    pos_p, = native.addresses(dev, (pos, "pos", torch.int32, shape[:1] if len(shape) == 3 else (shape[0], shape[2])))
    if k is None:
        if k_out is not None:
            raise ValueError("k_out given without k")
        (qp, qs), (qop, qos) = native.strided(dev, (q, "q", dtype, shape), (q_out, "q_out", dtype, shape))
        d = _rope_desc(dtype, layout, mscale, inverse, inv_freq.shape[0], shape, 0, qs, qos)
        kp = kop = None
    else:
        if not isinstance(k, torch.Tensor) or k.dim() != len(shape) or k.shape[1] == 0:
            raise ValueError("k: expected a tensor shaped like q but for its heads (one at least)")
        if k_out is None:
            k_out = k
        kshape = (shape[0], k.shape[1]) + shape[2:]
        (qp, qs), (qop, qos), (kp, ks), (kop, kos) = native.strided(
            dev, (q, "q", dtype, shape), (q_out, "q_out", dtype, shape), (k, "k", dtype, kshape),
            (k_out, "k_out", dtype, kshape))
        if kp == kop and ks != kos and not _same_rows(kshape, ks, kos):
            raise ValueError("k_out: in place needs the input's strides")
        d = _rope_desc(dtype, layout, mscale, inverse, inv_freq.shape[0], shape, kshape[1], qs, qos, ks, kos)
    if qp == qop and qs != qos and not _same_rows(shape, qs, qos):
        raise ValueError("q_out: in place needs the input's strides")
    _call("rswa_rope_1d", dev, stream, d, inv_freq.data_ptr(), pos_p, qp, qop, kp, kop)
    return q_out, k_out


def rswa_append_rope(ring_k, ring_v, k_new, v_new, wp, fill, q, tok_pos, page, q_out=None, base: float = 10000.0,
                     page_mod: int = 2, slot_out=None, status=None, stream=None):
    """rswa_append with k_new page2d-encoded on its way into the ring and q encoded into q_out
    (default: in place), one launch. Returns q_out."""
    B, H, n, D = ring_k.shape
    _want(ring_k, "ring_k", torch.bfloat16)
    _want(ring_v, "ring_v", torch.bfloat16, ring_k.shape)
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(q, "q", torch.bfloat16, (B, H, D))
    q_out = q if q_out is None else _want(q_out, "q_out", torch.bfloat16, (B, H, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(tok_pos, "tok_pos", torch.int32, (B,))
    _want(page, "page", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    if status is not None:
        _want(status, "status", status.dtype)
    dims = Dims(B, H, D, n, 0)
    _check("rswa_append_rope", load().rswa_append_rope(ctypes.byref(dims), _ptr(ring_k), _ptr(ring_v), _ptr(k_new),
                                                       _ptr(v_new), _ptr(wp), _ptr(fill), _ptr(slot_out), _ptr(q),
                                                       _ptr(q_out), _ptr(tok_pos), _ptr(page), float(base),
                                                       int(page_mod), _ptr(status), _stream(stream)))
    return q_out


def rswa_decode(q, pk, pv, prefix_len, ring_k, ring_v, wp, fill, out, workspace, lse=None, scale=None, stream=None):
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_decode", load().rswa_decode(ctypes.byref(dims), _ptr(q), _ptr(pk), _ptr(pv), _ptr(prefix_len),
                                             _ptr(ring_k), _ptr(ring_v), _ptr(wp), _ptr(fill), scale, _ptr(out),
                                             _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))


def srswa_index_pool(k_idx, prefix_len, kbar, heads: int = 1, stream=None):
    B, cap, DI = k_idx.shape
    _want(k_idx, "k_idx", torch.bfloat16)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(kbar, "kbar", torch.float32, (B, (cap + 31) // 32, DI))
    if DI != 32:
        raise ValueError("index dim must be 32")
    dims = Dims(B, heads, 128, 1, cap)
    _check("srswa_index_pool", load().srswa_index_pool(ctypes.byref(dims), _ptr(k_idx), _ptr(prefix_len), _ptr(kbar),
                                                       _stream(stream)))


def srswa_route(q_idx, kbar, prefix_len, blk_idx, blk_logp, workspace, probs=None, tau=None, idx_scale=1.0,
                prefix_cap: int | None = None, stream=None):
    B, nb_cap, DI = kbar.shape
    topk = blk_idx.shape[1]
    _want(q_idx, "q_idx", torch.float32, (B, DI))
    _want(kbar, "kbar", torch.float32)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    if probs is not None:
        _want(probs, "probs", torch.float32, (B, nb_cap))
    if tau is not None:
        _want(tau, "tau", torch.float32, (B,))
    _want(workspace, "workspace", torch.uint8)
    cap = nb_cap * 32 if prefix_cap is None else int(prefix_cap)
    if (cap + 31) // 32 != nb_cap:
        raise ValueError("prefix_cap does not match kbar's block count")
    dims = Dims(B, 1, 128, 1, cap)
    _check("srswa_route", load().srswa_route(ctypes.byref(dims), _ptr(q_idx), _ptr(kbar), _ptr(prefix_len),
                                             float(idx_scale), topk, _ptr(blk_idx), _ptr(blk_logp), _ptr(probs),
                                             _ptr(tau), _ptr(workspace), workspace.numel(), _stream(stream)))


def srswa_decode(q, pk, pv, prefix_len, blk_idx, blk_logp, ring_k, ring_v, wp, fill, out, workspace, lse=None,
                 scale=None, stream=None):
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    topk = blk_idx.shape[1]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_decode", load().srswa_decode(ctypes.byref(dims), _ptr(q), _ptr(pk), _ptr(pv), _ptr(prefix_len),
                                               _ptr(blk_idx), _ptr(blk_logp), topk, _ptr(ring_k), _ptr(ring_v),
                                               _ptr(wp), _ptr(fill), scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                               workspace.numel(), _stream(stream)))


def fp8_prefix_buffers(pk: torch.Tensor):
    """Empty E4M3 code tensors (uint8, pk's shape) and f32 block-scale tensors [B][H][ceil(cap/32)] for K and V."""
    B, H, cap, D = pk.shape
    nb = (cap + 31) // 32
    dev = pk.device
    return (torch.empty((B, H, cap, D), dtype=torch.uint8, device=dev),
            torch.empty((B, H, cap, D), dtype=torch.uint8, device=dev),
            torch.zeros((B, H, nb), dtype=torch.float32, device=dev),
            torch.zeros((B, H, nb), dtype=torch.float32, device=dev))


def rswa_quantize_prefix(pk, pv, prefix_len, pk8, pv8, k_scale, v_scale, status=None, stream=None):
    B, H, cap, D = pk.shape
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(pk8, "pk8", torch.uint8, pk.shape)
    _want(pv8, "pv8", torch.uint8, pk.shape)
    nb = (cap + 31) // 32
    _want(k_scale, "k_scale", torch.float32, (B, H, nb))
    _want(v_scale, "v_scale", torch.float32, (B, H, nb))
    dims = Dims(B, H, D, 1, cap)
    _check("rswa_quantize_prefix", load().rswa_quantize_prefix(ctypes.byref(dims), _ptr(pk), _ptr(pv),
                                                               _ptr(prefix_len), _ptr(pk8), _ptr(pv8),
                                                               _ptr(k_scale), _ptr(v_scale), _ptr(status),
                                                               _stream(stream)))


def _want_fp8_prefix(pk8, pv8, k_scale, v_scale):
    B, H, cap, D = pk8.shape
    _want(pk8, "pk8", torch.uint8)
    _want(pv8, "pv8", torch.uint8, pk8.shape)
    _want(k_scale, "k_scale", torch.float32, (B, H, (cap + 31) // 32))
    _want(v_scale, "v_scale", torch.float32, (B, H, (cap + 31) // 32))
    return B, H, cap, D


def rswa_decode_fp8(q, pk8, pv8, k_scale, v_scale, prefix_len, ring_k, ring_v, wp, fill, out, workspace, lse=None,
                    scale=None, stream=None):
    B, H, cap, D = _want_fp8_prefix(pk8, pv8, k_scale, v_scale)
    n = ring_k.shape[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_decode_fp8", load().rswa_decode_fp8(ctypes.byref(dims), _ptr(q), _ptr(pk8), _ptr(pv8),
                                                     _ptr(k_scale), _ptr(v_scale), _ptr(prefix_len), _ptr(ring_k),
                                                     _ptr(ring_v), _ptr(wp), _ptr(fill), scale, _ptr(out),
                                                     _ptr(lse), _ptr(workspace), workspace.numel(),
                                                     _stream(stream)))


def fp8_ring_buffers(ring_shape, device=None):
    """An FP8 ring: E4M3 code tensors (uint8) [B][H][n][D] and f32 row-scale tensors [B][H][n] for K and V."""
    B, H, n, D = ring_shape
    dev = device or "cuda"
    return (torch.zeros((B, H, n, D), dtype=torch.uint8, device=dev),
            torch.zeros((B, H, n, D), dtype=torch.uint8, device=dev),
            torch.ones((B, H, n), dtype=torch.float32, device=dev),
            torch.ones((B, H, n), dtype=torch.float32, device=dev))


def _want_fp8_ring(ring_k8, ring_v8, ring_kscale, ring_vscale):
    B, H, n, D = ring_k8.shape
    _want(ring_k8, "ring_k8", torch.uint8)
    _want(ring_v8, "ring_v8", torch.uint8, (B, H, n, D))
    _want(ring_kscale, "ring_kscale", torch.float32, (B, H, n))
    _want(ring_vscale, "ring_vscale", torch.float32, (B, H, n))
    return B, H, n, D


def rswa_append_fp8(ring_k8, ring_v8, ring_kscale, ring_vscale, k_new, v_new, wp, fill, slot_out=None, status=None,
                    stream=None):
    """rswa_append into an FP8 ring (each written row quantised with its own scale)."""
    B, H, n, D = _want_fp8_ring(ring_k8, ring_v8, ring_kscale, ring_vscale)
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    if status is not None:
        _want(status, "status", status.dtype)
    dims = Dims(B, H, D, n, 0)
    _check("rswa_append_fp8", load().rswa_append_fp8(ctypes.byref(dims), _ptr(ring_k8), _ptr(ring_v8),
                                                     _ptr(ring_kscale), _ptr(ring_vscale), _ptr(k_new), _ptr(v_new),
                                                     _ptr(wp), _ptr(fill), _ptr(slot_out), _ptr(status),
                                                     _stream(stream)))


def rswa_decode_fp8kv(q, pk8, pv8, k_scale, v_scale, prefix_len, ring_k8, ring_v8, ring_kscale, ring_vscale, wp, fill,
                      out, workspace, lse=None, scale=None, stream=None):
    """rswa_decode_fp8 with the ring read as E4M3 codes and row scales."""
    B, H, cap, D = _want_fp8_prefix(pk8, pv8, k_scale, v_scale)
    n = _want_fp8_ring(ring_k8, ring_v8, ring_kscale, ring_vscale)[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_decode_fp8kv", load().rswa_decode_fp8kv(ctypes.byref(dims), _ptr(q), _ptr(pk8), _ptr(pv8),
                                                         _ptr(k_scale), _ptr(v_scale), _ptr(prefix_len),
                                                         _ptr(ring_k8), _ptr(ring_v8), _ptr(ring_kscale),
                                                         _ptr(ring_vscale), _ptr(wp), _ptr(fill), scale, _ptr(out),
                                                         _ptr(lse), _ptr(workspace), workspace.numel(),
                                                         _stream(stream)))


def srswa_decode_fp8kv(q, pk8, pv8, k_scale, v_scale, prefix_len, blk_idx, blk_logp, ring_k8, ring_v8, ring_kscale,
                       ring_vscale, wp, fill, out, workspace, lse=None, scale=None, stream=None):
    """srswa_decode_fp8 with the ring read as E4M3 codes and row scales."""
    B, H, cap, D = _want_fp8_prefix(pk8, pv8, k_scale, v_scale)
    n = _want_fp8_ring(ring_k8, ring_v8, ring_kscale, ring_vscale)[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32)
    topk = blk_idx.shape[1]
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_decode_fp8kv", load().srswa_decode_fp8kv(ctypes.byref(dims), _ptr(q), _ptr(pk8), _ptr(pv8),
                                                           _ptr(k_scale), _ptr(v_scale), _ptr(prefix_len),
                                                           _ptr(blk_idx), _ptr(blk_logp), topk, _ptr(ring_k8),
                                                           _ptr(ring_v8), _ptr(ring_kscale), _ptr(ring_vscale),
                                                           _ptr(wp), _ptr(fill), scale, _ptr(out), _ptr(lse),
                                                           _ptr(workspace), workspace.numel(), _stream(stream)))


def srswa_decode_fp8(q, pk8, pv8, k_scale, v_scale, prefix_len, blk_idx, blk_logp, ring_k, ring_v, wp, fill, out,
                     workspace, lse=None, scale=None, stream=None):
    B, H, cap, D = _want_fp8_prefix(pk8, pv8, k_scale, v_scale)
    n = ring_k.shape[2]
    topk = blk_idx.shape[1]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_decode_fp8", load().srswa_decode_fp8(ctypes.byref(dims), _ptr(q), _ptr(pk8), _ptr(pv8),
                                                       _ptr(k_scale), _ptr(v_scale), _ptr(prefix_len),
                                                       _ptr(blk_idx), _ptr(blk_logp), topk, _ptr(ring_k),
                                                       _ptr(ring_v), _ptr(wp), _ptr(fill), scale, _ptr(out),
                                                       _ptr(lse), _ptr(workspace), workspace.numel(),
                                                       _stream(stream)))


def rswa_decode_append(q, k_new, v_new, pk, pv, prefix_len, ring_k, ring_v, wp, fill, out, workspace, lse=None,
                       slot_out=None, scale=None, stream=None):
    """rswa_append + rswa_decode in one launch (same results; wp / fill / ring updated)."""
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_decode_append", load().rswa_decode_append(ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new),
                                                           _ptr(pk), _ptr(pv), _ptr(prefix_len), _ptr(ring_k),
                                                           _ptr(ring_v), _ptr(wp), _ptr(fill), _ptr(slot_out), scale,
                                                           _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                                           _stream(stream)))


def _rope_arg(tok_pos, page, base, page_mod, B: int) -> Rope:
    _want(tok_pos, "tok_pos", torch.int32, (B,))
    _want(page, "page", torch.int32, (B,))
    return Rope(_ptr(tok_pos), _ptr(page), float(base), int(page_mod))


def rswa_decode_append_rope(q, k_new, v_new, pk, pv, prefix_len, ring_k, ring_v, wp, fill, tok_pos, page, out,
                            workspace, lse=None, slot_out=None, base: float = 10000.0, page_mod: int = 2, scale=None,
                            stream=None):
    """rswa_decode_append with q and k_new page2d-encoded inside the same launch (tok_pos, page:
    int32 [B], this step's positions)."""
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    rope = _rope_arg(tok_pos, page, base, page_mod, B)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_decode_append_rope", load().rswa_decode_append_rope(
        ctypes.byref(dims), ctypes.byref(rope), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(pk), _ptr(pv),
        _ptr(prefix_len), _ptr(ring_k), _ptr(ring_v), _ptr(wp), _ptr(fill), _ptr(slot_out), scale, _ptr(out),
        _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))


def srswa_decode_append(q, k_new, v_new, pk, pv, prefix_len, blk_idx, blk_logp, ring_k, ring_v, wp, fill, out,
                        workspace, lse=None, slot_out=None, scale=None, stream=None):
    """rswa_append + srswa_decode in one launch (same results; wp / fill / ring updated)."""
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    topk = blk_idx.shape[1]
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_decode_append", load().srswa_decode_append(ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new),
                                                             _ptr(pk), _ptr(pv), _ptr(prefix_len), _ptr(blk_idx),
                                                             _ptr(blk_logp), topk, _ptr(ring_k), _ptr(ring_v),
                                                             _ptr(wp), _ptr(fill), _ptr(slot_out), scale, _ptr(out),
                                                             _ptr(lse), _ptr(workspace), workspace.numel(),
                                                             _stream(stream)))


def srswa_route_tokens(q_idx, kbar, prefix_len, blk_idx, blk_logp, workspace, idx_scale=1.0, prefix_cap=None,
                       stream=None):
    """Per-token routes of a chunk: q_idx f32 [B][T][32] -> blk_idx int32 / blk_logp f32 [B][T][topk]."""
    B, nb_cap, DI = kbar.shape
    T = q_idx.shape[1]
    topk = blk_idx.shape[2]
    _want(q_idx, "q_idx", torch.float32, (B, T, DI))
    _want(kbar, "kbar", torch.float32)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, T, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, T, topk))
    _want(workspace, "workspace", torch.uint8)
    cap = nb_cap * 32 if prefix_cap is None else int(prefix_cap)
    dims = Dims(B, 1, 128, 1, cap)
    _check("srswa_route_tokens", load().srswa_route_tokens(ctypes.byref(dims), T, _ptr(q_idx), _ptr(kbar),
                                                           _ptr(prefix_len), float(idx_scale), topk, _ptr(blk_idx),
                                                           _ptr(blk_logp), _ptr(workspace), workspace.numel(),
                                                           _stream(stream)))


def srswa_prefill_workspace(batch: int, heads: int, T: int, prefix_cap: int, ring: int = 128, device=None):
    """A zero-filled workspace for srswa_prefill over `batch` x `heads` chunks of T queries."""
    dims = Dims(batch, heads, 128, ring, prefix_cap)
    n = load().srswa_prefill_workspace_bytes(ctypes.byref(dims), int(T))
    if n == 0:
        raise RswaError("srswa_prefill_workspace_bytes", 1, load().rswa_last_error().decode())
    return torch.zeros(int(n), dtype=torch.uint8, device=device or "cuda")


def srswa_prefill(q, k_out, v_out, pk, pv, prefix_len, blk_idx, blk_logp, out, workspace, lse=None, ring_k=None,
                  ring_v=None, wp=None, fill=None, scale=None, ring: int = 128, stream=None):
    """SR-SWA chunked prefill of T queries per (sequence, head), routes given per token.
    workspace: srswa_prefill_workspace(B, H, T, prefix_cap)."""
    B, H, T, D = q.shape
    cap = pk.shape[2]
    topk = blk_idx.shape[2]
    _want(q, "q", torch.bfloat16, (B, H, T, D))
    _want(k_out, "k_out", torch.bfloat16, (B, H, T, D))
    _want(v_out, "v_out", torch.bfloat16, (B, H, T, D))
    _want(pk, "pk", torch.bfloat16, (B, H, cap, D))
    _want(pv, "pv", torch.bfloat16, (B, H, cap, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, T, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, T, topk))
    _want(out, "out", torch.float32, (B, H, T, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H, T))
    n = ring
    if ring_k is not None:
        n = ring_k.shape[2]
        _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
        _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
        _want(wp, "wp", torch.int32, (B,))
        _want(fill, "fill", torch.int32, (B,))
    _want(workspace, "workspace", torch.uint8)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_prefill", load().srswa_prefill(ctypes.byref(dims), T, _ptr(q), _ptr(k_out), _ptr(v_out), _ptr(pk),
                                                 _ptr(pv), _ptr(prefix_len), _ptr(blk_idx), _ptr(blk_logp), topk,
                                                 _ptr(ring_k), _ptr(ring_v), _ptr(wp), _ptr(fill), scale, _ptr(out),
                                                 _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))


def rswa_prefill(q, k_out, v_out, pk, pv, prefix_len, out, workspace, lse=None, ring_k=None, ring_v=None, wp=None,
                 fill=None, write_ring=False, scale=None, ring: int | None = None, stream=None):
    """Chunked R-SWA prefill. q/k_out/v_out bf16 [B][H][T][D]; out f32 [B][H][T][D]."""
    B, H, T, D = q.shape
    cap = pk.shape[2]
    _want(q, "q", torch.bfloat16)
    _want(k_out, "k_out", torch.bfloat16, q.shape)
    _want(v_out, "v_out", torch.bfloat16, q.shape)
    _want(pk, "pk", torch.bfloat16, (B, H, cap, D))
    _want(pv, "pv", torch.bfloat16, (B, H, cap, D))
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(out, "out", torch.float32, (B, H, T, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H, T))
    _want(workspace, "workspace", torch.uint8)
    if ring_k is not None:
        n = ring_k.shape[2]
        _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
        _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
        _want(wp, "wp", torch.int32, (B,))
        _want(fill, "fill", torch.int32, (B,))
    else:
        if ring is None:
            raise ValueError("without a ring tensor, pass the window length as ring=n")
        n = int(ring)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("rswa_prefill", load().rswa_prefill(ctypes.byref(dims), T, _ptr(q), _ptr(k_out), _ptr(v_out), _ptr(pk),
                                               _ptr(pv), _ptr(prefix_len), _ptr(ring_k), _ptr(ring_v), _ptr(wp),
                                               _ptr(fill), scale, _ptr(out), _ptr(lse), 1 if write_ring else 0,
                                               _ptr(workspace), workspace.numel(), _stream(stream)))


def _want_routed(q, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx, blk_logp, tau, out, lse,
                 workspace):
    B, H, cap, D = pk.shape
    n = ring_k.shape[2]
    topk = blk_idx.shape[1]
    nb_cap = (cap + 31) // 32
    _want(q, "q", torch.bfloat16, (B, H, D))
    _want(q_idx, "q_idx", torch.float32, (B, 32))
    _want(kbar, "kbar", torch.float32, (B, nb_cap, 32))
    _want(pk, "pk", torch.bfloat16)
    _want(pv, "pv", torch.bfloat16, pk.shape)
    _want(prefix_len, "prefix_len", torch.int32, (B,))
    _want(ring_k, "ring_k", torch.bfloat16, (B, H, n, D))
    _want(ring_v, "ring_v", torch.bfloat16, (B, H, n, D))
    _want(wp, "wp", torch.int32, (B,))
    _want(fill, "fill", torch.int32, (B,))
    _want(blk_idx, "blk_idx", torch.int32, (B, topk))
    _want(blk_logp, "blk_logp", torch.float32, (B, topk))
    if tau is not None:
        _want(tau, "tau", torch.float32, (B,))
    _want(out, "out", torch.float32, (B, H, D))
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H))
    _want(workspace, "workspace", torch.uint8)
    return B, H, cap, D, n, topk


def srswa_decode_routed(q, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx, blk_logp, out,
                        workspace, lse=None, tau=None, idx_scale=1.0, scale=None, stream=None):
    """srswa_route + srswa_decode in one launch: the route (blk_idx, blk_logp, tau) is an output.
    workspace: new_workspace(dims, OP_SRSWA_ROUTED)."""
    B, H, cap, D, n, topk = _want_routed(q, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx,
                                         blk_logp, tau, out, lse, workspace)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_decode_routed", load().srswa_decode_routed(
        ctypes.byref(dims), _ptr(q), _ptr(q_idx), _ptr(kbar), float(idx_scale), topk, _ptr(pk), _ptr(pv),
        _ptr(prefix_len), _ptr(ring_k), _ptr(ring_v), _ptr(wp), _ptr(fill), scale, _ptr(blk_idx), _ptr(blk_logp),
        _ptr(tau), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))


def srswa_step(q, k_new, v_new, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx, blk_logp, out,
               workspace, lse=None, tau=None, slot_out=None, idx_scale=1.0, scale=None, stream=None):
    """The whole SR-SWA decode step in one launch: rswa_append + srswa_route + srswa_decode.
    workspace: new_workspace(dims, OP_SRSWA_ROUTED)."""
    B, H, cap, D, n, topk = _want_routed(q, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx,
                                         blk_logp, tau, out, lse, workspace)
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_step", load().srswa_step(
        ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_idx), _ptr(kbar), float(idx_scale), topk,
        _ptr(pk), _ptr(pv), _ptr(prefix_len), _ptr(ring_k), _ptr(ring_v), _ptr(wp), _ptr(fill), _ptr(slot_out), scale,
        _ptr(blk_idx), _ptr(blk_logp), _ptr(tau), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream)))


def srswa_step_rope(q, k_new, v_new, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, tok_pos, page,
                    blk_idx, blk_logp, out, workspace, lse=None, tau=None, slot_out=None, base: float = 10000.0,
                    page_mod: int = 2, idx_scale=1.0, scale=None, stream=None):
    """srswa_step with q and k_new page2d-encoded inside the same launch (tok_pos, page: int32 [B],
    this step's positions; the router's q_idx is not encoded). workspace: new_workspace(dims,
    OP_SRSWA_ROUTED)."""
    B, H, cap, D, n, topk = _want_routed(q, q_idx, kbar, pk, pv, prefix_len, ring_k, ring_v, wp, fill, blk_idx,
                                         blk_logp, tau, out, lse, workspace)
    _want(k_new, "k_new", torch.bfloat16, (B, H, D))
    _want(v_new, "v_new", torch.bfloat16, (B, H, D))
    if slot_out is not None:
        _want(slot_out, "slot_out", torch.int32, (B,))
    rope = _rope_arg(tok_pos, page, base, page_mod, B)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dims = Dims(B, H, D, n, cap)
    _check("srswa_step_rope", load().srswa_step_rope(
        ctypes.byref(dims), ctypes.byref(rope), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_idx), _ptr(kbar),
        float(idx_scale), topk, _ptr(pk), _ptr(pv), _ptr(prefix_len), _ptr(ring_k), _ptr(ring_v), _ptr(wp),
        _ptr(fill), _ptr(slot_out), scale, _ptr(blk_idx), _ptr(blk_logp), _ptr(tau), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def _int32(value, name: str) -> int:
    """An integer that fits the C argument (ctypes would cut it)."""
    n = int(value)
    if n != value or not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}: {value} is not an integer of 32 bits")
    return n


def _numel(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    return t.numel()


def _ring_shape(ring_k, B: int, H: int, D: int):
    if not isinstance(ring_k, torch.Tensor) or ring_k.dim() != 4:
        raise ValueError("ring_k: expected a tensor [B, H, n, D]")
    return (B, H, ring_k.shape[2], D)


def rswa_decode_scored(q, pk, pv, prefix_len, ring_k, ring_v, wp, fill, out, workspace, softcap: float = 0.0,
                       slopes=None, pos=None, ranges=None, lse=None, scale=None, stream=None):
    """R-SWA decode whose scores are softcap * tanh(scale q.k / softcap) (softcap > 0) minus
    slopes[h] * (pos - key position), over prefix rows ranges[b] = (lo, hi) and the ring. q bf16
    [B][H][D]; slopes f32 [H] with pos int32 [B]; ranges int32 [B][2]; out f32 [B][H][D], lse f32
    [B][H]. pos is read with slopes only. workspace: new_workspace(dims, OP_DECODE_SCORED)."""
    dev = _device_of(q, "q")
    if q.dim() != 3 or not isinstance(pk, torch.Tensor) or pk.dim() != 4:
        raise ValueError("expected q [B, H, D] and pk [B, H, cap, D]")
    if slopes is None:
        pos = None
    elif pos is None:
        raise ValueError("slopes need pos")
    B, H, D = row = tuple(q.shape)
    prefix = (B, H, pk.shape[2], D)
    ring = _ring_shape(ring_k, B, H, D)
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    ws_bytes = _numel(workspace, "workspace")
    a = _tensors().addresses(dev, (q, "q", bf16, row), (pk, "pk", bf16, prefix), (pv, "pv", bf16, prefix),
                   (prefix_len, "prefix_len", i32, (B,)), (ring_k, "ring_k", bf16, ring), (ring_v, "ring_v", bf16, ring),
                   (wp, "wp", i32, (B,)), (fill, "fill", i32, (B,)), (out, "out", f32, row), (lse, "lse", f32, (B, H), True),
                   (workspace, "workspace", torch.uint8, (ws_bytes,)), (slopes, "slopes", f32, (H,), True),
                   (pos, "pos", i32, (B,), True), (ranges, "ranges", i32, (B, 2), True))
    _call("rswa_decode_scored", dev, stream, _dims(B, H, D, ring[2], prefix[2]), Score(softcap, *a[11:]), *a[:8],
          1.0 / math.sqrt(D) if scale is None else scale, *a[8:11], ws_bytes)


def rswa_prefill_scored(q, k_out, v_out, pk, pv, prefix_len, out, workspace, softcap: float = 0.0, slopes=None,
                        pos=None, ranges=None, lse=None, ring_k=None, ring_v=None, wp=None, fill=None,
                        write_ring=False, scale=None, ring: int | None = None, stream=None):
    """Chunked R-SWA prefill with the scores of rswa_decode_scored. q/k_out/v_out bf16 [B][H][T][D]; slopes
    f32 [H] with pos int32 [B] (the position of the chunk's first query); ranges int32 [B][T][2], each
    query's document in the prefix; out bf16 [B][H][T][D], lse f32 [B][H][T]. Ring arguments as in
    rswa_prefill. workspace: new_workspace(dims, OP_PREFILL)."""
    dev = _device_of(q, "q")
    if q.dim() != 4 or not isinstance(pk, torch.Tensor) or pk.dim() != 4:
        raise ValueError("expected q [B, H, T, D] and pk [B, H, cap, D]")
    if slopes is None:
        pos = None
    elif pos is None:
        raise ValueError("slopes need pos")
    B, H, T, D = rows = tuple(q.shape)
    prefix = (B, H, pk.shape[2], D)
    if ring_k is not None:
        ring_shape = _ring_shape(ring_k, B, H, D)
        n = ring_shape[2]
    else:
        if ring is None:
            raise ValueError("without a ring tensor, pass the window length as ring=n")
        if ring_v is not None or wp is not None or fill is not None:
            raise ValueError("ring_k, ring_v, wp and fill go together")
        n, ring_shape = _int32(ring, "ring"), ()
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    ws_bytes = _numel(workspace, "workspace")
    ring_specs = ((ring_k, "ring_k", bf16, ring_shape), (ring_v, "ring_v", bf16, ring_shape), (wp, "wp", i32, (B,)),
                  (fill, "fill", i32, (B,))) if ring_k is not None else ((None, "", i32, (), True),) * 4
    a = _tensors().addresses(dev, (q, "q", bf16, rows), (k_out, "k_out", bf16, rows), (v_out, "v_out", bf16, rows),
                   (pk, "pk", bf16, prefix), (pv, "pv", bf16, prefix), (prefix_len, "prefix_len", i32, (B,)), *ring_specs,
                   (out, "out", bf16, rows), (lse, "lse", f32, (B, H, T), True),
                   (workspace, "workspace", torch.uint8, (ws_bytes,)), (slopes, "slopes", f32, (H,), True),
                   (pos, "pos", i32, (B,), True), (ranges, "ranges", i32, (B, T, 2), True))
    _call("rswa_prefill_scored", dev, stream, _dims(B, H, D, n, prefix[2]), Score(softcap, *a[13:]), T, *a[:10],
          1.0 / math.sqrt(D) if scale is None else scale, *a[10:12], 1 if write_ring else 0, a[12], ws_bytes)


def shared_workspace_bytes(dims: Dims, n_shared: int) -> int:
    """Workspace bytes of rswa_decode_shared; dims.prefix_cap is the private capacity."""
    n = load().rswa_decode_shared_workspace_bytes(ctypes.byref(dims), _int32(n_shared, "n_shared"))
    if n == 0:
        raise RswaError("rswa_decode_shared_workspace_bytes", 1, load().rswa_last_error().decode())
    return int(n)


def new_shared_workspace(dims: Dims, n_shared: int, device=None) -> torch.Tensor:
    """A zero-filled workspace tensor (uint8) for rswa_decode_shared over n_shared prefixes."""
    return torch.zeros(shared_workspace_bytes(dims, n_shared), dtype=torch.uint8, device=device or "cuda")


def rswa_decode_shared(q, sk, sv, shared_len, share_of, ring_k, ring_v, wp, fill, out, workspace, pk=None, pv=None,
                       prefix_len=None, lse=None, scale=None, stream=None):
    """R-SWA decode of sequences over shared prefixes sk / sv bf16 [P][H][cap][D] (shared_len int32 [P]):
    sequence b reads prefix share_of[b] (int32 [B], -1: none), its private prefix (pk, pv, prefix_len as
    in rswa_decode; optional) and its ring. q bf16 [B][H][D]; out bf16 [B][H][D], lse f32 [B][H].
    workspace: new_shared_workspace(Dims(B, H, D, n, private cap), P)."""
    dev = _device_of(q, "q")
    if q.dim() != 3 or not isinstance(sk, torch.Tensor) or sk.dim() != 4:
        raise ValueError("expected q [B, H, D] and sk [P, H, cap, D]")
    B, H, D = row = tuple(q.shape)
    P, scap = sk.shape[0], sk.shape[2]
    shared = (P, H, scap, D)
    ring = _ring_shape(ring_k, B, H, D)
    bf16, i32 = torch.bfloat16, torch.int32
    if pk is not None:
        if not isinstance(pk, torch.Tensor) or pk.dim() != 4:
            raise ValueError("pk: expected a tensor [B, H, cap, D]")
        prefix = (B, H, pk.shape[2], D)
        private = ((pk, "pk", bf16, prefix), (pv, "pv", bf16, prefix), (prefix_len, "prefix_len", i32, (B,)))
    else:
        if pv is not None or prefix_len is not None:
            raise ValueError("pk, pv and prefix_len go together")
        prefix, private = (B, H, 0, D), ((None, "", i32, (), True),) * 3
    ws_bytes = _numel(workspace, "workspace")
    a = _tensors().addresses(dev, (q, "q", bf16, row), (sk, "sk", bf16, shared), (sv, "sv", bf16, shared),
                   (shared_len, "shared_len", i32, (P,)), (share_of, "share_of", i32, (B,)), *private,
                   (ring_k, "ring_k", bf16, ring), (ring_v, "ring_v", bf16, ring), (wp, "wp", i32, (B,)),
                   (fill, "fill", i32, (B,)), (out, "out", bf16, row), (lse, "lse", torch.float32, (B, H), True),
                   (workspace, "workspace", torch.uint8, (ws_bytes,)))
    _call("rswa_decode_shared", dev, stream, _dims(B, H, D, ring[2], prefix[2]), P, scap, *a[:12],
          1.0 / math.sqrt(D) if scale is None else scale, *a[12:], ws_bytes)
