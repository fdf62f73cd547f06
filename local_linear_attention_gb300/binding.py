"""ctypes binding of liblla.so: the C-ABI entry points under the same names.

Every function here only checks and marshals arguments (device pointers, sizes, the current
torch stream) and calls the library; all arithmetic runs in liblla's CUDA kernels. There is no
fallback: if the library is missing or the tensors are not on a CUDA device the call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "LlaError", "library_path", "lla_forward", "lla_forward_ws", "lla_workspace_size",
    "lla_forward_host", "lla_moments", "lla_stream_status", "lla_status_string", "lla_version",
    "launch_count", "profile_enable", "profile_collect", "EXPORTED_SYMBOLS", "DTYPE_CODES",
    "lla_forward_noalloc", "NOALLOC_SCRATCH_BYTES", "PATH_AUTO", "PATH_CUDA_CORE",
    "PATH_TENSOR_CORE", "PATH_CG", "lla_parallax_forward", "lla_decode", "lla_parallax_decode",
    "FORM_CENTRED", "FORM_PAGE", "FAULT_WITHHOLD_KEYS", "lla_parallax_backward", "Options",
    "PagedCache", "lla_paged_append", "lla_paged_attention", "lla_paged_workspace_size",
    "lla_paged_evict", "lla_paged_tree_attention", "lla_paged_tree_workspace_size",
    "RotarySpec", "ROTARY_HALVES", "ROTARY_INTERLEAVED", "STRETCH_NONE", "STRETCH_POSITIONS", "STRETCH_BASE",
    "STRETCH_WAVELENGTHS", "lla_rotary", "lla_paged_append_rotary", "lla_paged_fork", "lla_paged_free", "lla_paged_grow",
    "lla_paged_copy", "lla_paged_compact",
]

LLA_OK = 0
DTYPE_CODES = {torch.float32: 0, torch.bfloat16: 1}
NUM_STAGES = 5
STAGE_NAMES = ("prep", "weights", "moments", "solve", "readout")

# Every function include/lla.h declares.
EXPORTED_SYMBOLS = (
    "lla_forward", "lla_workspace_size", "lla_forward_ws", "lla_forward_host", "lla_moments",
    "lla_stream_status", "lla_status_string", "lla_version", "lla_launch_count",
    "lla_profile_enable", "lla_profile_collect", "lla_forward_noalloc", "lla_decode",
    "lla_parallax_decode", "lla_parallax_forward", "lla_parallax_backward", "lla_forward_ex",
    "lla_parallax_forward_ex", "lla_decode_ex", "lla_parallax_decode_ex",
    "lla_parallax_backward_ex", "lla_paged_append", "lla_paged_workspace_size",
    "lla_paged_attention", "lla_paged_evict", "lla_paged_tree_workspace_size", "lla_paged_tree_attention",
    "lla_rotary_frequencies", "lla_rotary", "lla_paged_append_rotary", "lla_paged_fork", "lla_paged_free", "lla_paged_grow",
    "lla_paged_copy", "lla_paged_compact",
)

# LLA_NOALLOC_SCRATCH_BYTES in include/lla.h: the fixed scratch of lla_forward_noalloc.
NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None

PATH_AUTO, PATH_CUDA_CORE, PATH_TENSOR_CORE, PATH_CG = 0, 1, 2, 3
FORM_CENTRED, FORM_PAGE = 0, 1
FAULT_WITHHOLD_KEYS = 1
ROTARY_HALVES, ROTARY_INTERLEAVED = 0, 1
STRETCH_NONE, STRETCH_POSITIONS, STRETCH_BASE, STRETCH_WAVELENGTHS = 0, 1, 2, 3


class Options(ctypes.Structure):
    """lla_options: per-call choices of the *_ex entry points (all zero = the defaults)."""
    _fields_ = [("path", ctypes.c_int), ("form", ctypes.c_int), ("cg_max_iters", ctypes.c_int),
                ("cg_rel_tol", ctypes.c_float), ("test_fault", ctypes.c_int),
                ("reserved", ctypes.c_int * 3)]


# lla_paged_cache and lla_paged_query, packed in native alignment: a decode step makes these calls
# once per layer, and struct.pack takes a third of the time of a ctypes.Structure.
_CACHE = struct.Struct("@5P10i")
_QUERY = struct.Struct("@5P3if6i")
_SPEC = struct.Struct("@64df5i")  # lla_rotary_spec
_POINTERS, _INTS = [struct.Struct(f"@{n}P") for n in range(4)], [struct.Struct(f"@{n}i") for n in range(4)]


def _options(path=0, form=0, cg=None, test_fault=0):
    """An Options struct, or None when every choice is the default (the plain entry point)."""
    if not path and not form and cg is None and not test_fault:
        return None
    o = Options()
    o.path, o.form, o.test_fault = int(path), int(form), int(test_fault)
    if cg is not None:
        o.cg_max_iters, o.cg_rel_tol = int(cg[0]), float(cg[1])
    return o


class LlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lla_status_string(status)} (status {status})")


def library_path() -> str:
    return os.environ.get("LLA_LIBRARY",
                          os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblla.so"))


def _load():
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"liblla.so not found at {path}; build it with "
                          "`python -m local_linear_attention_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    dbl = ctypes.c_double
    fp = ctypes.POINTER(ctypes.c_float)
    op = ctypes.POINTER(Options)
    sig = {
        "lla_forward": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, vp]),
        "lla_workspace_size": (sz, [i, i, i, i, i, i]),
        "lla_forward_ws": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, vp, sz, vp]),
        "lla_forward_host": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, vp]),
        "lla_moments": (i, [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]),
        "lla_stream_status": (i, [vp]),
        "lla_status_string": (ctypes.c_char_p, [i]),
        "lla_version": (i, []),
        "lla_launch_count": (ctypes.c_ulonglong, []),
        "lla_profile_enable": (i, [i]),
        "lla_profile_collect": (i, [fp, i, ctypes.POINTER(ctypes.c_int)]),
        "lla_forward_noalloc": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, vp]),
        "lla_parallax_forward": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]),
        "lla_decode": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, vp]),
        "lla_parallax_decode": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]),
        "lla_parallax_backward": (i, [vp] * 9 + [i, i, i, i, i, f, i, vp]),
        "lla_forward_ex": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, op, vp, sz, vp]),
        "lla_parallax_forward_ex": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, op, vp]),
        "lla_decode_ex": (i, [vp, vp, vp, vp, i, i, i, i, i, f, f, i, op, vp]),
        "lla_parallax_decode_ex": (i, [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, op, vp]),
        "lla_parallax_backward_ex": (i, [vp] * 9 + [i, i, i, i, i, f, i, op, vp]),
        "lla_paged_append": (i, [vp, vp, vp, vp, i, vp]),
        "lla_paged_workspace_size": (sz, [vp, vp]),
        "lla_paged_attention": (i, [vp, vp, vp, sz, vp]),
        "lla_paged_evict": (i, [vp, vp, i, i, i, vp, vp]),
        "lla_paged_tree_workspace_size": (sz, [vp, vp]),
        "lla_paged_tree_attention": (i, [vp, vp, vp, vp, sz, vp]),
        "lla_rotary_frequencies": (i, [vp, i, i, dbl, i, dbl, i, dbl, dbl]),
        "lla_rotary": (i, [vp, vp, vp, vp, i, vp, i, i, i, i, i, vp]),
        "lla_paged_append_rotary": (i, [vp] * 8 + [i, vp, vp, i, vp]),
        "lla_paged_fork": (i, [vp, vp, vp, vp, vp]),
        "lla_paged_free": (i, [vp, vp, vp, vp]),
        "lla_paged_grow": (i, [vp, vp, vp, vp, vp, vp]),
        "lla_paged_copy": (i, [vp, vp, vp, i, vp]),
        "lla_paged_compact": (i, [vp, vp, i, vp, i, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def lla_status_string(status: int) -> str:
    return _load().lla_status_string(int(status)).decode()


def lla_version() -> int:
    return _load().lla_version()


def launch_count() -> int:
    return int(_load().lla_launch_count())


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(st: int, where: str):
    if st != LLA_OK:
        raise LlaError(st, where)


def _shapes(q, k, v):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k [B,H,T,d] and v [B,H,T,dv]")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in DTYPE_CODES:
        raise ValueError("q, k, v must share one dtype: float32 or bfloat16")
    B, H, T, d = q.shape
    return B, H, T, d, v.shape[3], DTYPE_CODES[q.dtype]


def _device_inputs(q, k, v):
    for t in (q, k, v):
        if not t.is_cuda:
            raise ValueError("liblla runs on CUDA tensors only")
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    return _shapes(q, k, v)


def _check_out(out, shape, like):
    if (tuple(out.shape) != tuple(shape) or out.dtype != like.dtype or out.device != like.device
            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous tensor of shape {tuple(shape)}, dtype "
                         f"{like.dtype} on {like.device}")


def lla_forward(q, k, v, h: float, lam: float, out=None, stream=None, *, path=0, form=0, cg=None,
                test_fault=0, workspace=None):
    """Causal LLA forward on device tensors; returns `out` ([B,H,T,dv], dtype of the inputs).

    path / form / cg=(max_iters, rel_tol) / test_fault are this call's lla_options (defaults:
    automatic path, centred form); with any of them, or a workspace tensor, the call goes through
    lla_forward_ex, otherwise through lla_forward."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    _check_out(out, (B, H, T, dv), q)
    opts = _options(path, form, cg, test_fault)
    if opts is None and workspace is None:
        st = _load().lla_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H,
                                 T, d, dv, float(h), float(lam), code, _stream_ptr(stream))
        _check(st, "lla_forward")
        return out
    wp, wb = (None, 0) if workspace is None else (
        workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = _load().lla_forward_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, T,
                                d, dv, float(h), float(lam), code,
                                ctypes.byref(opts) if opts is not None else None, wp, wb,
                                _stream_ptr(stream))
    _check(st, "lla_forward_ex")
    return out


def lla_parallax_forward(q, k, v, r, h: float, out=None, stream=None, *, path=0):
    """Causal Parallax forward with probe r ([B,H,T,d], like q); returns `out` ([B,H,T,dv]).
    path=PATH_CUDA_CORE forces the CUDA-core kernel (lla_parallax_forward_ex)."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    if r.shape != q.shape or r.dtype != q.dtype or not r.is_cuda or not r.is_contiguous():
        raise ValueError("r must be a contiguous CUDA tensor shaped and typed like q")
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    _check_out(out, (B, H, T, dv), q)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(), out.data_ptr(), B, H, T, d,
            dv, float(h), code)
    opts = _options(path)
    if opts is None:
        st = _load().lla_parallax_forward(*args, _stream_ptr(stream))
    else:
        st = _load().lla_parallax_forward_ex(*args, ctypes.byref(opts), _stream_ptr(stream))
    _check(st, "lla_parallax_forward")
    return out


def _decode_inputs(q, k, v):
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    if q.dim() != 3 or k.dim() != 4 or v.dim() != 4 or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("decode expects q [B,H,d], k [B,H,L,d], v [B,H,L,dv] of one dtype")
    B, H, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape[:3] != k.shape[:3]:
        raise ValueError("inconsistent decode shapes")
    if q.dtype not in DTYPE_CODES:
        raise ValueError("dtype must be float32 or bfloat16")
    return B, H, k.shape[2], d, v.shape[3], DTYPE_CODES[q.dtype]


def lla_decode(q, k, v, h: float, lam: float, out=None, stream=None, *, path=0):
    """LLA decode: q [B,H,d] against the cache k [B,H,L,d], v [B,H,L,dv]; returns [B,H,dv].
    path=PATH_CUDA_CORE forces the CUDA-core split kernel (lla_decode_ex)."""
    B, H, L, d, dv, code = _decode_inputs(q, k, v)
    if out is None:
        out = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check_out(out, (B, H, dv), q)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, L, d, dv, float(h),
            float(lam), code)
    opts = _options(path)
    if opts is None:
        st = _load().lla_decode(*args, _stream_ptr(stream))
    else:
        st = _load().lla_decode_ex(*args, ctypes.byref(opts), _stream_ptr(stream))
    _check(st, "lla_decode")
    return out


def lla_parallax_decode(q, k, v, r, h: float, out=None, stream=None, *, path=0):
    """Parallax decode with probe r [B,H,d] (like q); returns [B,H,dv]."""
    B, H, L, d, dv, code = _decode_inputs(q, k, v)
    if r.shape != q.shape or r.dtype != q.dtype or not r.is_cuda or not r.is_contiguous():
        raise ValueError("r must be a contiguous CUDA tensor shaped and typed like q")
    if out is None:
        out = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check_out(out, (B, H, dv), q)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(), out.data_ptr(), B, H, L, d,
            dv, float(h), code)
    opts = _options(path)
    if opts is None:
        st = _load().lla_parallax_decode(*args, _stream_ptr(stream))
    else:
        st = _load().lla_parallax_decode_ex(*args, ctypes.byref(opts), _stream_ptr(stream))
    _check(st, "lla_parallax_decode")
    return out


def lla_parallax_backward(q, k, v, r, dout, h: float, stream=None, *, path=0):
    """Gradients (dq, dk, dv, dr) of the causal Parallax forward for the upstream gradient dout
    ([B,H,T,dv], like the forward's output); each is shaped and typed like q, k, v, r."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    for name, x, like in (("r", r, q), ("dout", dout, None)):
        shape = q.shape if like is not None else (B, H, T, dv)
        if tuple(x.shape) != tuple(shape) or x.dtype != q.dtype or not x.is_cuda \
                or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor of shape {tuple(shape)} "
                             f"and dtype {q.dtype}")
    dq, dk, dvv, dr = (torch.empty_like(x) for x in (q, k, v, r))
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), r.data_ptr(), dout.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dvv.data_ptr(), dr.data_ptr(), B, H, T, d, dv, float(h),
            code)
    opts = _options(path)
    if opts is None:
        st = _load().lla_parallax_backward(*args, _stream_ptr(stream))
    else:
        st = _load().lla_parallax_backward_ex(*args, ctypes.byref(opts), _stream_ptr(stream))
    _check(st, "lla_parallax_backward")
    return dq, dk, dvv, dr


def lla_forward_noalloc(q, k, v, h: float, lam: float, out, stream=None):
    """lla_forward for callers that must not allocate device memory: the library's fixed scratch
    array is used, and `out` (a preallocated contiguous [B,H,T,dv] tensor of q's dtype on q's
    device) is required. The call runs with q's device current, so that the scratch array of
    that device is the one used."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    if not (k.device == q.device and v.device == q.device):
        raise ValueError("q, k, v must be on one device")
    _check_out(out, (B, H, T, dv), q)
    with torch.cuda.device(q.device):
        st = _load().lla_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                         B, H, T, d, dv, float(h), float(lam), code,
                                         _stream_ptr(stream))
    _check(st, "lla_forward_noalloc")
    return out


def lla_workspace_size(B, H, T, d, dv, dtype) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_load().lla_workspace_size(B, H, T, d, dv, code))


def lla_forward_ws(q, k, v, h: float, lam: float, workspace, out=None, stream=None):
    """lla_forward with a caller-owned device workspace (a uint8 CUDA tensor)."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=q.dtype, device=q.device)
    _check_out(out, (B, H, T, dv), q)
    st = _load().lla_forward_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, T,
                                d, dv, float(h), float(lam), code, workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(st, "lla_forward_ws")
    return out


def lla_forward_host(q, k, v, h: float, lam: float, out=None, stream=None):
    """End-to-end forward on HOST tensors (copies in, computes, copies out, synchronises)."""
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("lla_forward_host takes contiguous CPU tensors")
    B, H, T, d, dv, code = _shapes(q, k, v)
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=q.dtype, pin_memory=q.is_pinned())
    st = _load().lla_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H,
                                  T, d, dv, float(h), float(lam), code, _stream_ptr(stream))
    _check(st, "lla_forward_host")
    return out


def lla_moments(q, k, v, idx, h: float, stream=None):
    """Debug entry: raw max-shifted moments of the queries at flat indices idx (int64 CUDA)."""
    B, H, T, d, dv, code = _device_inputs(q, k, v)
    idx = idx.to(device=q.device, dtype=torch.int64).contiguous()
    n = idx.numel()
    f = dict(dtype=torch.float32, device=q.device)
    res = {"m": torch.empty(n, **f), "omega": torch.empty(n, **f), "sk": torch.empty(n, d, **f),
           "sv": torch.empty(n, dv, **f), "Skk": torch.empty(n, d, d, **f),
           "Svk": torch.empty(n, dv, d, **f)}
    st = _load().lla_moments(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(), n,
                             *(res[x].data_ptr() for x in ("m", "omega", "sk", "sv", "Skk", "Svk")),
                             B, H, T, d, dv, float(h), code, _stream_ptr(stream))
    _check(st, "lla_moments")
    return res


class RotarySpec:
    """How positions rotate the first `rot` features of a head (lla_rotary_spec): pairs (i, i + rot/2)
    (ROTARY_HALVES) or (2i, 2i + 1) (ROTARY_INTERLEAVED) by pos * freq[i] radians, times scale. freq is
    base^(-2i/rot), stretched for contexts `factor` times longer as lla_rotary_frequencies describes
    (STRETCH_*; `context`, `slow` and `fast` belong to STRETCH_WAVELENGTHS), or given, rot/2 numbers. A spec does not
    change: calls read the packed struct that is made here."""

    __slots__ = ("_packed",)

    def __init__(self, rot, layout=ROTARY_HALVES, base=10000.0, stretch=STRETCH_NONE, factor=1.0, context=0, slow=1.0,
                 fast=32.0, scale=None, freq=None):
        if freq is None:
            buf = ctypes.create_string_buffer(_SPEC.size)
            _check(_load().lla_rotary_frequencies(buf, rot, layout, base, stretch, factor, context, slow, fast),
                   "lla_rotary_frequencies")
            self._packed = buf.raw
            if scale is None:
                return
            freq = self.freq
        freq = tuple(float(x) for x in freq)
        if len(freq) != rot // 2 or len(freq) > 64:
            raise ValueError("freq must have rot/2 numbers, at most 64")
        self._packed = _SPEC.pack(*freq, *[0.0] * (64 - len(freq)), 1.0 if scale is None else scale, rot, layout, 0, 0, 0)

    @property
    def freq(self):
        return _SPEC.unpack(self._packed)[:self.rot // 2]

    @property
    def scale(self):
        return _SPEC.unpack(self._packed)[64]

    @property
    def rot(self):
        return _SPEC.unpack(self._packed)[65]

    @property
    def layout(self):
        return _SPEC.unpack(self._packed)[66]


def lla_rotary(x, spec: RotarySpec, positions=None, backward=False, out=None, stream=None):
    """Rotates x, a tensor [B, H, T, d] or up to three of them that share B, T and d (q, k and the probe of an
    attention, with any numbers of heads), by their positions [B, T] int32 (None: 0 .. T-1); returns the
    same. backward: the gradients with respect to x from those with respect to the result. out may be x."""
    single = isinstance(x, torch.Tensor)
    xs = (x,) if single else tuple(x)
    if not 1 <= len(xs) <= 3:
        raise ValueError("one to three tensors")
    first = xs[0]
    index = first.get_device()
    if index < 0:
        raise ValueError("liblla runs on CUDA tensors only")
    code = DTYPE_CODES.get(first.dtype)
    if code is None:
        raise ValueError("dtype must be float32 or bfloat16")
    if len(first.shape) != 4:
        raise ValueError("expected x [B, H, T, d]")
    B, _, T, d = first.shape
    heads = []
    for t in xs:
        s = t.shape
        if len(s) != 4 or (s[0], s[2], s[3]) != (B, T, d) or t.dtype != first.dtype or t.get_device() != index or \
                not t.is_contiguous():
            raise ValueError("the tensors must be contiguous [B, H, T, d] of one dtype, on one device, alike but for H")
        heads.append(s[1])
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != (B, T) or
                                  positions.get_device() != index or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 [B, T] tensor on the device of x")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif getattr(stream, "device_index", index) != index:
        raise ValueError(f"the stream must be one of {first.device}, where the tensors are")
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if out is not None:
        outs = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(outs) != len(xs) or any(o.shape != t.shape or o.dtype != t.dtype or o.get_device() != index or
                                       not o.is_contiguous() for o, t in zip(outs, xs)):
            raise ValueError("out must be like x")
    elif stream is None:
        outs = [torch.empty_like(t) for t in xs]
    else:  # what the call allocates belongs to its stream
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(raw, device=first.device) if raw else torch.cuda.default_stream(first.device)
        with torch.cuda.stream(stream):
            outs = [torch.empty_like(t) for t in xs]
    n = len(xs)
    args = (spec._packed, _POINTERS[n].pack(*[t.data_ptr() for t in xs]), _POINTERS[n].pack(*[t.data_ptr() for t in outs]),
            _INTS[n].pack(*heads), n, None if positions is None else positions.data_ptr(), B, T, d, 1 if backward else 0,
            code, raw)
    if torch._C._cuda_getDevice() == index:
        st = _load().lla_rotary(*args)
    else:
        with torch.cuda.device(index):
            st = _load().lla_rotary(*args)
    _check(st, "lla_rotary")
    return outs[0] if single else list(outs)


class PagedCache:
    """A paged key/value cache (lla_paged_cache): k_pages [num_pages, kv_heads, page_size, d],
    v_pages [num_pages, kv_heads, page_size, dv], page_table [num_seqs, max_pages] int32, lens
    [num_seqs] int32 and, where attention weights are tracked or evicted by, mass [num_pages,
    kv_heads, page_size] float32; all contiguous, on one CUDA device. The tensors are the caller's:
    the cache keeps references, and whoever writes new lengths or page numbers into them changes
    what later calls see. `page_table` may be a row range of a larger table."""

    __slots__ = ("k_pages", "v_pages", "page_table", "lens", "mass", "num_seqs", "kv_heads", "d", "dv",
                 "dtype", "device", "_packed", "_index")

    def __init__(self, k_pages, v_pages, page_table, lens, mass=None):
        device, dtype, index = k_pages.device, k_pages.dtype, k_pages.get_device()  # -1: not on a CUDA device
        code = DTYPE_CODES.get(dtype)
        try:
            num_pages, kv_heads, page, d = k_pages.shape
            v_heads = v_pages.shape
            dv = v_heads[3]
        except (ValueError, IndexError):
            num_pages = v_heads = None
        if num_pages is None or v_heads != (num_pages, kv_heads, page, dv):
            raise ValueError("expected k_pages [num_pages, kv_heads, page_size, d] and v_pages "
                             "[num_pages, kv_heads, page_size, dv]")
        if code is None or v_pages.dtype != dtype:
            raise ValueError("k_pages and v_pages must share one dtype: float32 or bfloat16")
        t_shape = page_table.shape
        if len(t_shape) != 2 or page_table.dtype != torch.int32:
            raise ValueError("page_table must be int32 [num_seqs, max_pages]")
        num_seqs, max_pages = t_shape
        if lens.dtype != torch.int32 or lens.shape != (num_seqs,):
            raise ValueError("lens must be int32 [num_seqs]")
        if mass is not None and (mass.shape != (num_pages, kv_heads, page) or mass.dtype != torch.float32):
            raise ValueError("mass must be float32 [num_pages, kv_heads, page_size]")
        if index < 0:
            raise ValueError("liblla runs on CUDA tensors only")
        if not (k_pages.is_contiguous() and v_pages.is_contiguous() and page_table.is_contiguous() and
                lens.is_contiguous() and v_pages.get_device() == index and page_table.get_device() == index and
                lens.get_device() == index and (mass is None or mass.is_contiguous() and mass.get_device() == index)):
            raise ValueError("the cache's tensors must be contiguous, on one device")
        self.num_seqs, self.kv_heads, self.d, self.dv = num_seqs, kv_heads, d, dv
        self.k_pages, self.v_pages, self.mass = k_pages, v_pages, mass
        self.page_table, self.lens, self.dtype, self.device, self._index = page_table, lens, dtype, device, index
        self._packed = _CACHE.pack(
            k_pages.data_ptr(), v_pages.data_ptr(), 0 if mass is None else mass.data_ptr(),
            page_table.data_ptr(), lens.data_ptr(), num_seqs, kv_heads, page, max_pages,
            num_pages, d, dv, code, 0, 0)


def _paged_rows(name, x, cache, shape):
    if x.shape != shape or x.dtype != cache.dtype or x.get_device() != cache._index or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {cache.dtype} tensor of shape {shape} on {cache.device}")


def _paged_starts(starts, cache):
    if starts.dtype != torch.int32 or starts.shape != (cache.num_seqs + 1,) or \
            starts.get_device() != cache._index or not starts.is_contiguous():
        raise ValueError("starts must be a contiguous int32 [num_seqs + 1] tensor on the cache's device")


def _paged_stream(cache, stream):
    """The raw handle of a stream that a call was given."""
    if getattr(stream, "device_index", cache._index) != cache._index:
        raise ValueError(f"the stream must be one of {cache.device}, where the cache is")
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(cache, stream):
    """What a call on another stream than the current one allocates belongs to that stream."""
    if not isinstance(stream, torch.cuda.Stream):  # a raw handle; 0 is the default stream's
        raw = _paged_stream(cache, stream)
        stream = torch.cuda.ExternalStream(raw, device=cache.device) if raw else torch.cuda.default_stream(cache.device)
    return torch.cuda.stream(stream)


def _paged_call(fn, cache, stream, *args):
    """Calls an entry point with the cache's device current: the library works on the current one, and the
    default stream's handle is the same on all of them. (A decode step makes this call once per
    layer, so the current device is asked for without torch.cuda's own checks.)"""
    raw = torch._C._cuda_getCurrentRawStream(cache._index) if stream is None else _paged_stream(cache, stream)
    if torch._C._cuda_getDevice() == cache._index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(cache._index):
            st = fn(*args, raw)
    if st:
        raise LlaError(st, fn.__name__)


def lla_paged_append(k, v, cache: PagedCache, starts, stream=None):
    """Writes the new tokens' keys k [tokens, kv_heads, d] and values v [tokens, kv_heads, dv] into
    their slots of the cache and sets their mass, if it has one, to zero. Sequence b's tokens are
    rows starts[b] .. starts[b+1]-1 and its last positions (cache.lens counts them already)."""
    tokens = k.shape[0]
    _paged_rows("k", k, cache, (tokens, cache.kv_heads, cache.d))
    _paged_rows("v", v, cache, (tokens, cache.kv_heads, cache.dv))
    _paged_starts(starts, cache)
    _paged_call(_load().lla_paged_append, cache, stream, cache._packed, k.data_ptr(), v.data_ptr(), starts.data_ptr(), tokens)


def lla_paged_append_rotary(k, v, cache: PagedCache, starts, spec: RotarySpec, q=None, r=None, offsets=None, q_out=None,
                            r_out=None, stream=None):
    """lla_paged_append with the keys rotated, and the queries q [tokens, q_heads, d] and probe r (like q) of
    the same tokens; returns (q_out, r_out), None where there is none. A token's position is that of its
    sequence's first new token's slot plus offsets [tokens] int32 (None: its own slot's). q_out may be q."""
    tokens = k.shape[0]
    _paged_rows("k", k, cache, (tokens, cache.kv_heads, cache.d))
    _paged_rows("v", v, cache, (tokens, cache.kv_heads, cache.dv))
    _paged_starts(starts, cache)
    if offsets is not None and (offsets.dtype != torch.int32 or offsets.shape != (tokens,) or
                                offsets.get_device() != cache._index or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 [tokens] tensor on the cache's device")
    if q is None and (r is not None or q_out is not None) or r is None and r_out is not None:
        raise ValueError("r comes with q, and outputs with their inputs")
    outs = []
    for name, x, y in (("q", q, q_out), ("r", r, r_out)):
        if x is not None:
            if len(q.shape) != 3:
                raise ValueError("expected q [tokens, q_heads, d]")
            _paged_rows(name, x, cache, (tokens, q.shape[1], cache.d))
            if y is None:
                if stream is None:
                    y = torch.empty_like(x)
                else:
                    with _on_stream(cache, stream):
                        y = x.new_empty(x.shape)
            else:
                _paged_rows(name + "_out", y, cache, x.shape)
        outs.append(y)
    ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    _paged_call(_load().lla_paged_append_rotary, cache, stream, cache._packed, spec._packed, k.data_ptr(), v.data_ptr(),
                ptr(q), ptr(r), ptr(outs[0]), ptr(outs[1]), 0 if q is None else q.shape[1], ptr(offsets),
                starts.data_ptr(), tokens)
    return tuple(outs)


def _paged_query(q, cache, starts, h, r, max_new, window, sinks, track_mass, out, lse, path):
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.d or q.dtype != cache.dtype or q.get_device() != cache._index or \
            not q.is_contiguous():
        raise ValueError(f"q must be a contiguous {cache.dtype} tensor [tokens, q_heads, {cache.d}] on {cache.device}")
    tokens, heads, _ = shape
    if r is not None:
        _paged_rows("r", r, cache, shape)
    _paged_starts(starts, cache)
    return _QUERY.pack(q.data_ptr(), 0 if r is None else r.data_ptr(), 0 if out is None else out.data_ptr(),
                       0 if lse is None else lse.data_ptr(), starts.data_ptr(), tokens,
                       tokens if max_new is None else max_new, heads, h, window, sinks,
                       1 if track_mass else 0, path, 0, 0)


def _paged_attend(fn, parents, q, cache, starts, h, r, max_new, window, sinks, track_mass, out, lse, workspace, stream,
                  path):
    shape = q.shape
    if out is not None:
        _paged_rows("out", out, cache, (*shape[:2], cache.dv))
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != torch.float32 or
                            lse.get_device() != cache._index or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [tokens, q_heads] tensor on the cache's device")
    if stream is None:
        if out is None:
            out = torch.empty_like(q) if cache.dv == cache.d else \
                torch.empty((*shape[:2], cache.dv), dtype=q.dtype, device=cache.device)
        if lse is None:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=cache.device)
    else:
        with _on_stream(cache, stream):
            out = q.new_empty((*shape[:2], cache.dv)) if out is None else out
            lse = q.new_empty(shape[:2], dtype=torch.float32) if lse is None else lse
    query = _paged_query(q, cache, starts, h, r, max_new, window, sinks, track_mass, out, lse, path)
    wp = wb = 0
    if workspace is not None:
        if workspace.get_device() != cache._index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _paged_call(fn, cache, stream, cache._packed, query, *parents, wp, wb)
    return out, lse


def lla_paged_attention(q, cache: PagedCache, starts, h: float, r=None, max_new=None, window=0,
                        sinks=0, track_mass=False, out=None, lse=None, workspace=None, stream=None,
                        *, path=0):
    """Attention of the new tokens q [tokens, q_heads, d] over the cache that they were appended to;
    returns (out [tokens, q_heads, dv], lse [tokens, q_heads] float32). With a probe r (like q) the
    Parallax output, else softmax attention. The token at position i sees positions j <= i, all of
    them (window = 0) or the last `window` and the first `sinks`. track_mass adds the weights to
    cache.mass. Rows that no sequence covers are not written: in tensors that this call allocates they hold
    anything. max_new: a bound of the tokens of one sequence (default: all); giving it lets a
    decode step run as one."""
    return _paged_attend(_load().lla_paged_attention, (), q, cache, starts, h, r, max_new, window, sinks, track_mass, out,
                         lse, workspace, stream, path)


def lla_paged_workspace_size(q, cache: PagedCache, starts, h: float, r=None, max_new=None, window=0,
                             sinks=0, track_mass=False, lse=None, *, path=0) -> int:
    """Bytes of device scratch that lla_paged_attention takes for these arguments (as `workspace`,
    or from the stream-ordered allocator)."""
    query = _paged_query(q, cache, starts, h, r, max_new, window, sinks, track_mass, None, lse, path)
    return int(_load().lla_paged_workspace_size(cache._packed, query))


MAX_NODES = 1024  # of a sequence's tree


def _paged_parents(parents, cache, tokens):
    if parents.dtype != torch.int32 or parents.shape != (tokens,) or parents.get_device() != cache._index or \
            not parents.is_contiguous():
        raise ValueError("parents must be a contiguous int32 [tokens] tensor on the cache's device")


def lla_paged_tree_attention(q, cache: PagedCache, starts, parents, h: float, r=None, max_new=None, window=0, sinks=0,
                             out=None, lse=None, workspace=None, stream=None, *, path=0):
    """Attention of trees of drafted tokens over the cache that they were appended to: sequence b's new
    tokens are nodes, parents [tokens] int32 holds of each its parent's index among them (below its
    own) or -1. A node sees the positions before the nodes, its ancestors and itself; its position is
    that of the first node's slot plus its depth. Otherwise as lla_paged_attention, but cache.mass gets no weights.
    max_new: a bound of the nodes of one sequence (default: all tokens, at most 1024)."""
    tokens = q.shape[0]
    _paged_parents(parents, cache, tokens)
    max_new = min(tokens, MAX_NODES) if max_new is None else max_new
    return _paged_attend(_load().lla_paged_tree_attention, (parents.data_ptr(),), q, cache, starts, h, r, max_new, window,
                         sinks, False, out, lse, workspace, stream, path)


def lla_paged_tree_workspace_size(q, cache: PagedCache, starts, h: float, r=None, max_new=None, window=0, sinks=0,
                                  lse=None, *, path=0) -> int:
    """Bytes of device scratch that lla_paged_tree_attention takes for these arguments."""
    max_new = min(q.shape[0], MAX_NODES) if max_new is None else max_new
    query = _paged_query(q, cache, starts, h, r, max_new, window, sinks, False, None, lse, path)
    return int(_load().lla_paged_tree_workspace_size(cache._packed, query))


def lla_paged_evict(cache: PagedCache, to: PagedCache, budget: int, sinks=0, recent=0, kept=None,
                    stream=None):
    """Keeps min(lens, budget) positions of every sequence and key/value head of `cache` -- the first
    `sinks`, the last `recent`, and those of the largest mass -- in `to`, whose lens, pages and mass
    are written; returns kept [num_seqs, kv_heads, budget] int32, their positions (-1 past the
    last)."""
    if cache.mass is None or to.mass is None:
        raise ValueError("eviction needs the mass of both caches")
    if cache._index != to._index:
        raise ValueError("the caches must be on one device")
    if budget < 1:
        raise ValueError("budget must be at least 1")
    shape = (cache.num_seqs, cache.kv_heads, budget)
    if kept is None:
        if stream is None:
            kept = torch.empty(shape, dtype=torch.int32, device=cache.device)
        else:
            with _on_stream(cache, stream):
                kept = torch.empty(shape, dtype=torch.int32, device=cache.device)
    elif kept.shape != shape or kept.dtype != torch.int32 or kept.get_device() != cache._index \
            or not kept.is_contiguous():
        raise ValueError(f"kept must be a contiguous int32 tensor of shape {shape}")
    _paged_call(_load().lla_paged_evict, cache, stream, cache._packed, to._packed, budget, sinks, recent, kept.data_ptr())
    return kept


def _paged_ints(name, x, cache, shape):
    if x.dtype != torch.int32 or x.shape != shape or x.get_device() != cache._index or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on the cache's device")


def _paged_new(cache, stream, *shapes):
    """Integer outputs that a call allocates, which belong to its stream."""
    if stream is None:
        return [torch.empty(s, dtype=torch.int32, device=cache.device) for s in shapes]
    with _on_stream(cache, stream):
        return [torch.empty(s, dtype=torch.int32, device=cache.device) for s in shapes]


def lla_paged_fork(cache: PagedCache, to: PagedCache, parents, refs, stream=None):
    """Sequence c of `to` (another table and lens over the same pages) becomes a copy of sequence parents[c] of
    `cache` (int32; -1: an empty one) that shares its pages; refs [num_pages] int32 counts the table entries that
    hold each page."""
    if cache._index != to._index:
        raise ValueError("the caches must be on one device")
    _paged_ints("parents", parents, to, (to.num_seqs,))
    _paged_ints("refs", refs, cache, cache.k_pages.shape[:1])
    _paged_call(_load().lla_paged_fork, cache, stream, cache._packed, to._packed, parents.data_ptr(), refs.data_ptr())


def lla_paged_free(cache: PagedCache, refs, keep=None, stream=None):
    """Shortens every sequence to its first keep[b] positions (int32; None: to none) and releases the pages
    behind them."""
    _paged_ints("refs", refs, cache, cache.k_pages.shape[:1])
    if keep is not None:
        _paged_ints("keep", keep, cache, (cache.num_seqs,))
    _paged_call(_load().lla_paged_free, cache, stream, cache._packed, None if keep is None else keep.data_ptr(),
                refs.data_ptr())


def lla_paged_grow(cache: PagedCache, starts, refs, copies=None, left=None, stream=None):
    """Room for the new tokens of `starts`: cache.lens grows by them and the table gets the lowest free pages.
    Returns (copies [num_seqs, 2], left [1]), int32: the pages (old, new) that lla_paged_copy has to copy in
    each layer because others hold the old one too (-1: none), and how many pages are free afterwards. left
    below zero: so many pages were missing, or table entries of sequences that would outgrow their rows, and nothing
    has changed; a sequence with copies of -2 was left out (see lla.h). Neither's new tokens may be appended."""
    _paged_starts(starts, cache)
    _paged_ints("refs", refs, cache, cache.k_pages.shape[:1])
    if copies is not None:
        _paged_ints("copies", copies, cache, (cache.num_seqs, 2))
    if left is not None:
        _paged_ints("left", left, cache, (1,))
    if copies is None:
        copies, = _paged_new(cache, stream, (cache.num_seqs, 2))
    if left is None:
        left, = _paged_new(cache, stream, (1,))
    _paged_call(_load().lla_paged_grow, cache, stream, cache._packed, starts.data_ptr(), refs.data_ptr(),
                copies.data_ptr(), left.data_ptr())
    return copies, left


def lla_paged_copy(cache: PagedCache, to: PagedCache, pairs, stream=None):
    """Copies page pairs[i, 0] of `cache` to page pairs[i, 1] of `to` (keys, values, and mass where both have
    it); pairs [n, 2] int32, negative numbers: skipped. Both may be one cache."""
    if cache._index != to._index:
        raise ValueError("the caches must be on one device")
    count = pairs.shape[0]
    _paged_ints("pairs", pairs, cache, (count, 2))
    _paged_call(_load().lla_paged_copy, cache, stream, cache._packed, to._packed, pairs.data_ptr(), count)


def lla_paged_compact(cache: PagedCache, starts, path, tokens=None, keep=None, stream=None):
    """Keeps one path of each sequence's new tokens: path [num_seqs, max_path] int32, rising indices among
    them, -1 past the last. They move to the front of the new tokens' slots; returns keep [num_seqs]
    int32, the lengths to give to lla_paged_free once all layers are done. tokens: a bound of the batch's
    (default: none)."""
    _paged_starts(starts, cache)
    if len(path.shape) != 2:
        raise ValueError("path must be [num_seqs, max_path]")
    _paged_ints("path", path, cache, (cache.num_seqs, path.shape[1]))
    if keep is not None:
        _paged_ints("keep", keep, cache, (cache.num_seqs,))
    else:
        keep, = _paged_new(cache, stream, (cache.num_seqs,))
    _paged_call(_load().lla_paged_compact, cache, stream, cache._packed, starts.data_ptr(),
                (1 << 30) - 1 if tokens is None else tokens, path.data_ptr(), path.shape[1], keep.data_ptr())
    return keep


def lla_stream_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(_load().lla_stream_status(_stream_ptr(stream)))


def profile_enable(on: bool = True):
    _check(_load().lla_profile_enable(1 if on else 0), "lla_profile_enable")


def profile_collect():
    """(summed ms per stage as a dict, number of recorded lla_forward calls)."""
    buf = (ctypes.c_float * NUM_STAGES)()
    n = ctypes.c_int(0)
    _check(_load().lla_profile_collect(buf, NUM_STAGES, ctypes.byref(n)), "lla_profile_collect")
    return dict(zip(STAGE_NAMES, list(buf))), n.value
