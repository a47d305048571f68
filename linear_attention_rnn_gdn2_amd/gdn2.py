"""Thin ctypes binding of ``libgdn2.so`` (see ``include/gdn2.h``).

Argument marshalling only: torch provides device memory and the current HIP
stream; every step of the computation runs in the library's gfx950 kernels.
There is no CPU fallback: if the library is missing, or a tensor is not on a
GPU, the call raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn2.so")

GDN2_DTYPE_BF16, GDN2_DTYPE_F32, GDN2_DTYPE_I32, GDN2_DTYPE_F16, GDN2_DTYPE_I64 = 1, 2, 3, 4, 5
_DTYPES = {torch.bfloat16: GDN2_DTYPE_BF16, torch.float32: GDN2_DTYPE_F32, torch.int32: GDN2_DTYPE_I32,
           torch.float16: GDN2_DTYPE_F16, torch.int64: GDN2_DTYPE_I64}
GDN2_STATE_KV, GDN2_STATE_VK = 0, 1
_LAYOUTS = {"kv": GDN2_STATE_KV, "vk": GDN2_STATE_VK}

STATUS = {0: "OK", -1: "NULL_ARG", -2: "DTYPE", -3: "SHAPE", -4: "HEADS",
          -5: "UNSUPPORTED", -6: "LAYOUT", -7: "ALIAS", -8: "HIP", -9: "WORKSPACE"}

EXPORTED = ["gdn2_chunk_fwd", "gdn2_chunk_fwd_opts", "gdn2_chunk_fwd_noalloc", "gdn2_chunk_fwd_check",
            "gdn2_split_plan",
            "gdn2_recurrent_fwd", "gdn2_recurrent_fwd_opts", "gdn2_recurrent_fwd_check",
            "gdn2_chunk_bwd", "gdn2_chunk_bwd_check", "gdn2_last_error", "gdn2_abi_version",
            "gdn2_delta_chunk_fwd", "gdn2_delta_chunk_fwd_check", "gdn2_delta_chunk_fwd_workspace",
            "gdn2_delta_chunk_bwd", "gdn2_delta_chunk_bwd_check", "gdn2_delta_chunk_bwd_workspace",
            "gdn2_delta_recurrent_fwd", "gdn2_delta_recurrent_fwd_check",
            "gdn2_qk_norm_rope_fwd", "gdn2_qk_norm_rope_fwd_check",
            "gdn2_qk_norm_rope_bwd", "gdn2_qk_norm_rope_bwd_check", "gdn2_qk_norm_rope_bwd_workspace",
            "gdn2_linear_scan_fwd", "gdn2_linear_scan_fwd_check", "gdn2_linear_scan_fwd_workspace",
            "gdn2_linear_scan_recurrent_fwd", "gdn2_linear_scan_recurrent_fwd_check",
            "gdn2_linear_scan_bwd", "gdn2_linear_scan_bwd_check", "gdn2_linear_scan_bwd_workspace",
            "gdn2_short_conv_fwd", "gdn2_short_conv_fwd_check",
            "gdn2_short_conv_recurrent_fwd", "gdn2_short_conv_recurrent_fwd_check",
            "gdn2_short_conv_bwd", "gdn2_short_conv_bwd_check", "gdn2_short_conv_bwd_workspace",
            "gdn2_layer_norm_fwd", "gdn2_layer_norm_fwd_check",
            "gdn2_layer_norm_bwd", "gdn2_layer_norm_bwd_check", "gdn2_layer_norm_bwd_workspace"]


class Gdn2Tensor(ctypes.Structure):
    """Mirror of ``gdn2_tensor``."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class Gdn2FwdOptions(ctypes.Structure):
    """Mirror of ``gdn2_fwd_options``."""
    _fields_ = [("struct_size", ctypes.c_int32), ("seq_split_chunks", ctypes.c_int32),
                ("state_layout", ctypes.c_int32), ("qk_l2norm", ctypes.c_int32)]


def make_options(seq_split=0, state_layout="kv", qk_l2norm=False):
    """A filled ``gdn2_fwd_options`` (state_layout "kv": [N, HV, K, V],
    "vk": [N, HV, V, K])."""
    if state_layout not in _LAYOUTS:
        raise ValueError(f"state_layout must be 'kv' or 'vk', not {state_layout!r}")
    return Gdn2FwdOptions(ctypes.sizeof(Gdn2FwdOptions), int(seq_split or 0), _LAYOUTS[state_layout],
                          1 if qk_l2norm else 0)


class Gdn2Error(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"gdn2 error {code} ({STATUS.get(code, '?')}): {message}")
        self.code = code
        self.status = STATUS.get(code, "?")


_lib = None


def load_library():
    """Load libgdn2.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no fallback implementation)")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(Gdn2Tensor)
        lib.gdn2_chunk_fwd.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, ctypes.c_void_p]
        lib.gdn2_chunk_fwd.restype = ctypes.c_int
        lib.gdn2_chunk_fwd_opts.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P,
                                            ctypes.POINTER(Gdn2FwdOptions), ctypes.c_void_p]
        lib.gdn2_chunk_fwd_opts.restype = ctypes.c_int
        lib.gdn2_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P,
                                               ctypes.POINTER(Gdn2FwdOptions), ctypes.c_void_p]
        lib.gdn2_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.gdn2_recurrent_fwd.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, ctypes.c_void_p]
        lib.gdn2_recurrent_fwd.restype = ctypes.c_int
        lib.gdn2_recurrent_fwd_opts.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P,
                                                ctypes.POINTER(Gdn2FwdOptions), ctypes.c_void_p]
        lib.gdn2_recurrent_fwd_opts.restype = ctypes.c_int
        lib.gdn2_recurrent_fwd_check.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P]
        lib.gdn2_recurrent_fwd_check.restype = ctypes.c_int
        lib.gdn2_split_plan.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
        lib.gdn2_split_plan.restype = ctypes.c_int
        lib.gdn2_chunk_fwd_check.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P]
        lib.gdn2_chunk_fwd_check.restype = ctypes.c_int
        lib.gdn2_chunk_bwd.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, P, P, P, P, P, P,
                                       ctypes.c_void_p]
        lib.gdn2_chunk_bwd.restype = ctypes.c_int
        lib.gdn2_chunk_bwd_check.argtypes = [P, P, P, P, P, P, ctypes.c_float, P, P, P, P, P, P, P, P, P, P, P]
        lib.gdn2_chunk_bwd_check.restype = ctypes.c_int
        A, F, I32, I64 = ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_int64  # A: an address
        for name, args in {
            "gdn2_delta_chunk_fwd": [A] * 5 + [F] + [A] * 4 + [A, A, I64, A],
            "gdn2_delta_chunk_fwd_check": [A] * 5 + [F] + [A] * 4 + [A],
            "gdn2_delta_recurrent_fwd": [A] * 5 + [F] + [A] * 4 + [A, A],
            "gdn2_delta_recurrent_fwd_check": [A] * 5 + [F] + [A] * 4 + [A],
            "gdn2_delta_chunk_bwd": [A] * 5 + [F] + [A] * 10 + [A, I64, A],
            "gdn2_delta_chunk_bwd_check": [A] * 5 + [F] + [A] * 10,
            "gdn2_qk_norm_rope_fwd": [A] * 8 + [A, A],
            "gdn2_qk_norm_rope_fwd_check": [A] * 8 + [A],
            "gdn2_qk_norm_rope_bwd": [A] * 12 + [A, A, I64, A],
            "gdn2_qk_norm_rope_bwd_check": [A] * 12 + [A],
            "gdn2_linear_scan_fwd": [A] * 8 + [A, I64, A],
            "gdn2_linear_scan_fwd_check": [A] * 8,
            "gdn2_linear_scan_recurrent_fwd": [A] * 8 + [A],
            "gdn2_linear_scan_recurrent_fwd_check": [A] * 8,
            "gdn2_linear_scan_bwd": [A] * 12 + [A, I64, A],
            "gdn2_linear_scan_bwd_check": [A] * 12,
            "gdn2_short_conv_fwd": [A] * 8 + [A],
            "gdn2_short_conv_fwd_check": [A] * 8,
            "gdn2_short_conv_recurrent_fwd": [A] * 8 + [A],
            "gdn2_short_conv_recurrent_fwd_check": [A] * 8,
            "gdn2_short_conv_bwd": [A] * 12 + [A, I64, A],
            "gdn2_short_conv_bwd_check": [A] * 12,
            "gdn2_layer_norm_fwd": [A] * 6 + [A],
            "gdn2_layer_norm_fwd_check": [A] * 6,
            "gdn2_layer_norm_bwd": [A] * 10 + [A, I64, A],
            "gdn2_layer_norm_bwd_check": [A] * 10,
        }.items():
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, ctypes.c_int
        for name, args in {"gdn2_delta_chunk_fwd_workspace": [I64, I32, I32],
                           "gdn2_delta_chunk_bwd_workspace": [I64, I32, I32, I32, I32, I32],
                           "gdn2_qk_norm_rope_bwd_workspace": [I64, I32, I32, I32],
                           "gdn2_linear_scan_fwd_workspace": [I64, I32, I32],
                           "gdn2_linear_scan_bwd_workspace": [I64, I32, I32],
                           "gdn2_short_conv_bwd_workspace": [I64, I32, I32],
                           "gdn2_layer_norm_bwd_workspace": [I64, I32, I32]}.items():
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, I64
        lib.gdn2_last_error.argtypes = []
        lib.gdn2_last_error.restype = ctypes.c_char_p
        lib.gdn2_abi_version.restype = ctypes.c_int
        _lib = lib
    return _lib


def last_error() -> str:
    return load_library().gdn2_last_error().decode()


def describe(t):
    """Build a gdn2_tensor descriptor for a torch tensor (None -> NULL)."""
    if t is None:
        return None
    d = Gdn2Tensor()
    d.data = t.data_ptr() if t.numel() > 0 else None
    d.dtype = _DTYPES.get(t.dtype, 0)
    d.ndim = t.dim()
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


def _ptr(d):
    return None if d is None else ctypes.byref(d)


def _scale_arg(scale):
    return 0.0 if scale is None else float(scale)


def check(q, k, v, g=None, beta=None, w=None, scale=None, initial_state=None,
          cu_seqlens=None, out=None, final_state=None):
    """Run the library's host-side validation only (no GPU needed).

    Returns the status code (0 = valid); never touches device memory."""
    lib = load_library()
    ds = [describe(x) for x in (q, k, v, g, beta, w)]
    rest = [describe(x) for x in (initial_state, cu_seqlens, out, final_state)]
    return lib.gdn2_chunk_fwd_check(*[_ptr(d) for d in ds], _scale_arg(scale),
                                    *[_ptr(d) for d in rest])


def split_plan(T, N, HV, num_cu):
    """The library's automatic segment length (0 = whole sequences) for T
    tokens in N sequences with HV value heads on ``num_cu`` compute units."""
    return load_library().gdn2_split_plan(int(T), int(N), int(HV), int(num_cu))


def _prepare(q, k, v, initial_state, cu_seqlens, output_final_state, out, final_state, g, beta, w,
             state_layout="kv"):
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("w", w),
                    ("initial_state", initial_state), ("cu_seqlens", cu_seqlens)):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
    T, HV, V = v.shape
    K = q.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if out is None:
        out = torch.empty_like(v, dtype=q.dtype, memory_format=torch.contiguous_format)
    if final_state is None and output_final_state:
        shape = (N, HV, V, K) if state_layout == "vk" else (N, HV, K, V)
        final_state = torch.empty(shape, dtype=torch.float32, device=v.device)
    descs = [describe(x) for x in (q, k, v, g, beta, w)]
    rest = [describe(x) for x in (initial_state, cu_seqlens, out, final_state)]
    return out, final_state, descs, rest


def chunk_fwd(q, k, v, g=None, beta=None, w=None, scale=None, initial_state=None,
              cu_seqlens=None, output_final_state=True, out=None, final_state=None,
              seq_split=None, state_layout="kv", qk_l2norm=False):
    """GDN-2 chunked prefill forward on the current HIP stream.

    q, k [T, H, K] and v, w [T, HV, V], beta [T, HV, K], out: bf16 or
    float16 (q's type); g [T, HV, K] float32, bf16 or float16;
    initial_state and final_state [N, HV, K, V] float32 or bf16
    ([N, HV, V, K] with ``state_layout="vk"``); cu_seqlens [N + 1] int32 or int64 (None: one
    sequence). Strided views are accepted where the rows are contiguous.
    ``scale`` None or 0 means 1/sqrt(K). Returns (out [T, HV, V],
    final_state or None); preallocated ``out`` / ``final_state`` are written
    in place. ``seq_split``: None or 0 automatic, -1 never split sequences,
    n > 0 split every sequence into segments of n 64-token chunks.
    ``qk_l2norm``: normalise q and k rows in the kernel.
    """
    lib = load_library()
    out, final_state, descs, rest = _prepare(q, k, v, initial_state, cu_seqlens, output_final_state, out,
                                             final_state, g, beta, w, state_layout)
    stream = torch.cuda.current_stream(v.device).cuda_stream
    if seq_split is None and state_layout == "kv" and not qk_l2norm:
        rc = lib.gdn2_chunk_fwd(*[_ptr(d) for d in descs], _scale_arg(scale),
                                *[_ptr(d) for d in rest], ctypes.c_void_p(stream))
    else:
        opts = make_options(seq_split, state_layout, qk_l2norm)
        rc = lib.gdn2_chunk_fwd_opts(*[_ptr(d) for d in descs], _scale_arg(scale),
                                     *[_ptr(d) for d in rest], ctypes.byref(opts), ctypes.c_void_p(stream))
    if rc != 0:
        raise Gdn2Error(rc, last_error())
    return out, final_state


def chunk_fwd_noalloc(q, k, v, g=None, beta=None, w=None, scale=None, initial_state=None,
                      cu_seqlens=None, out=None, final_state=None, seq_split=None, state_layout="kv",
                      qk_l2norm=False):
    """:func:`chunk_fwd` through ``gdn2_chunk_fwd_noalloc``: the library
    allocates no device memory (a split run's workspace is its fixed device
    array). ``out`` and ``final_state`` must be preallocated by the caller
    (``final_state`` None: not produced)."""
    lib = load_library()
    if out is None:
        raise ValueError("chunk_fwd_noalloc needs a preallocated out")
    _, _, descs, rest = _prepare(q, k, v, initial_state, cu_seqlens, False, out, final_state, g, beta, w,
                                 state_layout)
    stream = torch.cuda.current_stream(v.device).cuda_stream
    opts = make_options(seq_split, state_layout, qk_l2norm)
    rc = lib.gdn2_chunk_fwd_noalloc(*[_ptr(d) for d in descs], _scale_arg(scale), *[_ptr(d) for d in rest],
                                    ctypes.byref(opts), ctypes.c_void_p(stream))
    if rc != 0:
        raise Gdn2Error(rc, last_error())
    return out, final_state


def recurrent_fwd(q, k, v, g=None, beta=None, w=None, scale=None, initial_state=None,
                  cu_seqlens=None, output_final_state=True, out=None, final_state=None,
                  state_layout="kv", qk_l2norm=False):
    """The same forward evaluated token by token (decode and short spans).

    Tensors and options as in :func:`chunk_fwd`. ``final_state`` may be
    ``initial_state`` itself to update the state in place.
    """
    lib = load_library()
    out, final_state, descs, rest = _prepare(q, k, v, initial_state, cu_seqlens, output_final_state, out,
                                             final_state, g, beta, w, state_layout)
    stream = torch.cuda.current_stream(v.device).cuda_stream
    if state_layout == "kv" and not qk_l2norm:
        rc = lib.gdn2_recurrent_fwd(*[_ptr(d) for d in descs], _scale_arg(scale),
                                    *[_ptr(d) for d in rest], ctypes.c_void_p(stream))
    else:
        opts = make_options(0, state_layout, qk_l2norm)
        rc = lib.gdn2_recurrent_fwd_opts(*[_ptr(d) for d in descs], _scale_arg(scale),
                                         *[_ptr(d) for d in rest], ctypes.byref(opts), ctypes.c_void_p(stream))
    if rc != 0:
        raise Gdn2Error(rc, last_error())
    return out, final_state


BWD_GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dw", "d_initial_state")


def _bwd_descs(q, k, v, g, beta, w, initial_state, cu_seqlens, d_out, d_final_state, grads):
    ins = [describe(x) for x in (q, k, v, g, beta, w)]
    mid = [describe(x) for x in (initial_state, cu_seqlens, d_out, d_final_state)]
    outs = [describe(grads.get(n)) for n in BWD_GRADS]
    return ins, mid, outs


def chunk_bwd(q, k, v, g, beta, w, d_out, scale=None, initial_state=None, cu_seqlens=None,
              d_final_state=None, need_d_initial_state=True, grads=None):
    """Backward of :func:`chunk_fwd` on the current HIP stream.

    q, k [T, H, K], v, w [T, HV, V], beta [T, HV, K], d_out [T, HV, V]: one
    16-bit type, bf16 or float16; g [T, HV, K]: float32, bf16 or float16;
    initial_state and d_final_state [N, HV, K, V]: float32 (the states may
    be None: zero). Returns a dict with dq, dk ([T, H, K]), dv, dw
    ([T, HV, V]), dbeta ([T, HV, K]) in q's type, dg ([T, HV, K]) in g's
    type and d_initial_state (float32 [N, HV, K, V], or None when not
    requested). Tensors given in ``grads`` are written in place.
    """
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("w", w), ("d_out", d_out),
                    ("initial_state", initial_state), ("cu_seqlens", cu_seqlens), ("d_final_state", d_final_state)):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
    T, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    dev = v.device
    out = dict(grads or {})
    io, gt = q.dtype, g.dtype
    shapes = {"dq": ((T, H, K), io), "dk": ((T, H, K), io), "dv": ((T, HV, V), io), "dw": ((T, HV, V), io),
              "dbeta": ((T, HV, K), io), "dg": ((T, HV, K), gt), "d_initial_state": ((N, HV, K, V), torch.float32)}
    for n, (shp, dt) in shapes.items():
        if out.get(n) is None and (n != "d_initial_state" or need_d_initial_state):
            out[n] = torch.empty(shp, dtype=dt, device=dev)
    out.setdefault("d_initial_state", None)
    ins, mid, outs = _bwd_descs(q, k, v, g, beta, w, initial_state, cu_seqlens, d_out, d_final_state, out)
    stream = torch.cuda.current_stream(dev).cuda_stream
    rc = lib.gdn2_chunk_bwd(*[_ptr(d) for d in ins], _scale_arg(scale), *[_ptr(d) for d in mid],
                            *[_ptr(d) for d in outs], ctypes.c_void_p(stream))
    if rc != 0:
        raise Gdn2Error(rc, last_error())
    return out


def check_bwd(q, k, v, g, beta, w, d_out, scale=None, initial_state=None, cu_seqlens=None,
              d_final_state=None, grads=None):
    """The library's host-side validation of a backward call only (no GPU needed)."""
    lib = load_library()
    ins, mid, outs = _bwd_descs(q, k, v, g, beta, w, initial_state, cu_seqlens, d_out, d_final_state, grads or {})
    return lib.gdn2_chunk_bwd_check(*[_ptr(d) for d in ins], _scale_arg(scale), *[_ptr(d) for d in mid],
                                    *[_ptr(d) for d in outs])


# ------------------------------------------------ scalar-gated delta rule --

QK_NORMS = {"none": 0, "l2": 1, "rms": 2}
DELTA_GRADS = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")
_DESC = struct.Struct("@Pii4q4q")  # gdn2_tensor
assert _DESC.size == ctypes.sizeof(Gdn2Tensor)


class Gdn2QkOptions(ctypes.Structure):
    """Mirror of ``gdn2_qk_options``."""
    _fields_ = [("struct_size", ctypes.c_int32), ("norm", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float)]


def _describe_all(tensors):
    """The descriptors of a call's tensors in one buffer: (buffer, the
    address of each, None for None). A decode step is launch-bound, so the
    descriptors are packed at once rather than built field by field."""
    vals = []
    for t in tensors:
        if t is None:
            vals += _NO_DESC
            continue
        shape = t.shape
        n = len(shape)
        if n > 4:
            raise ValueError("at most 4 dimensions")
        pad = _ZEROS[n]
        vals += (t.data_ptr(), _DTYPES.get(t.dtype, 0), n, *shape, *pad, *t.stride(), *pad)
    packer = _packer(len(tensors))
    buf = ctypes.create_string_buffer(packer.size)
    packer.pack_into(buf, 0, *vals)
    base = ctypes.addressof(buf)
    return buf, [None if t is None else base + i * _DESC.size for i, t in enumerate(tensors)]


_ZEROS = [(0,) * (4 - n) for n in range(5)]
_NO_DESC = (0,) * 11


@functools.lru_cache(maxsize=None)
def _packer(n):
    return struct.Struct("@" + _DESC.format[1:] * n)


def _one_device(names, tensors):
    """The GPU that holds every given tensor."""
    index = dev = None
    for name, t in zip(names, tensors):
        if t is None or t.get_device() == index:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (there is no CPU path)")
        if dev is not None:
            raise ValueError(f"{name} is on {t.device}, {names[0]} on {dev}")
        index, dev = t.get_device(), t.device
    return dev


def _launch(dev, call):
    """call(stream) with `dev` current, on its current stream."""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)  # current_stream().cuda_stream without its object
    if torch.cuda.current_device() == dev.index:
        rc = call(stream)
    else:
        with torch.cuda.device(dev):
            rc = call(stream)
    if rc != 0:
        raise Gdn2Error(rc, last_error())


def _workspace(nbytes, given, dev):
    """The caller's workspace tensor, or one from torch's allocator (ordered
    on the current stream, and private to a graph that is being captured)."""
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    if not given.is_cuda or given.device != dev or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return given


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


_DELTA_NAMES = ("q", "k", "v", "g", "beta", "initial_state", "cu_seqlens", "out", "final_state")


def _rank3(**tensors):
    for name, t in tensors.items():
        if t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions, not {t.dim()}")


def _delta_outputs(q, k, v, cu_seqlens, output_final_state, out, final_state, state_layout):
    if state_layout not in _LAYOUTS:
        raise ValueError(f"state_layout must be 'kv' or 'vk', not {state_layout!r}")
    _rank3(q=q, k=k, v=v)
    T, HV, V = v.shape
    K = q.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if out is None:
        out = torch.empty_like(v, dtype=q.dtype, memory_format=torch.contiguous_format)
    if final_state is None and output_final_state and N >= 1:
        shape = (N, HV, V, K) if state_layout == "vk" else (N, HV, K, V)
        final_state = torch.empty(shape, dtype=torch.float32, device=v.device)
    return N, out, final_state


def delta_chunk_fwd_workspace(T, N, HV):
    """Bytes of workspace of :func:`delta_chunk_fwd`."""
    return load_library().gdn2_delta_chunk_fwd_workspace(int(T), int(N), int(HV))


def delta_chunk_bwd_workspace(T, N, H, HV, K, V):
    """Bytes of workspace of :func:`delta_chunk_bwd`."""
    return load_library().gdn2_delta_chunk_bwd_workspace(int(T), int(N), int(H), int(HV), int(K), int(V))


def delta_chunk_fwd(q, k, v, g=None, beta=None, scale=None, initial_state=None, cu_seqlens=None,
                    output_final_state=True, out=None, final_state=None, state_layout="kv", qk_l2norm=False,
                    workspace=None, seq_split=0):
    """The scalar-gated delta rule, chunked, on the current HIP stream.

    S = e^g S, u = beta (v - S^T k), S += k u^T, o = scale S^T q, with one g
    and one beta per token and value head. q, k [T, H, K], v [T, HV, V], out:
    bf16 or float16 (q's type), strided rows accepted; beta [T, HV]: q's
    type; g [T, HV]: float32, bf16 or float16 (any non-negative strides);
    states and cu_seqlens, scale, state_layout and qk_l2norm as in
    :func:`chunk_fwd`. Returns (out, final_state or None). ``workspace``: a
    contiguous device tensor of at least ``delta_chunk_fwd_workspace(T, N,
    HV)`` bytes (None: taken from torch's allocator). ``seq_split``: 0 lets
    few long sequences run as parallel segments, -1 walks each whole.
    """
    lib = load_library()
    tensors = [q, k, v, g, beta, initial_state, cu_seqlens, out, final_state]
    dev = _one_device(_DELTA_NAMES, tensors)
    N, out, final_state = _delta_outputs(q, k, v, cu_seqlens, output_final_state, out, final_state, state_layout)
    ws = _workspace(lib.gdn2_delta_chunk_fwd_workspace(v.shape[0], N, v.shape[1]), workspace, dev)
    keep, d = _describe_all([q, k, v, g, beta, initial_state, cu_seqlens, out, final_state])
    opts = None
    if state_layout != "kv" or qk_l2norm or seq_split:
        opts = make_options(seq_split, state_layout, qk_l2norm)
    _launch(dev, lambda stream: lib.gdn2_delta_chunk_fwd(*d[:5], _scale_arg(scale), *d[5:],
                                                         None if opts is None else ctypes.addressof(opts),
                                                         *_ws_args(ws), stream))
    return out, final_state


def delta_recurrent_fwd(q, k, v, g=None, beta=None, scale=None, initial_state=None, cu_seqlens=None,
                        output_final_state=True, out=None, final_state=None, state_layout="kv", qk_l2norm=False):
    """:func:`delta_chunk_fwd` evaluated token by token (decode and short
    spans), in float32. ``final_state`` may be ``initial_state`` itself to
    update the state in place."""
    lib = load_library()
    tensors = [q, k, v, g, beta, initial_state, cu_seqlens, out, final_state]
    dev = _one_device(_DELTA_NAMES, tensors)
    _, out, final_state = _delta_outputs(q, k, v, cu_seqlens, output_final_state, out, final_state, state_layout)
    keep, d = _describe_all([q, k, v, g, beta, initial_state, cu_seqlens, out, final_state])
    opts = None
    if state_layout != "kv" or qk_l2norm:
        opts = make_options(0, state_layout, qk_l2norm)
    _launch(dev, lambda stream: lib.gdn2_delta_recurrent_fwd(*d[:5], _scale_arg(scale), *d[5:],
                                                             None if opts is None else ctypes.addressof(opts), stream))
    return out, final_state


def check_delta(q, k, v, g=None, beta=None, scale=None, initial_state=None, cu_seqlens=None, out=None,
                final_state=None, seq_split=0, state_layout="kv", qk_l2norm=False, recurrent=False):
    """The library's host-side validation of a :func:`delta_chunk_fwd` or
    (``recurrent``) :func:`delta_recurrent_fwd` call only (no GPU needed):
    the status code."""
    lib = load_library()
    keep, d = _describe_all([q, k, v, g, beta, initial_state, cu_seqlens, out, final_state])
    opts = make_options(seq_split, state_layout, qk_l2norm)
    fn = lib.gdn2_delta_recurrent_fwd_check if recurrent else lib.gdn2_delta_chunk_fwd_check
    return fn(*d[:5], _scale_arg(scale), *d[5:], ctypes.addressof(opts))


def _delta_bwd_list(q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state, grads):
    return [q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state] + [grads.get(n) for n in DELTA_GRADS]


def delta_chunk_bwd(q, k, v, g, beta, d_out, scale=None, initial_state=None, cu_seqlens=None, d_final_state=None,
                    need_d_initial_state=True, grads=None, workspace=None):
    """Backward of :func:`delta_chunk_fwd` on the current HIP stream (without
    qk_l2norm: see :func:`qk_norm_rope_bwd`), K = V.

    Tensors as there, all dense, states float32 K-major. Returns a dict with
    dq, dk, dv, dbeta in q's type, dg in g's and d_initial_state (float32, or
    None when not requested). Tensors given in ``grads`` are written in
    place. ``workspace``: at least ``delta_chunk_bwd_workspace(...)`` bytes
    (None: taken from torch's allocator).
    """
    lib = load_library()
    out = dict(grads or {})
    names = ("q", "k", "v", "g", "beta", "initial_state", "cu_seqlens", "d_out", "d_final_state") + DELTA_GRADS
    dev = _one_device(names, _delta_bwd_list(q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state, out))
    _rank3(q=q, k=k, v=v)
    T, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    shapes = {"dq": ((T, H, K), q.dtype), "dk": ((T, H, K), q.dtype), "dv": ((T, HV, V), q.dtype),
              "dg": ((T, HV), torch.float32 if g is None else g.dtype), "dbeta": ((T, HV), q.dtype),
              "d_initial_state": ((N, HV, K, V), torch.float32)}
    for n, (shape, dtype) in shapes.items():
        if out.get(n) is None:
            skip = n == "d_initial_state" and not (need_d_initial_state and N >= 1)
            out[n] = None if skip else torch.empty(shape, dtype=dtype, device=dev)
    ws = _workspace(lib.gdn2_delta_chunk_bwd_workspace(T, N, H, HV, K, V), workspace, dev)
    keep, d = _describe_all(_delta_bwd_list(q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state, out))
    _launch(dev, lambda stream: lib.gdn2_delta_chunk_bwd(*d[:5], _scale_arg(scale), *d[5:], *_ws_args(ws), stream))
    return out


def check_delta_bwd(q, k, v, g, beta, d_out, scale=None, initial_state=None, cu_seqlens=None, d_final_state=None,
                    grads=None):
    """The library's host-side validation of a :func:`delta_chunk_bwd` call only (no GPU needed)."""
    lib = load_library()
    keep, d = _describe_all(_delta_bwd_list(q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state,
                                            grads or {}))
    return lib.gdn2_delta_chunk_bwd_check(*d[:5], _scale_arg(scale), *d[5:])


# ---------------------------------------- norms and rotation of q and k --

def rope_table(positions, rot, base=10000.0, position_scale=1.0, device="cuda"):
    """The cosines and sines of positions 0 .. positions - 1 for
    :func:`qk_norm_rope`: float32 [positions, rot], angle position *
    position_scale * base^(-2 i / rot), formed in float64 (float32 products
    lose far positions' angles). ``position_scale`` below 1 fits a long
    context into the positions a model was trained on."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be a positive even number, not {rot}")
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * float(position_scale) * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _qk_options(norm, eps, interleaved):
    if norm not in QK_NORMS:
        raise ValueError(f"norm must be 'l2', 'rms' or 'none', not {norm!r}")
    return Gdn2QkOptions(ctypes.sizeof(Gdn2QkOptions), QK_NORMS[norm], 1 if interleaved else 0, float(eps or 0.0))


_QK_NAMES = ("q", "k", "q_weight", "k_weight", "rope", "positions", "q_out", "k_out")
_QK_BWD_NAMES = ("q", "k", "dq_out", "dk_out", "q_weight", "k_weight", "rope", "positions", "dq", "dk", "dq_weight",
                 "dk_weight")


def qk_norm_rope(q, k, norm="l2", eps=None, q_weight=None, k_weight=None, rope=None, positions=None,
                 interleaved=False, q_out=None, k_out=None):
    """Per-head norms of q and k with the position rotation, in one launch.

    q [T, H, K], k [T, HK, K]: bf16 or float16, strided rows accepted.
    ``norm``: "l2" (x / max(|x|, eps), eps 1e-12), "rms" (x / sqrt(mean x^2 +
    eps), eps 1e-6) or "none"; weights [K] float32 or q's type. ``rope``
    float32 [P, rot] (see :func:`rope_table`) turns the first rot elements of
    each row by ``positions`` [T] (int32 or int64, in [0, P)), in pairs (i,
    i + rot / 2) or, ``interleaved``, (2 i, 2 i + 1). Returns (q_out, k_out).
    """
    lib = load_library()
    dev = _one_device(_QK_NAMES, [q, k, q_weight, k_weight, rope, positions, q_out, k_out])
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    keep, d = _describe_all([q, k, q_weight, k_weight, rope, positions, q_out, k_out])
    opts = _qk_options(norm, eps, interleaved)
    _launch(dev, lambda stream: lib.gdn2_qk_norm_rope_fwd(*d, ctypes.addressof(opts), stream))
    return q_out, k_out


def qk_norm_rope_bwd_workspace(T, H, HK, K):
    """Bytes of workspace of :func:`qk_norm_rope_bwd` with a weight's gradient."""
    return load_library().gdn2_qk_norm_rope_bwd_workspace(int(T), int(H), int(HK), int(K))


def qk_norm_rope_bwd(q, k, dq_out, dk_out, norm="l2", eps=None, q_weight=None, k_weight=None, rope=None,
                     positions=None, interleaved=False, grads=None, workspace=None):
    """Backward of :func:`qk_norm_rope`: a dict with dq, dk (q's and k's shape
    and type) and dq_weight, dk_weight (the weight's type, None without one).
    Tensors given in ``grads`` are written in place."""
    lib = load_library()
    out = dict(grads or {})
    dev = _one_device(_QK_BWD_NAMES, [q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, out.get("dq"),
                                      out.get("dk"), out.get("dq_weight"), out.get("dk_weight")])
    _rank3(q=q, k=k)
    for n, t in (("dq", q), ("dk", k), ("dq_weight", q_weight), ("dk_weight", k_weight)):
        if out.get(n) is None:
            out[n] = None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)
    dw = out["dq_weight"] is not None or out["dk_weight"] is not None
    nbytes = lib.gdn2_qk_norm_rope_bwd_workspace(q.shape[0], q.shape[1], k.shape[1], q.shape[2]) if dw else 0
    ws = _workspace(nbytes, workspace, dev)
    keep, d = _describe_all([q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, out["dq"], out["dk"],
                             out["dq_weight"], out["dk_weight"]])
    opts = _qk_options(norm, eps, interleaved)
    _launch(dev, lambda stream: lib.gdn2_qk_norm_rope_bwd(*d, ctypes.addressof(opts), *_ws_args(ws), stream))
    return out


def check_qk_norm_rope(q, k, norm="l2", eps=None, q_weight=None, k_weight=None, rope=None, positions=None,
                       interleaved=False, q_out=None, k_out=None):
    """The library's host-side validation of a :func:`qk_norm_rope` call only (no GPU needed)."""
    keep, d = _describe_all([q, k, q_weight, k_weight, rope, positions, q_out, k_out])
    opts = _qk_options(norm, eps, interleaved)
    return load_library().gdn2_qk_norm_rope_fwd_check(*d, ctypes.addressof(opts))


def check_qk_norm_rope_bwd(q, k, dq_out, dk_out, norm="l2", eps=None, q_weight=None, k_weight=None, rope=None,
                           positions=None, interleaved=False, grads=None):
    """The library's host-side validation of a :func:`qk_norm_rope_bwd` call only (no GPU needed)."""
    g = grads or {}
    keep, d = _describe_all([q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, g.get("dq"), g.get("dk"),
                             g.get("dq_weight"), g.get("dk_weight")])
    opts = _qk_options(norm, eps, interleaved)
    return load_library().gdn2_qk_norm_rope_bwd_check(*d, ctypes.addressof(opts))


# ------------------------------------- around the rule: recurrence, convolution, norm --

INPUT_SCALES = {"none": 0, "convex": 1, "unit": 2}
ACTIVATIONS = {"none": 0, "silu": 1}
NORMS = {"layer": 0, "rms": 1}


class Gdn2ScanOptions(ctypes.Structure):
    """Mirror of ``gdn2_scan_options``."""
    _fields_ = [("struct_size", ctypes.c_int32), ("input_scale", ctypes.c_int32)]


class Gdn2ConvOptions(ctypes.Structure):
    """Mirror of ``gdn2_conv_options``."""
    _fields_ = [("struct_size", ctypes.c_int32), ("activation", ctypes.c_int32)]


class Gdn2NormOptions(ctypes.Structure):
    """Mirror of ``gdn2_norm_options``."""
    _fields_ = [("struct_size", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float)]


def _choice(what, names, value):
    if value not in names:
        raise ValueError(f"{what} must be one of {', '.join(map(repr, names))}, not {value!r}")
    return names[value]


@functools.lru_cache(maxsize=None)
def _scan_options(input_scale):
    return Gdn2ScanOptions(ctypes.sizeof(Gdn2ScanOptions), _choice("input_scale", INPUT_SCALES, input_scale))


@functools.lru_cache(maxsize=None)
def _conv_options(activation):
    return Gdn2ConvOptions(ctypes.sizeof(Gdn2ConvOptions), _choice("activation", ACTIVATIONS, activation))


@functools.lru_cache(maxsize=64)
def _norm_options(norm, eps):
    return Gdn2NormOptions(ctypes.sizeof(Gdn2NormOptions), _choice("norm", NORMS, norm), float(eps or 0.0))


def _rank2(**tensors):
    for name, t in tensors.items():
        if t.dim() != 2:
            raise ValueError(f"{name} must have 2 dimensions, not {t.dim()}")


def _sequences(cu_seqlens):
    return 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


_SCAN_NAMES = ("x", "g", "w", "initial_state", "cu_seqlens", "out", "final_state")
SCAN_GRADS = ("dx", "dg", "dw", "d_initial_state")


def linear_scan_fwd_workspace(T, N, D):
    """Bytes of workspace of :func:`linear_scan_fwd`."""
    return load_library().gdn2_linear_scan_fwd_workspace(int(T), int(N), int(D))


def linear_scan_bwd_workspace(T, N, D):
    """Bytes of workspace of :func:`linear_scan_bwd`."""
    return load_library().gdn2_linear_scan_bwd_workspace(int(T), int(N), int(D))


def _scan_outputs(x, g, w, initial_state, cu_seqlens, output_final_state, out, final_state):
    dev = _one_device(_SCAN_NAMES, (x, g, w, initial_state, cu_seqlens, out, final_state))
    _rank2(x=x, g=g)
    N = _sequences(cu_seqlens)
    if out is None:
        out = _like(x)
    if final_state is None and output_final_state and N >= 1:
        final_state = torch.empty((N, x.shape[1]), dtype=torch.float32, device=dev)
    return dev, N, out, final_state


def linear_scan_fwd(x, g, w=None, initial_state=None, cu_seqlens=None, output_final_state=True, input_scale="none",
                    out=None, final_state=None, workspace=None):
    """The gated linear recurrence per channel, on the current HIP stream:
    h = e^g h + m w x, out = h, with m = 1 (``input_scale`` "none"), 1 - e^g
    ("convex") or sqrt(1 - e^(2 g)) ("unit").

    x, w, out [T, D]: bf16, float16 or float32 (x's type), rows with any
    token stride; g [T, D]: float32 or x's type, <= 0; states [N, D]: float32
    or bf16; cu_seqlens as in :func:`chunk_fwd`. Returns (out, final_state or
    None). ``workspace``: a contiguous device tensor of at least
    ``linear_scan_fwd_workspace(T, N, D)`` bytes (None: taken from torch's
    allocator).
    """
    lib = load_library()
    opts = _scan_options(input_scale)
    dev, N, out, final_state = _scan_outputs(x, g, w, initial_state, cu_seqlens, output_final_state, out, final_state)
    ws = _workspace(lib.gdn2_linear_scan_fwd_workspace(x.shape[0], N, x.shape[1]), workspace, dev)
    keep, d = _describe_all([x, g, w, initial_state, cu_seqlens, out, final_state])
    _launch(dev, lambda stream: lib.gdn2_linear_scan_fwd(*d, ctypes.addressof(opts), *_ws_args(ws), stream))
    return out, final_state


def linear_scan_recurrent_fwd(x, g, w=None, initial_state=None, cu_seqlens=None, output_final_state=True,
                              input_scale="none", out=None, final_state=None):
    """:func:`linear_scan_fwd` evaluated token by token (decode and short
    spans). ``final_state`` may be ``initial_state`` itself to update the
    state in place."""
    lib = load_library()
    opts = _scan_options(input_scale)
    dev, _, out, final_state = _scan_outputs(x, g, w, initial_state, cu_seqlens, output_final_state, out, final_state)
    keep, d = _describe_all([x, g, w, initial_state, cu_seqlens, out, final_state])
    _launch(dev, lambda stream: lib.gdn2_linear_scan_recurrent_fwd(*d, ctypes.addressof(opts), stream))
    return out, final_state


def linear_scan_bwd(x, g, w, d_out, initial_state=None, cu_seqlens=None, d_final_state=None, need_d_initial_state=True,
                    input_scale="none", grads=None, workspace=None):
    """Backward of :func:`linear_scan_fwd`: a dict with dx, dw (None without
    w) in x's type, dg in g's and d_initial_state (float32 [N, D], or None
    when not requested). d_final_state: float32 or None (zero). Tensors given
    in ``grads`` are written in place. ``workspace``: at least
    ``linear_scan_bwd_workspace(T, N, D)`` bytes."""
    lib = load_library()
    opts = _scan_options(input_scale)
    out = dict(grads or {})
    ins = [x, g, w, initial_state, cu_seqlens, d_out, d_final_state]
    dev = _one_device(_SCAN_NAMES[:5] + ("d_out", "d_final_state") + SCAN_GRADS, ins + [out.get(n) for n in SCAN_GRADS])
    _rank2(x=x, g=g)
    N = _sequences(cu_seqlens)
    for n, t in (("dx", x), ("dg", g), ("dw", w)):
        if out.get(n) is None:
            out[n] = None if t is None else _like(t)
    if out.get("d_initial_state") is None:
        need = need_d_initial_state and N >= 1
        out["d_initial_state"] = torch.empty((N, x.shape[1]), dtype=torch.float32, device=dev) if need else None
    ws = _workspace(lib.gdn2_linear_scan_bwd_workspace(x.shape[0], N, x.shape[1]), workspace, dev)
    keep, d = _describe_all(ins + [out[n] for n in SCAN_GRADS])
    _launch(dev, lambda stream: lib.gdn2_linear_scan_bwd(*d, ctypes.addressof(opts), *_ws_args(ws), stream))
    return out


def check_linear_scan(x, g, w=None, initial_state=None, cu_seqlens=None, out=None, final_state=None, input_scale="none",
                      recurrent=False):
    """The library's host-side validation of a :func:`linear_scan_fwd` or
    (``recurrent``) :func:`linear_scan_recurrent_fwd` call only (no GPU
    needed): the status code."""
    lib = load_library()
    keep, d = _describe_all([x, g, w, initial_state, cu_seqlens, out, final_state])
    fn = lib.gdn2_linear_scan_recurrent_fwd_check if recurrent else lib.gdn2_linear_scan_fwd_check
    return fn(*d, ctypes.addressof(_scan_options(input_scale)))


def check_linear_scan_bwd(x, g, w, d_out, initial_state=None, cu_seqlens=None, d_final_state=None, input_scale="none",
                          grads=None):
    """The library's host-side validation of a :func:`linear_scan_bwd` call only (no GPU needed)."""
    gr = grads or {}
    keep, d = _describe_all([x, g, w, initial_state, cu_seqlens, d_out, d_final_state] + [gr.get(n) for n in SCAN_GRADS])
    return load_library().gdn2_linear_scan_bwd_check(*d, ctypes.addressof(_scan_options(input_scale)))


_CONV_NAMES = ("x", "weight", "bias", "initial_state", "cu_seqlens", "out", "final_state")
CONV_GRADS = ("dx", "dweight", "dbias", "d_initial_state")


def _conv_outputs(x, weight, bias, initial_state, cu_seqlens, output_final_state, out, final_state):
    dev = _one_device(_CONV_NAMES, (x, weight, bias, initial_state, cu_seqlens, out, final_state))
    _rank2(x=x, weight=weight)
    N = _sequences(cu_seqlens)
    if out is None:
        out = _like(x)
    if final_state is None and output_final_state and N >= 1 and weight.shape[1] >= 1:
        final_state = torch.empty((N, weight.shape[1] - 1, x.shape[1]), dtype=x.dtype, device=dev)
    return dev, out, final_state


def short_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, output_final_state=True, activation="silu",
                   out=None, final_state=None):
    """The short causal convolution per channel, on the current HIP stream:
    p_t = bias + sum_j weight[:, j] x_{t - (K - 1) + j} over each sequence,
    out = p ("none") or p sigmoid(p) (``activation`` "silu").

    x, out [T, D]: bf16, float16 or float32, rows with any token stride;
    weight [D, K] (K 2 to 4) and bias [D]: float32 or x's type; states
    [N, K - 1, D] in x's type: the inputs before the first token, the oldest
    first (None: zeros), and the last K - 1 inputs; cu_seqlens as in
    :func:`chunk_fwd`. Returns (out, final_state or None).
    """
    lib = load_library()
    opts = _conv_options(activation)
    dev, out, final_state = _conv_outputs(x, weight, bias, initial_state, cu_seqlens, output_final_state, out, final_state)
    keep, d = _describe_all([x, weight, bias, initial_state, cu_seqlens, out, final_state])
    _launch(dev, lambda stream: lib.gdn2_short_conv_fwd(*d, ctypes.addressof(opts), stream))
    return out, final_state


def short_conv_recurrent_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, output_final_state=True,
                             activation="silu", out=None, final_state=None):
    """:func:`short_conv_fwd` evaluated token by token (decode and short
    spans). ``final_state`` may be ``initial_state`` itself to update the
    state in place."""
    lib = load_library()
    opts = _conv_options(activation)
    dev, out, final_state = _conv_outputs(x, weight, bias, initial_state, cu_seqlens, output_final_state, out, final_state)
    keep, d = _describe_all([x, weight, bias, initial_state, cu_seqlens, out, final_state])
    _launch(dev, lambda stream: lib.gdn2_short_conv_recurrent_fwd(*d, ctypes.addressof(opts), stream))
    return out, final_state


def short_conv_bwd_workspace(T, D, K):
    """Bytes of workspace of :func:`short_conv_bwd`."""
    return load_library().gdn2_short_conv_bwd_workspace(int(T), int(D), int(K))


def short_conv_bwd(x, weight, bias, d_out, initial_state=None, cu_seqlens=None, d_final_state=None,
                   need_d_initial_state=True, activation="silu", grads=None, workspace=None):
    """Backward of :func:`short_conv_fwd`: a dict with dx and d_initial_state
    (x's type; the second None when not requested), dweight and dbias (the
    weight's type, dbias None without bias). Tensors given in ``grads`` are
    written in place. ``workspace``: at least ``short_conv_bwd_workspace(T, D,
    K)`` bytes."""
    lib = load_library()
    opts = _conv_options(activation)
    out = dict(grads or {})
    ins = [x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state]
    dev = _one_device(_CONV_NAMES[:5] + ("d_out", "d_final_state") + CONV_GRADS, ins + [out.get(n) for n in CONV_GRADS])
    _rank2(x=x, weight=weight)
    N, (T, D), K = _sequences(cu_seqlens), x.shape, weight.shape[1]
    for n, t in (("dx", x), ("dweight", weight), ("dbias", bias)):
        if out.get(n) is None:
            out[n] = None if t is None else _like(t)
    if out.get("d_initial_state") is None:
        need = need_d_initial_state and N >= 1 and K >= 1
        out["d_initial_state"] = torch.empty((N, K - 1, D), dtype=x.dtype, device=dev) if need else None
    ws = _workspace(lib.gdn2_short_conv_bwd_workspace(T, D, K), workspace, dev)
    keep, d = _describe_all(ins + [out[n] for n in CONV_GRADS])
    _launch(dev, lambda stream: lib.gdn2_short_conv_bwd(*d, ctypes.addressof(opts), *_ws_args(ws), stream))
    return out


def check_short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, out=None, final_state=None,
                     activation="silu", recurrent=False):
    """The library's host-side validation of a :func:`short_conv_fwd` or
    (``recurrent``) :func:`short_conv_recurrent_fwd` call only (no GPU
    needed): the status code."""
    lib = load_library()
    keep, d = _describe_all([x, weight, bias, initial_state, cu_seqlens, out, final_state])
    fn = lib.gdn2_short_conv_recurrent_fwd_check if recurrent else lib.gdn2_short_conv_fwd_check
    return fn(*d, ctypes.addressof(_conv_options(activation)))


def check_short_conv_bwd(x, weight, bias, d_out, initial_state=None, cu_seqlens=None, d_final_state=None,
                         activation="silu", grads=None):
    """The library's host-side validation of a :func:`short_conv_bwd` call only (no GPU needed)."""
    gr = grads or {}
    keep, d = _describe_all([x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state]
                            + [gr.get(n) for n in CONV_GRADS])
    return load_library().gdn2_short_conv_bwd_check(*d, ctypes.addressof(_conv_options(activation)))


_NORM_NAMES = ("x", "gate", "weight", "bias", "out")
NORM_GRADS = ("dx", "dgate", "dweight", "dbias")


def _rows3(t):
    """A tensor of rows [T, D] as one head's, [T, 1, D]."""
    return t.unsqueeze(1) if t is not None and t.dim() == 2 else t


def _norm_rank(x):
    if x.dim() not in (2, 3):
        raise ValueError(f"x must have 2 or 3 dimensions, not {x.dim()}")


def layer_norm(x, weight=None, bias=None, gate=None, norm="layer", eps=None, out=None):
    """The norm of rows, on the current HIP stream: ``norm`` "layer" ((x -
    mean) / sqrt(var + eps), eps 1e-5) or "rms" (x / sqrt(mean x^2 + eps), eps
    1e-6), times weight, plus bias, times gate sigmoid(gate). ``eps`` None or
    0: these values.

    x, gate, out [T, H, D] or [T, D] (D up to 16384): bf16, float16 or
    float32, strided rows accepted; weight, bias [D]: float32 or x's type.
    Returns out.
    """
    lib = load_library()
    opts = _norm_options(norm, eps)
    dev = _one_device(_NORM_NAMES, (x, gate, weight, bias, out))
    _norm_rank(x)
    if out is None:
        out = _like(x)
    keep, d = _describe_all([_rows3(x), _rows3(gate), weight, bias, _rows3(out)])
    _launch(dev, lambda stream: lib.gdn2_layer_norm_fwd(*d, ctypes.addressof(opts), stream))
    return out


def layer_norm_bwd_workspace(T, H, D):
    """Bytes of workspace of :func:`layer_norm_bwd` with a weight's or bias's gradient."""
    return load_library().gdn2_layer_norm_bwd_workspace(int(T), int(H), int(D))


def layer_norm_bwd(x, d_out, weight=None, bias=None, gate=None, norm="layer", eps=None, grads=None, workspace=None):
    """Backward of :func:`layer_norm`: a dict with dx, dgate (x's shape and
    type), dweight and dbias (their tensors' types), None for an argument that
    is None. Tensors given in ``grads`` are written in place. ``workspace``:
    at least ``layer_norm_bwd_workspace(T, H, D)`` bytes."""
    lib = load_library()
    opts = _norm_options(norm, eps)
    out = dict(grads or {})
    dev = _one_device(("x", "gate", "weight", "bias", "d_out") + NORM_GRADS,
                      [x, gate, weight, bias, d_out] + [out.get(n) for n in NORM_GRADS])
    _norm_rank(x)
    for n, t in (("dx", x), ("dgate", gate), ("dweight", weight), ("dbias", bias)):
        if out.get(n) is None:
            out[n] = None if t is None else _like(t)
    sums = out["dweight"] is not None or out["dbias"] is not None
    heads = 1 if x.dim() == 2 else x.shape[1]
    ws = _workspace(lib.gdn2_layer_norm_bwd_workspace(x.shape[0], heads, x.shape[-1]) if sums else 0, workspace, dev)
    keep, d = _describe_all([_rows3(x), _rows3(gate), weight, bias, _rows3(d_out), _rows3(out["dx"]), _rows3(out["dgate"]),
                             out["dweight"], out["dbias"]])
    _launch(dev, lambda stream: lib.gdn2_layer_norm_bwd(*d, ctypes.addressof(opts), *_ws_args(ws), stream))
    return out


def check_layer_norm(x, weight=None, bias=None, gate=None, norm="layer", eps=None, out=None):
    """The library's host-side validation of a :func:`layer_norm` call only (no GPU needed)."""
    keep, d = _describe_all([_rows3(x), _rows3(gate), weight, bias, _rows3(out)])
    return load_library().gdn2_layer_norm_fwd_check(*d, ctypes.addressof(_norm_options(norm, eps)))


def check_layer_norm_bwd(x, d_out, weight=None, bias=None, gate=None, norm="layer", eps=None, grads=None):
    """The library's host-side validation of a :func:`layer_norm_bwd` call only (no GPU needed)."""
    g = grads or {}
    keep, d = _describe_all([_rows3(x), _rows3(gate), weight, bias, _rows3(d_out), _rows3(g.get("dx")),
                             _rows3(g.get("dgate")), g.get("dweight"), g.get("dbias")])
    return load_library().gdn2_layer_norm_bwd_check(*d, ctypes.addressof(_norm_options(norm, eps)))
