"""ctypes binding of libkda.so — argument marshalling only.

Every function here has the name of the C entry point it calls (``include/kda.h``)
and takes torch tensors that live on the GPU; each one checks shapes, dtypes and
contiguity, passes raw device pointers and the current CUDA stream, and raises
:class:`KdaError` on a non-OK status.  With ``stream=`` a call runs on that stream, its inputs must be
ready there, and what it allocates comes out of that stream's memory; the caller orders the
streams before it reads the results on another.  The calls whose kernels take a few microseconds go
through the ``_calls`` extension (``csrc/calls.cpp``), which does the same for well-formed arguments in
C++; every other argument comes back here to be named in an error, and all of them do, with a warning at
import, where it was not built.  All computation happens in the library's
CUDA kernels.  There is no fallback: if ``libkda.so`` is missing or fails to load,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import warnings

import torch

from gated_delta_rule_155_b200 import build

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")

KDA_OK = 0
KDA_F32, KDA_BF16 = 0, 1
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED",
                3: "KDA_ERR_MISALIGNED", 4: "KDA_ERR_CUDA", 5: "KDA_ERR_TIMEOUT",
                6: "KDA_ERR_WORKSPACE", 7: "KDA_ERR_INDEX"}


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.kda_status_string(status).decode() if _lib is not None else "?"
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({msg})")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"libkda.so not found at {_LIB_PATH}; build it with "
            "`python -m gated_delta_rule_155_b200.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [i]
    lib.kda_abi_version.restype = i
    lib.kda_forward_chunked.restype = i
    lib.kda_forward_chunked.argtypes = [vp] * 8 + [i] * 6 + [i, vp]
    lib.kda_decode_step.restype = i
    lib.kda_decode_step.argtypes = [vp] * 7 + [i] * 4 + [i, vp]
    lib.kda_layer_forward_varlen.restype = i
    lib.kda_layer_forward_varlen.argtypes = [vp] * 9 + [f] + [vp] * 3 + [f] + [vp] * 5 + [sz] + [i] * 5 + [i, vp]
    lib.kda_backward_workspace_size.restype = i
    lib.kda_backward_workspace_size.argtypes = [i] * 6 + [ctypes.POINTER(sz)]
    lib.kda_backward_chunked.restype = i
    lib.kda_backward_chunked.argtypes = [vp] * 15 + [sz] + [i] * 5 + [i, vp]
    lib.kda_forward_chunked_varlen.restype = i
    lib.kda_forward_chunked_varlen.argtypes = [vp] * 9 + [i] * 6 + [i, vp]
    lib.kda_layer_workspace_size.restype = i
    lib.kda_layer_workspace_size.argtypes = [i] * 6 + [ctypes.POINTER(sz)]
    lib.kda_layer_forward.restype = i
    lib.kda_layer_forward.argtypes = [vp] * 9 + [f] + [vp] * 3 + [f] + [vp] * 4 + [sz] + [i] * 5 + [i, vp]
    lib.kda_layer_forward_noalloc.restype = i
    lib.kda_layer_forward_noalloc.argtypes = [vp] * 9 + [f] + [vp] * 3 + [f] + [vp] * 3 + [i] * 5 + [i, vp]
    lib.kda_check_device_error.restype = i
    lib.kda_layer_decode_step.argtypes = [vp] * 12 + [f] + [vp] * 3 + [f] + [vp] * 2 + [i] * 4 + [i, vp]
    lib.kda_layer_decode_step.restype = i
    lib.kda_check_device_error.argtypes = [vp]
    lib.kda_gdr_workspace_size.restype = i
    lib.kda_gdr_workspace_size.argtypes = [i] * 8 + [ctypes.POINTER(sz)]
    lib.kda_gdr_forward.restype = i
    lib.kda_gdr_forward.argtypes = [vp] * 10 + [i] + [vp] * 2 + [sz] + [i] * 6 + [i, vp]
    lib.kda_gdr_backward.restype = i
    lib.kda_gdr_backward.argtypes = [vp] * 16 + [sz] + [i] * 6 + [i, vp]
    lib.kda_gdr_decode.restype = i
    lib.kda_gdr_decode.argtypes = [vp] * 7 + [i, vp] + [i] * 6 + [i, vp]
    lib.kda_pages_fork.restype = i
    lib.kda_pages_fork.argtypes = [vp, sz, i, i, vp, vp, vp, i, vp]
    lib.kda_pages_copy.restype = i
    lib.kda_pages_copy.argtypes = [vp, sz, i, i, vp, vp, i, vp]
    lib.kda_pages_free.restype = i
    lib.kda_pages_free.argtypes = [vp, i, vp, i, vp]
    lib.kda_pages_workspace_size.restype = i
    lib.kda_pages_workspace_size.argtypes = [i, ctypes.POINTER(sz)]
    lib.kda_pages_compact.restype = i
    lib.kda_pages_compact.argtypes = [vp, sz, i, i, vp, vp, i, vp, vp, sz, vp]
    lib.kda_set_wait_test_hooks.restype = i
    lib.kda_set_wait_test_hooks.argtypes = [ctypes.c_ulonglong, i]
    return lib


_lib = _load()


class _NoCalls:
    """In place of the short calls where they were not built: takes no call."""

    def __getattr__(self, name):
        return lambda *a: None


def _load_calls():
    path = build.calls_path()
    try:
        if not os.path.exists(path):
            raise ImportError(f"{os.path.basename(path)} not found")
        spec = importlib.util.spec_from_file_location(f"{__package__}._calls", path)
        _calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_calls)
    except ImportError as e:
        warnings.warn(f"the _calls extension does not load ({e}): short calls are marshalled in Python, 10 to 20 us each; build it with "
                      "`python -m gated_delta_rule_155_b200.build`", RuntimeWarning, stacklevel=3)
        return _NoCalls()
    names = ("kda_gdr_decode", "kda_gdr_workspace_size", "kda_gdr_forward", "kda_gdr_backward", "kda_pages_fork",
             "kda_pages_free", "kda_pages_workspace_size", "kda_pages_compact")
    _calls.init(*(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in names))
    return _calls


# The calls whose kernels take a few microseconds, in C++: None where an argument is not well-formed (the
# Python function then checks them one by one and raises), a status where the library refuses.  Only marshalling:
# without them the Python functions make the same calls of the library.
_calls = _load_calls()

EXPORTED_SYMBOLS = ("kda_status_string", "kda_abi_version", "kda_forward_chunked",
                    "kda_decode_step", "kda_layer_workspace_size", "kda_layer_forward",
                    "kda_layer_forward_noalloc", "kda_layer_decode_step", "kda_forward_chunked_varlen",
                    "kda_backward_workspace_size", "kda_backward_chunked", "kda_layer_forward_varlen",
                    "kda_gdr_workspace_size", "kda_gdr_forward", "kda_gdr_backward", "kda_gdr_decode",
                    "kda_pages_fork", "kda_pages_copy", "kda_pages_free", "kda_pages_workspace_size",
                    "kda_pages_compact", "kda_check_device_error", "kda_set_wait_test_hooks")

NOALLOC_SCRATCH_BYTES = 64 << 20  # KDA_NOALLOC_SCRATCH_BYTES


def library():
    """The loaded ctypes library handle."""
    return _lib


_Tensor, _empty = torch.Tensor, torch.empty
_cuda_getDevice, _cuda_getCurrentRawStream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


# The marshalling runs before every launch, and a decode kernel takes 4 us: raw pointers as ints (what the
# argument types convert), the device and stream of torch's C side, and one look at a well-formed tensor.
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return _cuda_getCurrentRawStream(_cuda_getDevice())
    return stream.cuda_stream


_IO_CODES = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}


def _io_code(dtype):
    code = _IO_CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported io dtype {dtype}")
    return code


def _taken(r, where):
    if r.__class__ is int:
        raise KdaError(r, where)
    return r


def _torch_stream(stream):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream)


def _new(stream, make, *args, **kw):
    """make(*args, **kw), which a call on `stream` writes and the caller gets.  Out of that stream's memory: a block of
    the current stream's may have a last user that still runs there, and nothing orders `stream` behind it.  The
    caller may drop it while the current stream works on it, so it is kept until that is over."""
    if stream is None:
        return make(*args, **kw)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(_torch_stream(stream)):
        t = make(*args, **kw)
    t.record_stream(current)
    return t


def _workspace(stream, need, device):
    """A workspace of `need` bytes for a call on `stream`, out of that stream's memory (as _new); no other uses it."""
    if need == 0:
        return None
    if stream is None:
        return _empty(need, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_torch_stream(stream)):
        return _empty(need, dtype=torch.uint8, device=device)


def _on(stream, *tensors):
    """What the caller gave, allocated on another stream perhaps, is kept until its use on `stream` is over."""
    if stream is not None:
        stream = _torch_stream(stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _check(status, where):
    if status != KDA_OK:
        raise KdaError(status, where)


def _need(t, shape, dtype, name, *, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    # the library launches on the current device, so every tensor must live there
    cur = torch.cuda.current_device()
    if t.device.index is not None and t.device.index != cur:
        raise ValueError(f"{name} is on cuda:{t.device.index} but the current device is cuda:{cur}; "
                         f"call under torch.cuda.device({t.device.index})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_all(checks):
    """_need for each (tensor, shape, dtype, name), with one look at those that are well-formed."""
    cur = _cuda_getDevice()
    for t, shape, dtype, name in checks:
        if not (t.__class__ is _Tensor and t.shape == shape and t.dtype is dtype and t.is_contiguous()
                and t.get_device() == cur):
            _need(t, shape, dtype, name)


def kda_forward_chunked(q, k, v, g, beta, initial_state=None, out=None, final_state=None,
                        *, chunk=64, stream=None):
    """Chunked prefill.  q, k, g: [B, T, H, dk]; v: [B, T, H, dv]; beta: [B, T, H] (io dtype);
    initial_state / final_state: [B, H, dk, dv] fp32 or None.  Returns (out, final_state)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    io = q.dtype
    for t, s, n in ((q, (B, T, H, dk), "q"), (k, (B, T, H, dk), "k"), (g, (B, T, H, dk), "g"),
                    (v, (B, T, H, dv), "v"), (beta, (B, T, H), "beta")):
        _need(t, s, io, n)
    _need(initial_state, (B, H, dk, dv), torch.float32, "initial_state", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (B, T, H, dv), dtype=io, device=q.device)
    _need(out, (B, T, H, dv), io, "out")
    _need(final_state, (B, H, dk, dv), torch.float32, "final_state", allow_none=True)
    _check(_lib.kda_forward_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                    _ptr(initial_state), _ptr(out), _ptr(final_state),
                                    B, T, H, dk, dv, chunk, _io_code(io), _stream(stream)),
           "kda_forward_chunked")
    return out, final_state


def kda_forward_chunked_varlen(q, k, v, g, beta, cu_seqlens, initial_state=None, out=None,
                               final_state=None, *, chunk=64, stream=None):
    """Chunked prefill of N packed sequences.  q, k, g: [T_total, H, dk]; v: [T_total, H, dv];
    beta: [T_total, H] (io dtype); cu_seqlens: int32 CUDA tensor [N + 1] of sequence offsets
    (0 .. T_total, non-decreasing); initial_state / final_state: [N, H, dk, dv] fp32 or None.
    Returns (out [T_total, H, dv], final_state)."""
    Tt, H, dk = q.shape
    dv = v.shape[-1]
    io = q.dtype
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
    N = cu_seqlens.numel() - 1
    _need(cu_seqlens, (N + 1,), torch.int32, "cu_seqlens")
    for t, s, n in ((q, (Tt, H, dk), "q"), (k, (Tt, H, dk), "k"), (g, (Tt, H, dk), "g"),
                    (v, (Tt, H, dv), "v"), (beta, (Tt, H), "beta")):
        _need(t, s, io, n)
    _need(initial_state, (N, H, dk, dv), torch.float32, "initial_state", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (Tt, H, dv), dtype=io, device=q.device)
    _need(out, (Tt, H, dv), io, "out")
    _need(final_state, (N, H, dk, dv), torch.float32, "final_state", allow_none=True)
    _check(_lib.kda_forward_chunked_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                           _ptr(initial_state), _ptr(out), _ptr(final_state),
                                           _ptr(cu_seqlens), N, Tt, H, dk, dv, chunk, _io_code(io),
                                           _stream(stream)),
           "kda_forward_chunked_varlen")
    return out, final_state


def kda_backward_workspace_size(B, T, H, dk, dv, dtype):
    n = ctypes.c_size_t(0)
    _check(_lib.kda_backward_workspace_size(B, T, H, dk, dv, _io_code(dtype), ctypes.byref(n)),
           "kda_backward_workspace_size")
    return int(n.value)


def kda_backward_chunked(q, k, v, g, beta, d_out, initial_state=None, d_final_state=None, *,
                         grads=None, d_initial_state=None, workspace=None, stream=None):
    """Gradients of kda_forward_chunked.  Returns dict dq, dk, dv, dg, dbeta (io dtype) and
    d_initial_state (fp32 [B, H, dk, dv]).  ``grads`` may hold preallocated outputs;
    ``workspace`` (uint8 CUDA tensor) is allocated with torch when not given."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    io = q.dtype
    for t, s, n in ((q, (B, T, H, dk), "q"), (k, (B, T, H, dk), "k"), (g, (B, T, H, dk), "g"),
                    (v, (B, T, H, dv), "v"), (beta, (B, T, H), "beta"), (d_out, (B, T, H, dv), "d_out")):
        _need(t, s, io, n)
    _need(initial_state, (B, H, dk, dv), torch.float32, "initial_state", allow_none=True)
    _need(d_final_state, (B, H, dk, dv), torch.float32, "d_final_state", allow_none=True)
    gr = dict(grads or {})
    shapes = {"dq": (B, T, H, dk), "dk": (B, T, H, dk), "dg": (B, T, H, dk), "dv": (B, T, H, dv),
              "dbeta": (B, T, H)}
    for n, s in shapes.items():
        if gr.get(n) is None:
            gr[n] = _new(stream, torch.empty, s, dtype=io, device=q.device)
        _need(gr[n], s, io, n)
    if d_initial_state is None:
        d_initial_state = _new(stream, torch.empty, (B, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(d_initial_state, (B, H, dk, dv), torch.float32, "d_initial_state")
    need = kda_backward_workspace_size(B, T, H, dk, dv, io)
    if workspace is None:
        workspace = _workspace(stream, need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.kda_backward_chunked(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(d_out), _ptr(d_final_state),
        _ptr(gr["dq"]), _ptr(gr["dk"]), _ptr(gr["dv"]), _ptr(gr["dg"]), _ptr(gr["dbeta"]), _ptr(d_initial_state),
        _ptr(workspace), ws_bytes, B, T, H, dk, dv, _io_code(io), _stream(stream)), "kda_backward_chunked")
    gr["d_initial_state"] = d_initial_state
    return gr


def kda_decode_step(q, k, v, g, beta, state, out=None, *, stream=None):
    """One decode step; ``state`` [B, H, dk, dv] fp32 is updated in place.  Returns out [B, H, dv]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    io = q.dtype
    for t, s, n in ((q, (B, H, dk), "q"), (k, (B, H, dk), "k"), (g, (B, H, dk), "g"),
                    (v, (B, H, dv), "v"), (beta, (B, H), "beta")):
        _need(t, s, io, n)
    _need(state, (B, H, dk, dv), torch.float32, "state")
    if out is None:
        out = _new(stream, torch.empty, (B, H, dv), dtype=io, device=q.device)
    _need(out, (B, H, dv), io, "out")
    _check(_lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                _ptr(out), B, H, dk, dv, _io_code(io), _stream(stream)),
           "kda_decode_step")
    return out


def _lb(bound):
    """The gate's lower bound as the C ABI takes it: -inf for none."""
    return float("-inf") if bound is None else float(bound)


def kda_layer_workspace_size(B, T, H, dk, dv, dtype):
    n = ctypes.c_size_t(0)
    _check(_lib.kda_layer_workspace_size(B, T, H, dk, dv, _io_code(dtype), ctypes.byref(n)),
           "kda_layer_workspace_size")
    return int(n.value)


def kda_layer_forward(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, g_raw, A_log, dt_bias, b_raw,
                      o_gate_raw, o_norm_w=None, *, norm_eps=1e-6, initial_state=None, out=None,
                      final_state=None, workspace=None, gate_lower_bound=None, stream=None):
    """KDA layer core (prologue -> chunked gated delta rule -> epilogue).  Returns (out, final_state).
    ``workspace`` (a uint8 CUDA tensor) is allocated with torch when not given.
    ``gate_lower_bound`` (<= 0, e.g. -5.0) bounds every log-decay g from below; None: unbounded."""
    B, T, H, dk = g_raw.shape
    dv = o_gate_raw.shape[-1]
    io = g_raw.dtype
    f32 = torch.float32
    for t, s, d, n in ((q_raw, (B, T, H * dk), io, "q_raw"), (k_raw, (B, T, H * dk), io, "k_raw"),
                       (v_raw, (B, T, H * dv), io, "v_raw"), (b_raw, (B, T, H), io, "b_raw"),
                       (o_gate_raw, (B, T, H, dv), io, "o_gate_raw"),
                       (conv_q, (H * dk, 4), f32, "conv_q"), (conv_k, (H * dk, 4), f32, "conv_k"),
                       (conv_v, (H * dv, 4), f32, "conv_v"), (A_log, (H,), f32, "A_log")):
        _need(t, s, d, n)
    _need(dt_bias, (H * dk,), f32, "dt_bias", allow_none=True)
    _need(o_norm_w, (dv,), f32, "o_norm_w", allow_none=True)
    _need(initial_state, (B, H, dk, dv), f32, "initial_state", allow_none=True)
    _need(final_state, (B, H, dk, dv), f32, "final_state", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (B, T, H, dv), dtype=io, device=g_raw.device)
    _need(out, (B, T, H, dv), io, "out")
    need = kda_layer_workspace_size(B, T, H, dk, dv, io)
    if workspace is None:
        workspace = _workspace(stream, need, g_raw.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.kda_layer_forward(
        _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
        _ptr(g_raw), _ptr(A_log), _ptr(dt_bias), _lb(gate_lower_bound), _ptr(b_raw), _ptr(o_gate_raw),
        _ptr(o_norm_w), float(norm_eps), _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(workspace),
        ws_bytes, B, T, H, dk, dv, _io_code(io), _stream(stream)), "kda_layer_forward")
    return out, final_state


def kda_layer_forward_varlen(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, g_raw, A_log, dt_bias, b_raw,
                             o_gate_raw, cu_seqlens, o_norm_w=None, *, norm_eps=1e-6, initial_state=None,
                             out=None, final_state=None, workspace=None, gate_lower_bound=None, stream=None):
    """The layer core over N packed sequences.  q_raw, k_raw: [T_total, H*dk]; v_raw: [T_total, H*dv];
    g_raw: [T_total, H, dk]; b_raw: [T_total, H]; o_gate_raw: [T_total, H, dv]; cu_seqlens: int32 CUDA
    [N + 1]; states [N, H, dk, dv].  Returns (out [T_total, H, dv], final_state)."""
    Tt, H, dk = g_raw.shape
    dv = o_gate_raw.shape[-1]
    io = g_raw.dtype
    f32 = torch.float32
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
    N = cu_seqlens.numel() - 1
    _need(cu_seqlens, (N + 1,), torch.int32, "cu_seqlens")
    for t, s, d, n in ((q_raw, (Tt, H * dk), io, "q_raw"), (k_raw, (Tt, H * dk), io, "k_raw"),
                       (v_raw, (Tt, H * dv), io, "v_raw"), (b_raw, (Tt, H), io, "b_raw"),
                       (o_gate_raw, (Tt, H, dv), io, "o_gate_raw"),
                       (conv_q, (H * dk, 4), f32, "conv_q"), (conv_k, (H * dk, 4), f32, "conv_k"),
                       (conv_v, (H * dv, 4), f32, "conv_v"), (A_log, (H,), f32, "A_log")):
        _need(t, s, d, n)
    _need(dt_bias, (H * dk,), f32, "dt_bias", allow_none=True)
    _need(o_norm_w, (dv,), f32, "o_norm_w", allow_none=True)
    _need(initial_state, (N, H, dk, dv), f32, "initial_state", allow_none=True)
    _need(final_state, (N, H, dk, dv), f32, "final_state", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (Tt, H, dv), dtype=io, device=g_raw.device)
    _need(out, (Tt, H, dv), io, "out")
    need = kda_layer_workspace_size(1, Tt, H, dk, dv, io)
    if workspace is None:
        workspace = _workspace(stream, need, g_raw.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.kda_layer_forward_varlen(
        _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
        _ptr(g_raw), _ptr(A_log), _ptr(dt_bias), _lb(gate_lower_bound), _ptr(b_raw), _ptr(o_gate_raw),
        _ptr(o_norm_w), float(norm_eps), _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(cu_seqlens),
        _ptr(workspace), ws_bytes, N, Tt, H, dk, dv, _io_code(io), _stream(stream)), "kda_layer_forward_varlen")
    return out, final_state


def kda_layer_decode_step(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, cache_q, cache_k, cache_v, g_raw,
                          A_log, dt_bias, b_raw, o_gate_raw, state, o_norm_w=None, *, norm_eps=1e-6,
                          out=None, gate_lower_bound=None, stream=None):
    """One decode step of the layer core.  ``cache_*`` [B, 3, H*d] (io dtype, oldest tap first)
    and ``state`` [B, H, dk, dv] fp32 are updated in place.  Returns out [B, H, dv]."""
    B, H, dk = g_raw.shape
    dv = o_gate_raw.shape[-1]
    io = g_raw.dtype
    f32 = torch.float32
    for t, s_, d, n in ((q_raw, (B, H * dk), io, "q_raw"), (k_raw, (B, H * dk), io, "k_raw"),
                        (v_raw, (B, H * dv), io, "v_raw"), (b_raw, (B, H), io, "b_raw"),
                        (o_gate_raw, (B, H, dv), io, "o_gate_raw"),
                        (cache_q, (B, 3, H * dk), io, "cache_q"), (cache_k, (B, 3, H * dk), io, "cache_k"),
                        (cache_v, (B, 3, H * dv), io, "cache_v"),
                        (conv_q, (H * dk, 4), f32, "conv_q"), (conv_k, (H * dk, 4), f32, "conv_k"),
                        (conv_v, (H * dv, 4), f32, "conv_v"), (A_log, (H,), f32, "A_log"),
                        (state, (B, H, dk, dv), f32, "state")):
        _need(t, s_, d, n)
    _need(dt_bias, (H * dk,), f32, "dt_bias", allow_none=True)
    _need(o_norm_w, (dv,), f32, "o_norm_w", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (B, H, dv), dtype=io, device=g_raw.device)
    _need(out, (B, H, dv), io, "out")
    _check(_lib.kda_layer_decode_step(
        _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
        _ptr(cache_q), _ptr(cache_k), _ptr(cache_v), _ptr(g_raw), _ptr(A_log), _ptr(dt_bias),
        _lb(gate_lower_bound), _ptr(b_raw), _ptr(o_gate_raw), _ptr(o_norm_w), float(norm_eps), _ptr(state), _ptr(out),
        B, H, dk, dv, _io_code(io), _stream(stream)), "kda_layer_decode_step")
    return out


def kda_layer_forward_noalloc(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, g_raw, A_log, dt_bias,
                              b_raw, o_gate_raw, o_norm_w=None, *, norm_eps=1e-6, initial_state=None,
                              out=None, final_state=None, gate_lower_bound=None, stream=None):
    """kda_layer_forward with its scratch in the library's own fixed device buffer (no
    workspace argument, no allocation inside the call except ``out`` when it is not given —
    pass ``out`` to allocate nothing at all).  Sizes needing more than NOALLOC_SCRATCH_BYTES
    of scratch raise KdaError (KDA_ERR_WORKSPACE).  Returns (out, final_state)."""
    B, T, H, dk = g_raw.shape
    dv = o_gate_raw.shape[-1]
    io = g_raw.dtype
    f32 = torch.float32
    for t, s, d, n in ((q_raw, (B, T, H * dk), io, "q_raw"), (k_raw, (B, T, H * dk), io, "k_raw"),
                       (v_raw, (B, T, H * dv), io, "v_raw"), (b_raw, (B, T, H), io, "b_raw"),
                       (o_gate_raw, (B, T, H, dv), io, "o_gate_raw"),
                       (conv_q, (H * dk, 4), f32, "conv_q"), (conv_k, (H * dk, 4), f32, "conv_k"),
                       (conv_v, (H * dv, 4), f32, "conv_v"), (A_log, (H,), f32, "A_log")):
        _need(t, s, d, n)
    _need(dt_bias, (H * dk,), f32, "dt_bias", allow_none=True)
    _need(o_norm_w, (dv,), f32, "o_norm_w", allow_none=True)
    _need(initial_state, (B, H, dk, dv), f32, "initial_state", allow_none=True)
    _need(final_state, (B, H, dk, dv), f32, "final_state", allow_none=True)
    if out is None:
        out = _new(stream, torch.empty, (B, T, H, dv), dtype=io, device=g_raw.device)
    _need(out, (B, T, H, dv), io, "out")
    _check(_lib.kda_layer_forward_noalloc(
        _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
        _ptr(g_raw), _ptr(A_log), _ptr(dt_bias), _lb(gate_lower_bound), _ptr(b_raw), _ptr(o_gate_raw),
        _ptr(o_norm_w), float(norm_eps), _ptr(initial_state), _ptr(out), _ptr(final_state),
        B, T, H, dk, dv, _io_code(io), _stream(stream)), "kda_layer_forward_noalloc")
    return out, final_state


def _gdr_shapes(q, k, v, g, beta, cu_seqlens):
    """(N, T_total, Hk, Hv, dk, dv, leading shape) of the head-gated delta rule's inputs: packed
    [T_total, ...] with cu_seqlens, [B, T, ...] without."""
    sq, sv, io = q.shape, v.shape, q.dtype
    if cu_seqlens is not None:
        sc = cu_seqlens.shape
        if len(sc) != 1 or sc[0] < 2:
            raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
        if len(sq) != 3 or len(sv) != 3:
            raise ValueError("with cu_seqlens, q and v are [T_total, H, d]")
        Tt, Hk, dk = sq
        N, lead = sc[0] - 1, (Tt,)
        _need_all(((cu_seqlens, sc, torch.int32, "cu_seqlens"),))
    else:
        if len(sq) != 4 or len(sv) != 4:
            raise ValueError("without cu_seqlens, q and v are [B, T, H, d]")
        N, T, Hk, dk = sq
        Tt, lead = N * T, (N, T)
    Hv, dv = sv[-2:]
    gates = (*lead, Hv)
    _need_all(((q, sq, io, "q"), (k, sq, io, "k"), (v, (*gates, dv), io, "v"), (g, gates, io, "g"), (beta, gates, io, "beta")))
    return N, Tt, Hk, Hv, dk, dv, lead


def _ws_bytes(workspace):
    if workspace is None:
        return 0
    _need_all(((workspace, workspace.shape, torch.uint8, "workspace"),))
    return workspace.numel()


def _paged_state(state, index, N, tail, name):
    """Checks a state buffer: [N, *tail], or [pages, *tail] where an index is given.  Its pages."""
    if state is None:
        if index is not None:
            raise ValueError(f"{name}_index needs {name}_state")
        return 0
    if index is None:
        _need_all(((state, (N,) + tail, torch.float32, f"{name}_state"),))
        return 0
    P = state.shape[0]
    _need_all(((index, (N,), torch.int32, f"{name}_index"), (state, (P,) + tail, torch.float32, f"{name}_state")))
    return P


@functools.lru_cache(maxsize=256)
def kda_gdr_workspace_size(N, T_total, Hk, Hv, dk, dv, dtype, *, backward=False):
    n = ctypes.c_size_t(0)
    _check(_lib.kda_gdr_workspace_size(N, T_total, Hk, Hv, dk, dv, _io_code(dtype), int(backward), ctypes.byref(n)),
           "kda_gdr_workspace_size")
    return int(n.value)


def kda_gdr_forward(q, k, v, g, beta, cu_seqlens=None, initial_state=None, out=None, final_state=None, *,
                    initial_index=None, final_index=None, workspace=None, stream=None):
    """The gated delta rule with one gate per value head, chunked.  q, k: [T_total, Hk, dk]; v:
    [T_total, Hv, dv]; g, beta: [T_total, Hv] (io dtype) for the sequences of cu_seqlens, or [B, T, ...]
    without it; value head h uses key head h // (Hv // Hk).  States are fp32 [N, Hv, dk, dv], or pages
    [P, Hv, dk, dv] with an int32 index [N] (initial: -1 starts from zeros; final: -1 is not kept; the
    two buffers have the same number of pages).  ``workspace`` (a uint8 CUDA tensor of
    kda_gdr_workspace_size bytes) is allocated with torch when not given.  Rows of no sequence are not written: in an
    ``out`` that is allocated here they hold anything.  Returns (out, final_state)."""
    if stream is None and workspace is None:
        r = _calls.gdr_forward(q, k, v, g, beta, cu_seqlens, initial_state, out, final_state, initial_index, final_index)
        if r is not None:
            return _taken(r, "kda_gdr_forward"), final_state
    N, Tt, Hk, Hv, dk, dv, lead = _gdr_shapes(q, k, v, g, beta, cu_seqlens)
    p0 = _paged_state(initial_state, initial_index, N, (Hv, dk, dv), "initial")
    p1 = _paged_state(final_state, final_index, N, (Hv, dk, dv), "final")
    if p0 and p1 and p0 != p1:
        raise ValueError(f"initial_state has {p0} pages, final_state {p1}")
    if out is None:
        out = _new(stream, torch.empty_like, v)
    else:
        _need_all(((out, v.shape, q.dtype, "out"),))
    if workspace is None:
        workspace = _workspace(stream, kda_gdr_workspace_size(N, Tt, Hk, Hv, dk, dv, q.dtype), q.device)
    _check(_lib.kda_gdr_forward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(initial_index), _ptr(out),
        _ptr(final_state), _ptr(final_index), max(p0, p1), _ptr(cu_seqlens), _ptr(workspace), _ws_bytes(workspace),
        N, Tt, Hk, Hv, dk, dv, _io_code(q.dtype), _stream(stream)), "kda_gdr_forward")
    _on(stream, out, workspace)
    return out, final_state


def kda_gdr_backward(q, k, v, g, beta, d_out, cu_seqlens=None, initial_state=None, d_final_state=None, *,
                     grads=None, d_initial_state=None, workspace=None, stream=None):
    """Gradients of kda_gdr_forward (dense states).  Returns a dict dq, dk, dv, dg, dbeta (io dtype,
    shaped as the inputs) and d_initial_state (fp32, None unless a buffer is passed).  ``grads`` may
    hold preallocated outputs; ``workspace`` is allocated with torch when not given.  Rows of no sequence are not
    written: where T_total has some behind the last sequence, give gradients that hold zeros there."""
    if grads is None and stream is None and workspace is None:
        r = _calls.gdr_backward(q, k, v, g, beta, d_out, cu_seqlens, initial_state, d_final_state, d_initial_state)
        if r is not None:
            dq, dk, dv, dg, db = _taken(r, "kda_gdr_backward")
            return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": db, "d_initial_state": d_initial_state}
    N, Tt, Hk, Hv, dk, dv, lead = _gdr_shapes(q, k, v, g, beta, cu_seqlens)
    _need(d_out, lead + (Hv, dv), q.dtype, "d_out")
    for t, n in ((initial_state, "initial_state"), (d_final_state, "d_final_state"),
                 (d_initial_state, "d_initial_state")):
        _need(t, (N, Hv, dk, dv), torch.float32, n, allow_none=True)
    gr = dict(grads or {})
    for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
        if gr.get(n) is None:
            gr[n] = _new(stream, torch.empty_like, t)
        else:
            _need_all(((gr[n], t.shape, q.dtype, n),))
    if workspace is None:
        workspace = _workspace(stream, kda_gdr_workspace_size(N, Tt, Hk, Hv, dk, dv, q.dtype, backward=True), q.device)
    _check(_lib.kda_gdr_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), _ptr(d_out),
        _ptr(d_final_state), _ptr(gr["dq"]), _ptr(gr["dk"]), _ptr(gr["dv"]), _ptr(gr["dg"]), _ptr(gr["dbeta"]),
        _ptr(d_initial_state), _ptr(workspace), _ws_bytes(workspace), N, Tt, Hk, Hv, dk, dv, _io_code(q.dtype),
        _stream(stream)), "kda_gdr_backward")
    _on(stream, workspace, *gr.values())
    gr["d_initial_state"] = d_initial_state
    return gr


def kda_gdr_decode(q, k, v, g, beta, state, index=None, out=None, *, stream=None):
    """One or a few tokens per sequence, states updated in place.  q, k: [N, T, Hk, dk]; v: [N, T, Hv, dv];
    g, beta: [N, T, Hv], or all without T for one token; state: fp32 [N, Hv, dk, dv], or pages
    [P, Hv, dk, dv] with ``index`` int32 [N] (-1: an idle row, whose out is left alone).  Returns out."""
    if stream is None:
        r = _calls.gdr_decode(q, k, v, g, beta, state, index, out)
        if r is not None:
            return _taken(r, "kda_gdr_decode")
    sq, sv, io = q.shape, v.shape, q.dtype
    if len(sq) == 4 and len(sv) == 4:
        N, T, Hk, dk = sq
        lead = (N, T)
    elif len(sq) == 3 and len(sv) == 3:
        N, Hk, dk = sq
        lead, T = (N,), 1
    else:
        raise ValueError("q and v are [N, T, H, d], or [N, H, d] for one token")
    Hv, dv = sv[-2:]
    gates = (*lead, Hv)
    shape = (*gates, dv)
    if index is None:
        P, idx = N, None
    else:
        P = state.shape[0]
        _need_all(((index, (N,), torch.int32, "index"),))
        idx = index.data_ptr()
    _need_all(((q, sq, io, "q"), (k, sq, io, "k"), (v, shape, io, "v"), (g, gates, io, "g"), (beta, gates, io, "beta"),
               (state, (P, Hv, dk, dv), torch.float32, "state")))
    if out is None:
        out = _new(stream, _empty, shape, dtype=io, device=q.device)
    else:
        _need_all(((out, shape, io, "out"),))
    st = _lib.kda_gdr_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(),
                             idx, P, out.data_ptr(), N, T, Hk, Hv, dk, dv, _io_code(io), _stream(stream))
    if st:
        raise KdaError(st, "kda_gdr_decode")
    _on(stream, out)
    return out


def _cache(cache):
    """(layers, pages, bytes of a page) of a cache [layers, pages, ...] of any dtype."""
    if cache.dim() < 3:
        raise ValueError("cache must be [layers, pages, ...]")
    _need_all(((cache, cache.shape, cache.dtype, "cache"),))
    L, P = cache.shape[:2]
    return L, P, (cache.numel() // max(1, L * P)) * cache.element_size()


def _ids(t, name):
    if t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D tensor of page numbers")
    _need_all(((t, t.shape, torch.int32, name),))
    return t.shape[0]


def kda_pages_fork(cache, refs, parents, children=None, *, stream=None):
    """A free page for each of ``parents`` (int32 [n]), lowest first, with the parent's contents in every
    layer of ``cache`` [L, P, ...] (zeros for -1); ``refs`` (int32 [P]) of the new pages become 1.
    Returns their numbers, int32 [n]: -1 where no page is left or the parent is not live."""
    if stream is None and children is None:
        r = _calls.pages_fork(cache, refs, parents)
        if r is not None:
            return _taken(r, "kda_pages_fork")
    L, P, nbytes = _cache(cache)
    n = _ids(parents, "parents")
    if children is None:
        children = _new(stream, torch.empty_like, parents)
    _need_all(((refs, (P,), torch.int32, "refs"), (children, (n,), torch.int32, "children")))
    _check(_lib.kda_pages_fork(_ptr(cache), nbytes, L, P, _ptr(refs), _ptr(parents), _ptr(children), n, _stream(stream)),
           "kda_pages_fork")
    _on(stream, children)
    return children


def kda_pages_copy(cache, src, dst, *, stream=None):
    """Page dst[i] <- page src[i] in every layer of ``cache`` [L, P, ...] (src -1: zeros; dst -1: nothing)."""
    L, P, nbytes = _cache(cache)
    n = _ids(src, "src")
    _need(dst, (n,), torch.int32, "dst")
    _check(_lib.kda_pages_copy(_ptr(cache), nbytes, L, P, _ptr(src), _ptr(dst), n, _stream(stream)), "kda_pages_copy")


def kda_pages_free(refs, ids, *, stream=None):
    """One holder less for each page of ``ids`` (int32 [n], -1: nothing); a page is free at refs 0."""
    if stream is None:
        r = _calls.pages_free(refs, ids)
        if r is not None:
            _taken(r, "kda_pages_free")
            return
    n = _ids(ids, "ids")
    P = _ids(refs, "refs")
    _check(_lib.kda_pages_free(_ptr(refs), P, _ptr(ids), n, _stream(stream)), "kda_pages_free")


@functools.lru_cache(maxsize=256)
def kda_pages_workspace_size(pages):
    n = ctypes.c_size_t(0)
    _check(_lib.kda_pages_workspace_size(pages, ctypes.byref(n)), "kda_pages_workspace_size")
    return int(n.value)


def kda_pages_compact(cache, refs, table=None, live=None, *, workspace=None, stream=None):
    """Moves the live pages of ``cache`` [L, P, ...] to the lowest numbers, ``refs`` (int32 [P]) with them,
    and renumbers ``table`` (int32, any page numbers, -1 stays) in place.  Returns their count, int32 [1]."""
    if stream is None and live is None and workspace is None:
        r = _calls.pages_compact(cache, refs, table)
        if r is not None:
            return _taken(r, "kda_pages_compact")
    L, P, nbytes = _cache(cache)
    _need_all(((refs, (P,), torch.int32, "refs"),))
    n = 0
    if table is not None:
        _need_all(((table, table.shape, torch.int32, "table"),))
        n = table.numel()
    if live is None:
        live = _new(stream, torch.empty, 1, dtype=torch.int32, device=cache.device)
    else:
        _need_all(((live, (1,), torch.int32, "live"),))
    if workspace is None:
        workspace = _workspace(stream, kda_pages_workspace_size(P), cache.device)
    _check(_lib.kda_pages_compact(_ptr(cache), nbytes, L, P, _ptr(refs), _ptr(table), n, _ptr(live), _ptr(workspace),
                                  _ws_bytes(workspace), _stream(stream)), "kda_pages_compact")
    _on(stream, live, workspace)
    return live


def kda_check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel flagged a bounded-wait timeout, a bad page index or a
    CUDA error."""
    _check(_lib.kda_check_device_error(_stream(stream)), "kda_check_device_error")


def kda_set_wait_test_hooks(wait_limit_ns=0, skip_load_chunk=-1):
    """Limit of the tensor-core kernels' bounded waits (0: the default 2 s) and an injected
    failure (the tile load of chunk `skip_load_chunk` is never issued; -1: off; c <= -2: that of chunk -2 - c
    in the launch before the walks of the head-gated rule).  Process-wide."""
    _check(_lib.kda_set_wait_test_hooks(int(wait_limit_ns), int(skip_load_chunk)), "kda_set_wait_test_hooks")


# short names
forward_chunked = kda_forward_chunked
forward_chunked_varlen = kda_forward_chunked_varlen
backward_chunked = kda_backward_chunked
decode_step = kda_decode_step
layer_forward = kda_layer_forward
gdr_forward = kda_gdr_forward
gdr_backward = kda_gdr_backward
gdr_decode = kda_gdr_decode
pages_fork = kda_pages_fork
pages_copy = kda_pages_copy
pages_free = kda_pages_free
pages_compact = kda_pages_compact
layer_workspace_size = kda_layer_workspace_size
check_device_error = kda_check_device_error
