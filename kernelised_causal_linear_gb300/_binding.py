"""Thin ctypes binding of liblinattn.so with the C ABI's own names.

Only argument marshalling happens here: tensors become device pointers and
sizes, enums become ints, and a non-zero status becomes an exception.  Every
step of the computation runs in the library's CUDA kernels.  There is no
fallback: if the library has not been built, importing this module raises.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

from . import build as _build

LIB_PATH: Path = _build.LIB

if not LIB_PATH.exists():
    raise ImportError(
        f"liblinattn.so not found at {LIB_PATH}; build it first with "
        "`python -c 'import __graft_entry__ as g; g.build()'` "
        "(kernelised_causal_linear_gb300.build.build())")

_lib = ctypes.CDLL(str(LIB_PATH))

LA_OK = 0
STATUS_NAMES = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_CUDA",
                4: "LA_ERR_TIMEOUT", 5: "LA_ERR_DEVICE_CHECK", 6: "LA_ERR_WORKSPACE",
                7: "LA_ERR_TOO_LARGE"}
FEATURE_MAPS = {"elu1": 0, "identity_norm": 1, "none": 2, "l2": 3}
ACTIVATIONS = {"silu": 0, "sigmoid": 1, "none": 2}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_vp, _i64, _i, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_f = ctypes.c_float
_fp = ctypes.POINTER(ctypes.c_float)

_lib.la_version.restype = _i
_lib.la_version.argtypes = []
_lib.la_status_string.restype = ctypes.c_char_p
_lib.la_status_string.argtypes = [_i]
_lib.la_forward_workspace_size.restype = _sz
_lib.la_forward_workspace_size.argtypes = [_i64, _i64, _i64, _i, _i, _i, _i]
_lib.la_state_workspace_size.restype = _sz
_lib.la_state_workspace_size.argtypes = [_i64, _i64, _i64, _i, _i, _i]
_lib.la_forward.restype = _i
_lib.la_forward.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _i, _i, _fp, _i, _vp,
                            _sz, _vp]
_lib.la_state.restype = _i
_lib.la_state.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _i, _fp, _i, _vp, _sz,
                          _vp]
_lib.la_decode_step.restype = _i
_lib.la_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i, _i, _i, _fp, _i,
                                _vp]
_lib.la_forward_with_state.restype = _i
_lib.la_forward_with_state.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                       _i, _i, _i, _fp, _i, _vp, _sz, _vp]
_lib.la_gla_workspace_size.restype = _sz
_lib.la_gla_workspace_size.argtypes = [_i64, _i64, _i64, _i, _i]
_lib.la_forward_gla.restype = _i
_lib.la_forward_gla.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _i, _i, _vp,
                                _sz, _vp]
_lib.la_decode_step_gla.restype = _i
_lib.la_decode_step_gla.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i, _i, _i, _i,
                                    _vp]
_lib.la_state_prefix.restype = _i
_lib.la_state_prefix.argtypes = [_vp, _vp, _i, ctypes.POINTER(ctypes.c_int64), _i, _vp, _vp, _i64,
                                 _i64, _i, _i, _fp, _vp]
_lib.la_favor_features.restype = _i
_lib.la_favor_features.argtypes = [_vp, _vp, _vp, _i64, _i, _i, _i, _i, _vp]
_lib.la_delta_workspace_size.restype = _sz
_lib.la_delta_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i, _i, _i]
_lib.la_forward_delta.restype = _i
_lib.la_forward_delta.argtypes = [_vp] * 8 + [_i64] * 4 + [_i, _i, _i, _f, _i, _vp, _sz, _vp]
_lib.la_decode_step_delta.restype = _i
_lib.la_decode_step_delta.argtypes = [_vp] * 7 + [_i64] * 3 + [_i, _i, _i, _f, _i, _vp]
_lib.la_delta_backward_workspace_size.restype = _sz
_lib.la_delta_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i, _i, _i]
_lib.la_backward_delta.restype = _i
_lib.la_backward_delta.argtypes = [_vp] * 14 + [_i64] * 4 + [_i, _i, _i, _f, _i, _vp, _sz, _vp]
_lib.la_norm_gate.restype = _i
_lib.la_norm_gate.argtypes = [_vp] * 4 + [_i64] * 3 + [_i, _i, _i, _f, _i, _i, _vp]
_lib.la_norm_gate_backward_workspace_size.restype = _sz
_lib.la_norm_gate_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i]
_lib.la_norm_gate_backward.restype = _i
_lib.la_norm_gate_backward.argtypes = [_vp] * 7 + [_i64] * 3 + [_i, _i, _i, _f, _i, _i, _vp, _sz,
                                                               _vp]
_lib.la_forward_conv.restype = _i
_lib.la_forward_conv.argtypes = [_vp, _i64, _i64] + [_vp] * 6 + [_i64] * 4 + [_i, _i, _i, _vp]
_lib.la_decode_step_conv.restype = _i
_lib.la_decode_step_conv.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i, _i, _i, _vp]
_lib.la_conv_backward_workspace_size.restype = _sz
_lib.la_conv_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i, _i]
_lib.la_backward_conv.restype = _i
_lib.la_backward_conv.argtypes = [_vp, _vp, _vp, _i64, _i64] + [_vp] * 8 + [_i64] * 4 + [_i, _i, _i, _vp, _sz, _vp]
_strides = ctypes.POINTER(ctypes.c_int64)
_lib.la_ssm_workspace_size.restype = _sz
_lib.la_ssm_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i, _i]
_lib.la_forward_ssm.restype = _i
_lib.la_forward_ssm.argtypes = [_vp] * 12 + [_strides] + [_i64] * 4 + [_i, _i, _i, _vp, _sz, _vp]
_lib.la_decode_step_ssm.restype = _i
_lib.la_decode_step_ssm.argtypes = [_vp] * 10 + [_strides] + [_i64] * 3 + [_i, _i, _i, _vp]
_lib.la_ssm_backward_workspace_size.restype = _sz
_lib.la_ssm_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i, _i]
_lib.la_backward_ssm.restype = _i
_lib.la_backward_ssm.argtypes = [_vp] * 21 + [_strides] + [_i64] * 4 + [_i, _i, _i, _vp, _sz, _vp]
_lib.la_forward_noalloc.restype = _i
_lib.la_forward_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _i, _i, _fp,
                                    _i, _vp]
_lib.la_forward_path.restype = ctypes.c_char_p
_lib.la_forward_path.argtypes = [_i64, _i64, _i64, _i, _i, _i, _i, _i, _i]
_lib.la_debug_set_tc_faults.restype = _i
_lib.la_debug_set_tc_faults.argtypes = [ctypes.c_uint64, _i]
_lib.la_launch_count.restype = ctypes.c_uint64
_lib.la_launch_count.argtypes = []
_lib.la_get_device_status.restype = _i
_lib.la_get_device_status.argtypes = [_vp]


class LinAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {la_status_string(code)}")


def la_version() -> int:
    return _lib.la_version()


def la_status_string(code: int) -> str:
    return _lib.la_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != LA_OK:
        raise LinAttnError(code, where)


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _gamma_arg(gamma, H: int):
    if gamma is None:
        return None, None
    g = torch.as_tensor(gamma, dtype=torch.float32, device="cpu").contiguous().reshape(-1)
    if g.numel() != H:
        raise ValueError(f"gamma must have H={H} entries, got {g.numel()}")
    return ctypes.cast(g.data_ptr(), _fp), g  # keep g alive for the call


def _fm(feature_map) -> int:
    return FEATURE_MAPS[feature_map] if isinstance(feature_map, str) else int(feature_map)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in DTYPES:
        raise TypeError(f"unsupported input dtype {t.dtype}; use bfloat16 or float32")
    return DTYPES[t.dtype]


def _dev_ptr(t: torch.Tensor | None, name: str) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def la_forward_workspace_size(B, H, N, d, dv, causal=True, dtype=torch.bfloat16) -> int:
    return int(_lib.la_forward_workspace_size(B, H, N, d, dv, int(bool(causal)),
                                              DTYPES[dtype]))


def la_state_workspace_size(B, H, N, d, dv, dtype=torch.bfloat16) -> int:
    return int(_lib.la_state_workspace_size(B, H, N, d, dv, DTYPES[dtype]))


def la_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor | None = None,
               *, causal: bool = True, feature_map="elu1", gamma=None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q, k: [B,H,N,d]; v: [B,H,N,dv] (bf16 or fp32, CUDA) -> out [B,H,N,dv] fp32.

    ``workspace`` may be passed to reuse scratch across calls (a uint8 CUDA
    tensor of at least la_forward_workspace_size() bytes); otherwise one is
    allocated by PyTorch for this call.
    """
    B, H, N, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    need = la_forward_workspace_size(B, H, N, d, dv, causal, q.dtype) if q.dtype in DTYPES else 0
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_forward(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                           _dev_ptr(out, "out"), B, H, N, d, dv, int(bool(causal)),
                           _fm(feature_map), gp, _dtype(q), _dev_ptr(workspace, "workspace"),
                           workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(code, "la_forward")
    return out


def la_forward_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       *, causal: bool = True, feature_map="elu1", gamma=None,
                       stream=None) -> torch.Tensor:
    """la_forward with no workspace argument and no allocation anywhere: for
    callers that cannot allocate device memory (their host application owns
    all of it, or they must not risk the device-wide synchronisation of
    cudaMalloc / cudaFree).  Scratch comes from a fixed device array inside the
    library; ``out`` must be given, since creating it would allocate.  Calls
    that overlap on the GPU share that array and race."""
    B, H, N, d = q.shape
    dv = v.shape[-1]
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_forward_noalloc(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                                   _dev_ptr(out, "out"), B, H, N, d, dv, int(bool(causal)),
                                   _fm(feature_map), gp, _dtype(q), _stream_handle(stream))
    _check(code, "la_forward_noalloc")
    return out


def la_forward_with_state(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                          out: torch.Tensor | None = None, *, S0: torch.Tensor | None = None,
                          z0: torch.Tensor | None = None, S_out: torch.Tensor | None = None,
                          z_out: torch.Tensor | None = None, return_state: bool = True,
                          feature_map="elu1", gamma=None, workspace: torch.Tensor | None = None,
                          stream=None):
    """Causal forward continued from (S0, z0) [B,H,d,dv] / [B,H,d] (None: zero
    state), returning (out, S_out, z_out).  q = None computes the final state
    only (out is then None).  S_out / z_out may be S0 / z0 (in-place)."""
    B, H, N, d = k.shape
    dv = v.shape[-1]
    if q is not None and out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=k.device)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=k.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=k.device)
    need = la_forward_workspace_size(B, H, N, d, dv, True, k.dtype) if k.dtype in DTYPES else 0
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=k.device)
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_forward_with_state(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(out, "out"),
        _dev_ptr(S0, "S0"), _dev_ptr(z0, "z0"), _dev_ptr(S_out, "S_out"), _dev_ptr(z_out, "z_out"),
        B, H, N, d, dv, _fm(feature_map), gp, _dtype(k), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(code, "la_forward_with_state")
    return out, S_out, z_out


def la_state(k: torch.Tensor, v: torch.Tensor, S: torch.Tensor | None = None,
             z: torch.Tensor | None = None, *, feature_map="elu1", gamma=None,
             workspace: torch.Tensor | None = None, stream=None):
    """State after the N tokens of k [B,H,N,d], v [B,H,N,dv] -> (S [B,H,d,dv], z [B,H,d])."""
    B, H, N, d = k.shape
    dv = v.shape[-1]
    if S is None:
        S = torch.empty((B, H, d, dv), dtype=torch.float32, device=k.device)
    if z is None:
        z = torch.empty((B, H, d), dtype=torch.float32, device=k.device)
    need = la_state_workspace_size(B, H, N, d, dv, k.dtype) if k.dtype in DTYPES else 0
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=k.device)
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_state(_dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(S, "S"), _dev_ptr(z, "z"),
                         B, H, N, d, dv, _fm(feature_map), gp, _dtype(k),
                         _dev_ptr(workspace, "workspace"),
                         workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(code, "la_state")
    return S, z


def la_decode_step(S: torch.Tensor, z: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                   v: torch.Tensor, out: torch.Tensor | None = None, *, feature_map="elu1",
                   gamma=None, stream=None) -> torch.Tensor:
    """One token per sequence: q, k [B,H,d], v [B,H,dv]; S, z updated in place."""
    B, H, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_decode_step(_dev_ptr(S, "S"), _dev_ptr(z, "z"), _dev_ptr(q, "q"),
                               _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(out, "out"), B, H, d,
                               dv, _fm(feature_map), gp, _dtype(q), _stream_handle(stream))
    _check(code, "la_decode_step")
    return out


def la_gla_workspace_size(B, H, N, d, dv) -> int:
    return int(_lib.la_gla_workspace_size(B, H, N, d, dv))


def la_forward_gla(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                   out: torch.Tensor | None = None, *, feature_map="elu1",
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal forward with per-key-channel decay alpha [B,H,N,d] (fp32, in (0, 1])."""
    B, H, N, d = q.shape
    dv = v.shape[-1]
    if alpha.dtype != torch.float32:
        raise TypeError("alpha must be float32")
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    need = int(_lib.la_gla_workspace_size(B, H, N, d, dv))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    code = _lib.la_forward_gla(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                               _dev_ptr(alpha, "alpha"), _dev_ptr(out, "out"), B, H, N, d, dv,
                               _fm(feature_map), _dtype(q), _dev_ptr(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(),
                               _stream_handle(stream))
    _check(code, "la_forward_gla")
    return out


def la_decode_step_gla(S, z, q, k, v, alpha, out=None, *, feature_map="elu1", stream=None):
    """One token per sequence with per-key-channel decay alpha [B,H,d] (fp32)."""
    B, H, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    code = _lib.la_decode_step_gla(_dev_ptr(S, "S"), _dev_ptr(z, "z"), _dev_ptr(q, "q"),
                                   _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(alpha, "alpha"),
                                   _dev_ptr(out, "out"), B, H, d, dv, _fm(feature_map), _dtype(q),
                                   _stream_handle(stream))
    _check(code, "la_decode_step_gla")
    return out


def la_state_prefix(S_parts: torch.Tensor, z_parts: torch.Tensor, part_len, upto: int,
                    S_out: torch.Tensor | None = None, z_out: torch.Tensor | None = None, *,
                    gamma=None, stream=None):
    """State before part `upto` from every part's own state: S_parts
    [P,B,H,d,dv], z_parts [P,B,H,d], part_len P token counts -> (S, z)."""
    P, B, H, d, dv = S_parts.shape
    if S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=S_parts.device)
    if z_out is None:
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=S_parts.device)
    lens = (ctypes.c_int64 * P)(*[int(x) for x in part_len])
    gp, _keep = _gamma_arg(gamma, H)
    code = _lib.la_state_prefix(_dev_ptr(S_parts, "S_parts"), _dev_ptr(z_parts, "z_parts"), P,
                                lens, int(upto), _dev_ptr(S_out, "S_out"), _dev_ptr(z_out, "z_out"),
                                B, H, d, dv, gp, _stream_handle(stream))
    _check(code, "la_state_prefix")
    return S_out, z_out


def la_favor_features(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None, *,
                      out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Positive random features of x [..., d] with Gaussian rows w [r, d]
    (fp32): exp(w . x' - |x'|^2 / 2) / sqrt(r), x' = x / d^(1/4) -> [..., r]."""
    d = x.shape[-1]
    r = w.shape[0]
    if w.dtype != torch.float32 or tuple(w.shape) != (r, d):
        raise ValueError("w must be a float32 [r, d] tensor")
    if out is None:
        out = torch.empty(x.shape[:-1] + (r,), dtype=out_dtype, device=x.device)
    code = _lib.la_favor_features(_dev_ptr(x, "x"), _dev_ptr(w, "w"), _dev_ptr(out, "out"),
                                  x.numel() // d, d, r, _dtype(x), DTYPES[out.dtype],
                                  _stream_handle(stream))
    _check(code, "la_favor_features")
    return out


def _arg(t: torch.Tensor | None, name: str, shape, dtype, index: int) -> int | None:
    """Device pointer of a tensor that has to have this shape, type and place."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other arguments on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _apart(name: str, out: int | None, *inputs) -> None:
    """An output may not be one of the inputs: other blocks still read those."""
    if out and out in inputs:
        raise ValueError(f"{name} shares its memory with an input")


def _current(t: torch.Tensor, name: str) -> int:
    """The device of a call: its tensors' device, which has to be the current one."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    current = torch._C._cuda_getDevice()  # a CUDA tensor exists: there is a context
    if index != current:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{current}")
    if t.dtype not in DTYPES:
        _dtype(t)
    return index


# a number in place of the device costs torch.empty 2 us more
_DEVICES = [torch.device("cuda", i) for i in range(64)]


class _Call:
    """The stream of a call and what is allocated for it: outputs and scratch
    belong to that stream, so none is handed out again before it has run."""

    def __init__(self, stream, index: int):
        self.index = index
        self.handle = torch._C._cuda_getCurrentRawStream(index)
        self.side = None  # the call's stream where it is not the current one
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            if handle != self.handle:
                self.handle = handle
                self.side = torch.cuda.ExternalStream(handle, device=index) if handle else \
                    torch.cuda.default_stream(index)

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=_DEVICES[self.index])
        if self.side is not None:
            # allocated for the current stream: the call's own may write only
            # once what had the memory before is done, and the memory stays
            # until the call is
            self.side.wait_stream(torch.cuda.current_stream(self.index))
            t.record_stream(self.side)
        return t

    def scratch(self, workspace, need):
        """Pointer and size of the given workspace, or of a new one."""
        if workspace is None:
            if need == 0:
                return None, 0
            workspace = self.empty(need, torch.uint8)
        elif workspace.get_device() != self.index:
            raise ValueError(f"workspace is on {workspace.device}, not cuda:{self.index}")
        return _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _delta_sizes(k, v):
    x, y = k.shape, v.shape
    if len(x) != len(y) or x[0] != y[0] or (len(x) == 4 and x[2] != y[2]):
        raise ValueError(f"k {tuple(x)} and v {tuple(y)} do not belong together")
    return y[0], y[1], x[1], x[-1], y[-1]


def la_delta_workspace_size(B, H, Hk, N, d, dv, dtype=torch.bfloat16) -> int:
    return int(_lib.la_delta_workspace_size(B, H, Hk, N, d, dv, DTYPES[dtype]))


def la_delta_backward_workspace_size(B, H, Hk, N, d, dv, dtype=torch.bfloat16) -> int:
    return int(_lib.la_delta_backward_workspace_size(B, H, Hk, N, d, dv, DTYPES[dtype]))


def la_forward_delta(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                     beta: torch.Tensor, log_alpha: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, *, feature_map="l2",
                     scale: float | None = None, S0: torch.Tensor | None = None,
                     S_out: torch.Tensor | None = None, return_state: bool = False,
                     workspace: torch.Tensor | None = None, stream=None):
    """Gated delta rule over whole sequences -> (out, S_out).

    q, k [B,Hk,N,d], v [B,H,N,dv] (bf16 or fp32), beta and log_alpha [B,H,N]
    fp32 (None: no decay); out [B,H,N,dv] in v's type.  S0 is the state before
    the first token (None: zero); the final state is written when S_out is
    given or return_state is set, else None is returned for it.  q = None
    computes the final state alone.  scale defaults to 1/sqrt(d)."""
    if k.dim() != 4:
        raise ValueError("k must be [B,Hk,N,d]")
    dev = _current(k, "k")
    B, H, Hk, d, dv = _delta_sizes(k, v)
    N = k.shape[2]
    call = _Call(stream, dev)
    if q is not None and out is None:
        out = call.empty((B, H, N, dv), k.dtype)
    if S_out is None and (return_state or q is None):
        S_out = call.empty((B, H, d, dv), torch.float32)
    f32, gates, state = torch.float32, (B, H, N), (B, H, d, dv)
    ptrs = (_arg(q, "q", k.shape, k.dtype, dev), _arg(k, "k", k.shape, k.dtype, dev),
            _arg(v, "v", (B, H, N, dv), k.dtype, dev), _arg(beta, "beta", gates, f32, dev),
            _arg(log_alpha, "log_alpha", gates, f32, dev),
            _arg(out, "out", (B, H, N, dv), k.dtype, dev), _arg(S0, "S0", state, f32, dev),
            _arg(S_out, "S_out", state, f32, dev))
    _apart("out", ptrs[5], *ptrs[:3])
    ws = call.scratch(workspace, la_delta_workspace_size(B, H, Hk, N, d, dv, k.dtype))
    code = _lib.la_forward_delta(*ptrs, B, H, Hk, N, d, dv, _fm(feature_map),
                                 d ** -0.5 if scale is None else float(scale), _dtype(k), *ws,
                                 call.handle)
    _check(code, "la_forward_delta")
    return out, S_out


def la_decode_step_delta(S: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         beta: torch.Tensor, log_alpha: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, *, feature_map="l2",
                         scale: float | None = None, stream=None) -> torch.Tensor:
    """One token per sequence: q, k [B,Hk,d], v [B,H,dv], beta and log_alpha
    [B,H]; S [B,H,d,dv] updated in place -> out [B,H,dv] in v's type."""
    if k.dim() != 3:
        raise ValueError("k must be [B,Hk,d]")
    dev = _current(k, "k")
    B, H, Hk, d, dv = _delta_sizes(k, v)
    call = _Call(stream, dev)
    if out is None:
        out = call.empty((B, H, dv), k.dtype)
    f32 = torch.float32
    ptrs = (_arg(S, "S", (B, H, d, dv), f32, dev), _arg(q, "q", k.shape, k.dtype, dev),
            _arg(k, "k", k.shape, k.dtype, dev), _arg(v, "v", (B, H, dv), k.dtype, dev),
            _arg(beta, "beta", (B, H), f32, dev), _arg(log_alpha, "log_alpha", (B, H), f32, dev),
            _arg(out, "out", (B, H, dv), k.dtype, dev))
    _apart("out", ptrs[6], *ptrs[1:4])
    code = _lib.la_decode_step_delta(
        *ptrs, B, H, Hk, d, dv, _fm(feature_map), d ** -0.5 if scale is None else float(scale), _dtype(k), call.handle)
    _check(code, "la_decode_step_delta")
    return out


def la_backward_delta(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      beta: torch.Tensor, log_alpha: torch.Tensor | None = None, *,
                      feature_map="l2", scale: float | None = None,
                      S0: torch.Tensor | None = None, dS_out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """Gradients of la_forward_delta -> (dq, dk, dv, dbeta, dlog_alpha, dS0),
    with None for dlog_alpha without log_alpha and for dS0 without S0.  dout
    and dS_out (None: zero) are the gradients of out and of the final state."""
    if k.dim() != 4:
        raise ValueError("k must be [B,Hk,N,d]")
    dev = _current(k, "k")
    B, H, Hk, d, dv = _delta_sizes(k, v)
    N = k.shape[2]
    call = _Call(stream, dev)
    f32, gates, state, vs = torch.float32, (B, H, N), (B, H, d, dv), (B, H, N, dv)
    ins = (_arg(dout, "dout", vs, k.dtype, dev), _arg(dS_out, "dS_out", state, f32, dev),
           _arg(q, "q", k.shape, k.dtype, dev), _arg(k, "k", k.shape, k.dtype, dev),
           _arg(v, "v", vs, k.dtype, dev), _arg(beta, "beta", gates, f32, dev),
           _arg(log_alpha, "log_alpha", gates, f32, dev), _arg(S0, "S0", state, f32, dev))
    grads = (call.empty(k.shape, k.dtype), call.empty(k.shape, k.dtype), call.empty(vs, k.dtype),
             call.empty(gates, f32), call.empty(gates, f32) if log_alpha is not None else None,
             call.empty(state, f32) if S0 is not None else None)
    ws = call.scratch(workspace, la_delta_backward_workspace_size(B, H, Hk, N, d, dv, k.dtype))
    code = _lib.la_backward_delta(*ins, *(None if g is None else g.data_ptr() for g in grads), B, H,
                                  Hk, N, d, dv, _fm(feature_map),
                                  d ** -0.5 if scale is None else float(scale), _dtype(k), *ws,
                                  call.handle)
    _check(code, "la_backward_delta")
    return grads


def _act(activation) -> int:
    return ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)


def _norm_weight(weight, H, dv, dev):
    """(pointer, 1 if there is a row for each head)."""
    heads = weight is not None and weight.dim() == 2
    return _arg(weight, "weight", (H, dv) if heads else (dv,), torch.float32, dev), int(heads)


def la_norm_gate_backward_workspace_size(B, H, N, dv) -> int:
    return int(_lib.la_norm_gate_backward_workspace_size(B, H, N, dv))


def la_norm_gate(x: torch.Tensor, gate: torch.Tensor | None = None,
                 weight: torch.Tensor | None = None, y: torch.Tensor | None = None, *,
                 activation="silu", eps: float = 1e-6, stream=None) -> torch.Tensor:
    """Head-major x [B,H,N,dv] -> token-major y [B,N,H,dv]: RMS norm of each
    row, times weight (fp32 [dv] or [H,dv]), times activation(gate) with gate
    [B,N,H,dv].  y has gate's type (x's without a gate, or that of a given y)."""
    if x.dim() != 4:
        raise ValueError("x must be [B,H,N,dv]")
    dev = _current(x, "x")
    B, H, N, dv = x.shape
    call = _Call(stream, dev)
    dtype = gate.dtype if gate is not None else y.dtype if y is not None else x.dtype
    if y is None:
        y = call.empty((B, N, H, dv), dtype)
    _dtype(y)
    w, heads = _norm_weight(weight, H, dv, dev)
    ptrs = (_arg(x, "x", x.shape, x.dtype, dev), _arg(gate, "gate", (B, N, H, dv), dtype, dev), w,
            _arg(y, "y", (B, N, H, dv), dtype, dev))
    _apart("y", ptrs[3], *ptrs[:2])
    code = _lib.la_norm_gate(*ptrs, B, H, N, dv, _act(activation), heads, float(eps), _dtype(x),
                             DTYPES[dtype], call.handle)
    _check(code, "la_norm_gate")
    return y


def la_norm_gate_backward(dy: torch.Tensor, x: torch.Tensor, gate: torch.Tensor | None = None,
                          weight: torch.Tensor | None = None, *, activation="silu",
                          eps: float = 1e-6, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of la_norm_gate from dy [B,N,H,dv] -> (dx [B,H,N,dv], dgate,
    dweight), None for a gate or weight that was not given."""
    if x.dim() != 4:
        raise ValueError("x must be [B,H,N,dv]")
    dev = _current(x, "x")
    B, H, N, dv = x.shape
    call = _Call(stream, dev)
    _dtype(dy)
    w, heads = _norm_weight(weight, H, dv, dev)
    ins = (_arg(dy, "dy", (B, N, H, dv), dy.dtype, dev), _arg(x, "x", x.shape, x.dtype, dev),
           _arg(gate, "gate", (B, N, H, dv), dy.dtype, dev), w)
    grads = (call.empty(x.shape, x.dtype),
             call.empty(dy.shape, dy.dtype) if gate is not None else None,
             call.empty(weight.shape, torch.float32) if weight is not None else None)
    need = la_norm_gate_backward_workspace_size(B, H, N, dv) if weight is not None else 0
    ws = call.scratch(workspace, need)
    code = _lib.la_norm_gate_backward(*ins, *(None if g is None else g.data_ptr() for g in grads),
                                      B, H, N, dv, _act(activation), heads, float(eps), _dtype(x),
                                      _dtype(dy), *ws, call.handle)
    _check(code, "la_norm_gate_backward")
    return grads


def _rows(t: torch.Tensor | None, name: str, shape, lead: int, dtype, index: int):
    """Pointer and row strides of an input whose dimensions from `lead` on (channels, or
    groups and states) are neighbours and whose first ones, (batch,) or (batch, token),
    have any strides."""
    if t is None:
        return (None, 0) if lead == 1 else (None, 0, 0)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other arguments on cuda:{index}")
    strides = t.stride()
    if (strides[-1] != 1 and shape[-1] != 1) or (
            len(shape) - lead == 2 and shape[-2] != 1 and strides[-2] != shape[-1]):
        raise ValueError(f"{name}'s channels must be next to one another")
    # the stride of a dimension of one says nothing
    batch = strides[0] if shape[0] != 1 else 0
    if lead == 1:
        return t.data_ptr(), batch
    return t.data_ptr(), batch, strides[1] if shape[1] != 1 else 0


def _lengths(t, B, index):
    return _arg(t, "lengths", (B,), torch.int32, index)


def la_conv_backward_workspace_size(B, N, C, W, dtype=torch.bfloat16) -> int:
    return int(_lib.la_conv_backward_workspace_size(B, N, C, W, DTYPES[dtype]))


def _filter(weight, bias, C, dev):
    if weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    return _arg(weight, "weight", (C, W), torch.float32, dev), _arg(bias, "bias", (C,), torch.float32, dev), W


def la_forward_conv(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                    y: torch.Tensor | None = None, *, activation="silu", heads: int | None = None,
                    S0: torch.Tensor | None = None, S_out: torch.Tensor | None = None,
                    return_state: bool = False, lengths: torch.Tensor | None = None, stream=None):
    """Short causal convolution of x [B,N,C] (bf16 or fp32, any batch and token
    strides) with weight [C,W] and bias [C] (fp32) -> (y, S_out).

    y is token-major [B,N,C], or head-major [B,heads,N,C/heads] for the attention
    calls.  S0 [B,W-1,C] holds the inputs before the first token (None: zeros); the
    last W-1 inputs are written when S_out is given (it may be S0) or return_state is
    set.  lengths (int32 [B]): row b ends after lengths[b] tokens, y is zero behind."""
    if x.dim() != 3:
        raise ValueError("x must be [B,N,C]")
    dev = _current(x, "x")
    B, N, C = x.shape
    if heads is not None and (heads < 1 or C % heads):
        raise ValueError(f"heads must divide the {C} channels")
    call = _Call(stream, dev)
    shape = (B, N, C) if heads is None else (B, heads, N, C // heads)
    if y is None:
        y = call.empty(shape, x.dtype)
    w, b, W = _filter(weight, bias, C, dev)
    window = (B, W - 1, C)
    if S_out is None and return_state:
        S_out = call.empty(window, x.dtype)
    xs = _rows(x, "x", x.shape, 2, x.dtype, dev)
    yp = _arg(y, "y", shape, x.dtype, dev)
    _apart("y", yp, xs[0])
    code = _lib.la_forward_conv(*xs, w, b, yp, _arg(S0, "S0", window, x.dtype, dev),
                                _arg(S_out, "S_out", window, x.dtype, dev), _lengths(lengths, B, dev),
                                B, N, C, heads or 1, W, _act(activation), _dtype(x), call.handle)
    _check(code, "la_forward_conv")
    return y, S_out


def la_decode_step_conv(S: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        bias: torch.Tensor | None = None, y: torch.Tensor | None = None, *,
                        activation="silu", stream=None) -> torch.Tensor:
    """One token per sequence: x [B,C] (any row stride); the window S [B,W-1,C] moves on
    in place -> y [B,C]."""
    if x.dim() != 2:
        raise ValueError("x must be [B,C]")
    dev = _current(x, "x")
    B, C = x.shape
    call = _Call(stream, dev)
    if y is None:
        y = call.empty((B, C), x.dtype)
    w, b, W = _filter(weight, bias, C, dev)
    xs = _rows(x, "x", x.shape, 1, x.dtype, dev)
    yp = _arg(y, "y", (B, C), x.dtype, dev)
    _apart("y", yp, xs[0])
    code = _lib.la_decode_step_conv(_arg(S, "S", (B, W - 1, C), x.dtype, dev), *xs, w, b, yp, B, C, W,
                                    _act(activation), _dtype(x), call.handle)
    _check(code, "la_decode_step_conv")
    return y


def la_backward_conv(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                     bias: torch.Tensor | None = None, *, activation="silu",
                     S0: torch.Tensor | None = None, dS_out: torch.Tensor | None = None,
                     lengths: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Gradients of la_forward_conv -> (dx, dweight, dbias, dS0), with None for dbias
    without bias and for dS0 without S0.  dy is [B,N,C], or [B,heads,N,C/heads] for a
    head-major y; dS_out (None: zero) is the gradient of the final window."""
    if x.dim() != 3 or dy.dim() not in (3, 4):
        raise ValueError("x must be [B,N,C], dy [B,N,C] or [B,heads,N,C/heads]")
    dev = _current(x, "x")
    B, N, C = x.shape
    heads = dy.shape[1] if dy.dim() == 4 else 1
    if heads < 1 or C % heads:
        raise ValueError(f"heads must divide the {C} channels")
    call = _Call(stream, dev)
    w, b, W = _filter(weight, bias, C, dev)
    window, f32 = (B, W - 1, C), torch.float32
    shape = (B, heads, N, C // heads) if dy.dim() == 4 else (B, N, C)
    ins = (_arg(dy, "dy", shape, x.dtype, dev), _arg(dS_out, "dS_out", window, x.dtype, dev),
           *_rows(x, "x", x.shape, 2, x.dtype, dev), w, b, _arg(S0, "S0", window, x.dtype, dev),
           _lengths(lengths, B, dev))
    grads = (call.empty((B, N, C), x.dtype), call.empty((C, W), f32),
             call.empty((C,), f32) if bias is not None else None,
             call.empty(window, x.dtype) if S0 is not None else None)
    ws = call.scratch(workspace, la_conv_backward_workspace_size(B, N, C, W, x.dtype))
    code = _lib.la_backward_conv(*ins, *(None if g is None else g.data_ptr() for g in grads), B, N, C,
                                 heads, W, _act(activation), _dtype(x), *ws, call.handle)
    _check(code, "la_backward_conv")
    return grads


def la_ssm_workspace_size(B, N, C, G, n, dtype=torch.bfloat16) -> int:
    return int(_lib.la_ssm_workspace_size(B, N, C, G, n, DTYPES[dtype]))


def la_ssm_backward_workspace_size(B, N, C, G, n, dtype=torch.bfloat16) -> int:
    return int(_lib.la_ssm_backward_workspace_size(B, N, C, G, n, DTYPES[dtype]))


def _ssm_inputs(x, delta, A, Bm, Cm, D, z, delta_bias, dev, lead):
    """Groups and states, pointers in the calls' order from x to delta_bias, strides on the host."""
    wide, shared, dtype, f32 = x.shape, Bm.shape, x.dtype, torch.float32
    if len(wide) != lead + 1 or len(shared) != lead + 2 or shared[:lead] != wide[:lead]:
        raise ValueError("x must be [B,C] and Bm [B,G,n]" if lead == 1 else "x must be [B,N,C] and Bm [B,N,G,n]")
    C, G, n = wide[-1], shared[-2], shared[-1]
    rows = (_rows(x, "x", wide, lead, dtype, dev), _rows(delta, "delta", wide, lead, dtype, dev),
            _rows(Bm, "Bm", shared, lead, dtype, dev), _rows(Cm, "Cm", shared, lead, dtype, dev),
            _rows(z, "z", wide, lead, dtype, dev))
    ptrs = (rows[0][0], rows[1][0], _arg(A, "A", (C, n), f32, dev), rows[2][0], rows[3][0],
            _arg(D, "D", (C,), f32, dev), rows[4][0], _arg(delta_bias, "delta_bias", (C,), f32, dev))
    strides = []
    for r in rows:
        strides += r[1:]
    return G, n, ptrs, strides


_STRIDES = {k: ctypes.c_int64 * k for k in (5, 10, 12)}


def _host_strides(strides):
    return _STRIDES[len(strides)](*strides)


def la_forward_ssm(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                   Cm: torch.Tensor, out: torch.Tensor | None = None, *,
                   D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                   delta_bias: torch.Tensor | None = None, softplus: bool = True,
                   S0: torch.Tensor | None = None, S_out: torch.Tensor | None = None,
                   return_state: bool = False, lengths: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """Selective state-space scan over whole sequences -> (out, S_out).

    x, delta, z [B,N,C] and Bm, Cm [B,N,G,n] (bf16 or fp32, any batch and token strides),
    A [C,n], D and delta_bias [C] fp32; out [B,N,C] in x's type:
    S_t = exp(dt A) S_{t-1} + dt x Bm, out = (Cm S_t + D x) silu(z) with
    dt = softplus(delta + delta_bias).  S0 [B,C,n] is the state before the first token
    (None: zero); the final state is written when S_out is given (it may be S0) or
    return_state is set.  lengths (int32 [B]): row b ends after lengths[b] tokens, out is
    zero behind."""
    dev = _current(x, "x")
    G, n, ptrs, strides = _ssm_inputs(x, delta, A, Bm, Cm, D, z, delta_bias, dev, 2)
    B, N, C = x.shape
    call = _Call(stream, dev)
    if out is None:
        out = call.empty((B, N, C), x.dtype)
    state = (B, C, n)
    if S_out is None and return_state:
        S_out = call.empty(state, torch.float32)
    op = _arg(out, "out", (B, N, C), x.dtype, dev)
    _apart("out", op, ptrs[0], ptrs[1], ptrs[6])
    ws = call.scratch(workspace, la_ssm_workspace_size(B, N, C, G, n, x.dtype))
    code = _lib.la_forward_ssm(*ptrs, op, _arg(S0, "S0", state, torch.float32, dev),
                               _arg(S_out, "S_out", state, torch.float32, dev), _lengths(lengths, B, dev),
                               _host_strides(strides), B, N, C, G, n, int(bool(softplus)), _dtype(x), *ws,
                               call.handle)
    _check(code, "la_forward_ssm")
    return out, S_out


def la_decode_step_ssm(S: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
                       Bm: torch.Tensor, Cm: torch.Tensor, out: torch.Tensor | None = None, *,
                       D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                       delta_bias: torch.Tensor | None = None, softplus: bool = True,
                       stream=None) -> torch.Tensor:
    """One token per sequence: x, delta, z [B,C], Bm, Cm [B,G,n] (any row stride); the state
    S [B,C,n] (fp32) is updated in place -> out [B,C] in x's type."""
    dev = _current(x, "x")
    G, n, ptrs, strides = _ssm_inputs(x, delta, A, Bm, Cm, D, z, delta_bias, dev, 1)
    B, C = x.shape
    call = _Call(stream, dev)
    if out is None:
        out = call.empty((B, C), x.dtype)
    op = _arg(out, "out", (B, C), x.dtype, dev)
    _apart("out", op, ptrs[0], ptrs[1], ptrs[6])
    code = _lib.la_decode_step_ssm(_arg(S, "S", (B, C, n), torch.float32, dev), *ptrs, op,
                                   _host_strides(strides), B, C, G, n, int(bool(softplus)), _dtype(x),
                                   call.handle)
    _check(code, "la_decode_step_ssm")
    return out


def la_backward_ssm(dout: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
                    Bm: torch.Tensor, Cm: torch.Tensor, *, D: torch.Tensor | None = None,
                    z: torch.Tensor | None = None, delta_bias: torch.Tensor | None = None,
                    softplus: bool = True, S0: torch.Tensor | None = None,
                    dS_out: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """Gradients of la_forward_ssm -> (dx, ddelta, dA, dBm, dCm, dD, dz, ddelta_bias, dS0),
    with None for what was not given.  dout [B,N,C] (any batch and token strides) and dS_out
    [B,C,n] (None: zero) are the gradients of out and of the final state."""
    dev = _current(x, "x")
    G, n, ptrs, strides = _ssm_inputs(x, delta, A, Bm, Cm, D, z, delta_bias, dev, 2)
    B, N, C = x.shape
    call = _Call(stream, dev)
    dop, *ds = _rows(dout, "dout", x.shape, 2, x.dtype, dev)
    f32, state = torch.float32, (B, C, n)
    ins = (dop, _arg(dS_out, "dS_out", state, f32, dev), *ptrs, _arg(S0, "S0", state, f32, dev),
           _lengths(lengths, B, dev))

    def like(t, shape, dtype):
        return call.empty(shape, dtype) if t is not None else None

    grads = (call.empty((B, N, C), x.dtype), call.empty((B, N, C), x.dtype), call.empty((C, n), f32),
             call.empty((B, N, G, n), x.dtype), call.empty((B, N, G, n), x.dtype), like(D, (C,), f32),
             like(z, (B, N, C), x.dtype), like(delta_bias, (C,), f32), like(S0, state, f32))
    ws = call.scratch(workspace, la_ssm_backward_workspace_size(B, N, C, G, n, x.dtype))
    code = _lib.la_backward_ssm(*ins, *(None if g is None else g.data_ptr() for g in grads),
                                _host_strides(strides + ds), B, N, C, G, n, int(bool(softplus)), _dtype(x),
                                *ws, call.handle)
    _check(code, "la_backward_ssm")
    return grads


def la_forward_path(B, H, N, d, dv, causal=True, feature_map="elu1", has_decay=False,
                    dtype=torch.bfloat16) -> str:
    return _lib.la_forward_path(B, H, N, d, dv, int(bool(causal)), _fm(feature_map),
                                int(bool(has_decay)), DTYPES[dtype]).decode()


def la_debug_set_tc_faults(wait_ns: int, withheld_segment: int = -1) -> None:
    """Test hook of the single-pass kernel's give-up path (see linattn.h)."""
    _check(_lib.la_debug_set_tc_faults(int(wait_ns), int(withheld_segment)),
           "la_debug_set_tc_faults")


def la_launch_count() -> int:
    return int(_lib.la_launch_count())


def la_get_device_status(stream=None) -> int:
    return int(_lib.la_get_device_status(_stream_handle(stream)))


# raw handle, for callers that want the C functions directly (tests of the ABI)
raw = _lib
