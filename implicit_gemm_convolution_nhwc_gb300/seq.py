"""Python binding of the sequence operators (include/conv_seq.h): the causal depthwise convolution along time, the
selective state-space scan and the root-mean-square norm, for prompts, training and single tokens.

As in the package's other calls, the caller owns every tensor and the workspace, nothing is allocated or synchronised, and
a failed check raises. All tensors of a call are on the current device (a library call launches there). Token tensors are [n, l, c] (single tokens: [n, c]) with the last dimension contiguous and any
other strides, so a slice of a projection's output is used in place. The formulas, the meaning of `lengths` and of `slots`
and the rules on overlap stand in the header.

    y = seq.causal_conv_fwd(x, w, y, bias, silu=True, state_out=state)
    y = seq.scan_fwd(x, dt, A, B, C, y, D=D, z=z, dt_bias=dt_bias, softplus=True, state_out=state,
                     ws=seq.scan_workspace(x, B))
    y = seq.rms_norm_fwd(x, w, y, residual=residual, residual_out=residual)
"""
from __future__ import annotations

import ctypes
import importlib.util
import struct

import torch

from . import BF16, F16, F32, ConvError, _build, _stream, load

# Every symbol include/conv_seq.h declares.
EXPORTS = ["seq_conv_fwd", "seq_conv_bwd", "seq_conv_workspace_bytes", "seq_conv_step", "seq_scan_fwd", "seq_scan_bwd",
           "seq_scan_workspace_bytes_for", "seq_scan_workspace_bytes", "seq_scan_checkpoint_bytes", "seq_scan_step",
           "seq_norm_fwd", "seq_norm_bwd", "seq_norm_workspace_bytes"]

_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_F32, _F8, _I32 = torch.float32, torch.float8_e4m3fn, torch.int32

# The scalars at the head of the header's argument structs; the tensors after them are checked and packed by
# csrc/seqcall.c, in the structs' order: (tensor, kind, shape, dtype) each.
_CONV_HEAD, _SCAN_HEAD, _NORM_HEAD = struct.Struct("=4q4i"), struct.Struct("=5q2i"), struct.Struct("=2q4ifi")
_DENSE, _VIEW, _TOKEN, _GROUPS, _TOKEN_GROUPS, _WORKSPACE, _NUMBER = range(7)
_LAYOUT = {_DENSE: "contiguous", _VIEW: "its last dimension contiguous", _TOKEN: "its last dimension contiguous",
           _GROUPS: "its last two dimensions dense", _TOKEN_GROUPS: "its last two dimensions dense",
           _WORKSPACE: "contiguous"}
_NO_VIEW = (None, _VIEW, None, None)
_NONE = (None, _DENSE, None, None)
_ZERO = (0, _NUMBER, None, None)

_calls = {}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch.cuda.current_stream without its object
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _entry(name: str):
    """(the module's call, the address of a library function)."""
    if "call" not in _calls:
        lib = load()
        spec = importlib.util.spec_from_file_location("seqcall", _build.build_seqcall())
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _calls["lib"], _calls["call"] = lib, module.call
    _calls[name] = found = _calls["call"], ctypes.cast(getattr(_calls["lib"], name), ctypes.c_void_p).value
    return found


def _device(x, name: str) -> int:
    """x's device, which has to be the current one: the library launches, and asks for the number of SMs, there."""
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{name}: a CUDA tensor is required, got one on {x.device}")
    if device != _current_device():
        raise ValueError(f"{name}: on {x.device}, but the current device is cuda:{_current_device()}")
    return device


def _call(name: str, names, stream, x, head: bytes, *items):
    call, entry = _calls.get(name) or _entry(name)
    device = _device(x, names[0])
    handle = _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)
    st = call(entry, handle, device, head, *items)
    if st > 0:
        raise ConvError(st, name)
    if st < 0:
        t, kind, shape, dtype = items[4 * (-1 - st):4 * (-st)]
        what = "" if kind == _WORKSPACE else f" {tuple(shape)} of {dtype},"
        raise ValueError(f"{names[-1 - st]}: a tensor{what} {_LAYOUT[kind]}, on cuda:{device} is required, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device} with strides {t.stride()}")


def _bytes(name: str, *sizes) -> int:
    fn = _calls.get(name)
    if fn is None:
        fn = getattr(load(), name)
        fn.argtypes = [ctypes.c_int64] * min(len(sizes), 5) + [ctypes.c_int32] * max(len(sizes) - 5, 0) + [ctypes.c_void_p]
        fn.restype = ctypes.c_int
        _calls[name] = fn
    out = ctypes.c_uint64()
    st = fn(*sizes, ctypes.addressof(out))
    if st != 0:
        raise ConvError(st, name)
    return out.value


def _code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: {t.dtype} is not a type the library takes")
    return code


def _scratch(nbytes: int, device):
    return None if nbytes == 0 else torch.empty(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------ causal convolution


def _conv_head(x, w, silu, rows: int):
    shape = x.shape
    if len(shape) != rows:
        raise ValueError(f"x: {rows} dimensions are required, got {len(shape)}")
    taps = w.shape
    if len(taps) != 2 or taps[0] != shape[-1]:
        raise ValueError(f"w: [channels, width] is required, got {tuple(taps)}")
    n, l, c = shape if rows == 3 else (shape[0], 1, shape[1])
    width = taps[1]
    return shape, taps, n, c, (n, width - 1, c), _CONV_HEAD.pack(n, l, c, width, _code(x, "x"), _code(w, "w"),
                                                                1 if silu else 0, 0)


_CONV_NAMES = ("x", "y", "dy", "dx", "w", "bias", "state", "state_out", "lengths", "dstate_out", "dstate", "dw", "db",
               "slots", "n_slots", "ws")
_CONV_STEP_NAMES = _CONV_NAMES[:7] + ("state",) + _CONV_NAMES[8:]


def causal_conv_fwd(x, w, y, bias=None, *, silu=False, state=None, state_out=None, lengths=None, stream=None):
    """y[t] = act(bias + sum_j w[:, j] x[t - (width-1) + j]) for x [n, l, c] and w [c, width], width 1..4. `state` holds the
    width-1 tokens before the first ([n, width-1, c]; zeros without it), `state_out` gets those before the next."""
    shape, taps, n, c, kept, head = _conv_head(x, w, silu, 3)
    dtype, wtype = x.dtype, w.dtype
    _call("seq_conv_fwd", _CONV_NAMES, stream, x, head, x, _VIEW, shape, dtype, y, _VIEW, shape, dtype, *_NO_VIEW, *_NO_VIEW,
          w, _DENSE, taps, wtype, bias, _DENSE, (c,), wtype, state, _DENSE, kept, dtype, state_out, _DENSE, kept, dtype,
          lengths, _DENSE, (n,), _I32, *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, *_ZERO, None, _WORKSPACE, None, None)
    return y


def causal_conv_workspace_bytes(n: int, l: int, c: int, width: int) -> int:
    return _bytes("seq_conv_workspace_bytes", n, l, c, width)


def causal_conv_workspace(x, w):
    """The backward pass's workspace for x [n, l, c] and w [c, width]."""
    return _scratch(causal_conv_workspace_bytes(*x.shape, w.shape[1]), x.device)


def causal_conv_bwd(x, w, dy, dx, dw, bias=None, db=None, *, silu=False, state=None, dstate_out=None, dstate=None,
                    lengths=None, ws=None, stream=None):
    """Gradients of causal_conv_fwd: dx like x, dw [c, width] and db [c] in fp32, dstate like state. `dstate_out` is the
    gradient that arrives at state_out."""
    shape, taps, n, c, kept, head = _conv_head(x, w, silu, 3)
    dtype, wtype = x.dtype, w.dtype
    _call("seq_conv_bwd", _CONV_NAMES, stream, x, head, x, _VIEW, shape, dtype, *_NO_VIEW, dy, _VIEW, shape, dtype,
          dx, _VIEW, shape, dtype, w, _DENSE, taps, wtype, bias, _DENSE, (c,), wtype, state, _DENSE, kept, dtype, *_NONE,
          lengths, _DENSE, (n,), _I32, dstate_out, _DENSE, kept, dtype, dstate, _DENSE, kept, dtype, dw, _DENSE, taps, _F32,
          db, _DENSE, (c,), _F32, *_NONE, *_ZERO, ws, _WORKSPACE, None, None)
    return dx, dw, db


def causal_conv_step(x, w, state, y, bias=None, *, silu=False, slots=None, stream=None):
    """One token of each sequence: x, y [n, c]. `state` [pool, width-1, c] moves on in place; sequence i uses entry slots[i]
    (entry i without slots), and a slot outside the pool marks an empty row, whose y is 0."""
    shape, taps, n, c, kept, head = _conv_head(x, w, silu, 2)
    dtype, wtype, pool = x.dtype, w.dtype, state.shape[0]
    _call("seq_conv_step", _CONV_STEP_NAMES, stream, x, head, x, _TOKEN, shape, dtype, y, _TOKEN, shape, dtype, *_NO_VIEW,
          *_NO_VIEW, w, _DENSE, taps, wtype, bias, _DENSE, (c,), wtype, *_NONE, state, _DENSE, (pool, *kept[1:]), dtype,
          *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, slots, _DENSE, (n,), _I32, pool, _NUMBER, None, None,
          None, _WORKSPACE, None, None)
    return y


# ------------------------------------------------------------ selective scan


def _scan_head(x, B, softplus, rows: int):
    shape, bc = x.shape, B.shape
    if len(shape) != rows:
        raise ValueError(f"x: {rows} dimensions are required, got {len(shape)}")
    if len(bc) != rows + 1 or bc[:-2] != shape[:-1]:
        raise ValueError(f"B: {(*shape[:-1], 'groups', 'states')} is required, got {tuple(bc)}")
    n, l, c = shape if rows == 3 else (shape[0], 1, shape[1])
    s = bc[-1]
    return shape, bc, n, l, c, s, _SCAN_HEAD.pack(n, l, c, s, bc[-2], _code(x, "x"), 1 if softplus else 0)


_SCAN_NAMES = ("x", "dt", "z", "B", "C", "y", "A", "D", "dt_bias", "state", "state_out", "lengths", "checkpoints", "dy",
               "dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dstate_out", "dstate", "slots", "n_slots", "ws")
_SCAN_STEP_NAMES = _SCAN_NAMES[:10] + ("state",) + _SCAN_NAMES[11:]


def scan_workspace_bytes(n: int, l: int, c: int, s: int, g: int = 1, backward: bool = False,
                         sm_count: int | None = None) -> int:
    if sm_count is None:
        return _bytes("seq_scan_workspace_bytes", n, l, c, s, g, int(backward))
    return _bytes("seq_scan_workspace_bytes_for", n, l, c, s, g, int(backward), sm_count)


def scan_workspace(x, B, backward: bool = False):
    """The workspace for x [n, l, c] and B [n, l, g, s]: of the forward pass, or one that serves both (backward=True)."""
    _device(x, "x")
    return _scratch(scan_workspace_bytes(*x.shape, B.shape[3], B.shape[2], backward), x.device)


def _checkpoint_floats(n: int, l: int, c: int, s: int) -> int:
    return _bytes("seq_scan_checkpoint_bytes", n, l, c, s) // 4


def scan_checkpoints(x, B):
    """Room for the states that the forward pass keeps for the backward pass."""
    return torch.empty(_checkpoint_floats(*x.shape, B.shape[3]), dtype=_F32, device=x.device)


def scan_fwd(x, dt, A, B, C, y, *, D=None, z=None, dt_bias=None, softplus=False, state=None, state_out=None,
             checkpoints=None, lengths=None, ws=None, stream=None):
    """h[t] = exp(delta A) h[t-1] + delta x B, y = (C . h + D x) silu(z) with delta = dt + dt_bias or its softplus, over
    x, dt, z [n, l, c], B, C [n, l, g, s], A [c, s]. state and state_out are [n, c, s] in fp32 (16-byte aligned where s is a
    multiple of 4, as all states of the scan)."""
    shape, bc, n, l, c, s, head = _scan_head(x, B, softplus, 3)
    dtype, kept, per = x.dtype, (n, c, s), (c,)
    _call("seq_scan_fwd", _SCAN_NAMES, stream, x, head, x, _VIEW, shape, dtype, dt, _VIEW, shape, dtype, z, _VIEW, shape, dtype,
          B, _GROUPS, bc, dtype, C, _GROUPS, bc, dtype, y, _VIEW, shape, dtype, A, _DENSE, (c, s), _F32, D, _DENSE, per, _F32,
          dt_bias, _DENSE, per, _F32, state, _DENSE, kept, _F32, state_out, _DENSE, kept, _F32, lengths, _DENSE, (n,), _I32,
          *_kept(checkpoints, n, l, c, s), *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW,
          *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, *_ZERO, ws, _WORKSPACE, None, None)
    return y


def _kept(checkpoints, n, l, c, s):
    if checkpoints is None:
        return _NONE
    return checkpoints, _DENSE, (_checkpoint_floats(n, l, c, s),), _F32


def scan_bwd(x, dt, A, B, C, dy, checkpoints, dx, ddt, dA, dB, dC, *, D=None, dD=None, z=None, dz=None, dt_bias=None,
             ddt_bias=None, softplus=False, dstate_out=None, dstate=None, lengths=None, ws=None, stream=None):
    """Gradients of scan_fwd with the same arguments, from the checkpoints it wrote: dx, ddt, dz, dB, dC like their
    tensors; dA, dD, ddt_bias and dstate in fp32. `dstate_out` is the gradient that arrives at state_out."""
    shape, bc, n, l, c, s, head = _scan_head(x, B, softplus, 3)
    dtype, kept, per = x.dtype, (n, c, s), (c,)
    _call("seq_scan_bwd", _SCAN_NAMES, stream, x, head, x, _VIEW, shape, dtype, dt, _VIEW, shape, dtype, z, _VIEW, shape, dtype,
          B, _GROUPS, bc, dtype, C, _GROUPS, bc, dtype, *_NO_VIEW, A, _DENSE, (c, s), _F32, D, _DENSE, per, _F32,
          dt_bias, _DENSE, per, _F32, *_NONE, *_NONE, lengths, _DENSE, (n,), _I32, *_kept(checkpoints, n, l, c, s),
          dy, _VIEW, shape, dtype, dx, _VIEW, shape, dtype, ddt, _VIEW, shape, dtype, dz, _VIEW, shape, dtype,
          dB, _GROUPS, bc, dtype, dC, _GROUPS, bc, dtype, dA, _DENSE, (c, s), _F32, dD, _DENSE, per, _F32,
          ddt_bias, _DENSE, per, _F32, dstate_out, _DENSE, kept, _F32, dstate, _DENSE, kept, _F32, *_NONE, *_ZERO,
          ws, _WORKSPACE, None, None)
    return dx, ddt, dA, dB, dC


def scan_step(x, dt, A, B, C, state, y, *, D=None, z=None, dt_bias=None, softplus=False, slots=None, stream=None):
    """One token of each sequence: x, dt, z, y [n, c], B, C [n, g, s]. `state` [pool, c, s] in fp32 moves on in place;
    slots as for causal_conv_step."""
    shape, bc, n, l, c, s, head = _scan_head(x, B, softplus, 2)
    dtype, per, pool = x.dtype, (c,), state.shape[0]
    _call("seq_scan_step", _SCAN_STEP_NAMES, stream, x, head, x, _TOKEN, shape, dtype, dt, _TOKEN, shape, dtype,
          z, _TOKEN, shape, dtype, B, _TOKEN_GROUPS, bc, dtype, C, _TOKEN_GROUPS, bc, dtype, y, _TOKEN, shape, dtype,
          A, _DENSE, (c, s), _F32, D, _DENSE, per, _F32, dt_bias, _DENSE, per, _F32, *_NONE,
          state, _DENSE, (pool, c, s), _F32, *_NONE, *_NONE, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW,
          *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, slots, _DENSE, (n,), _I32, pool, _NUMBER, None, None,
          None, _WORKSPACE, None, None)
    return y


# ------------------------------------------------------------ root-mean-square norm


_NORM_NAMES = ("x", "residual", "y", "residual_out", "dy", "dresidual", "dx", "w", "scale", "rstd", "dw", "ws")
_NORM_BWD_NAMES = _NORM_NAMES[:3] + ("r",) + _NORM_NAMES[4:]


def rms_norm_fwd(x, w, y, *, residual=None, residual_out=None, scale=None, group=0, eps=1e-6, rstd=None, stream=None):
    """r = x + residual, y = r / sqrt(mean(r^2) + eps) * w over rows x [n, c]. r goes to residual_out (which may be x or
    residual), 1 / sqrt(..) to rstd [n] for the backward pass. A y of torch.float8_e4m3fn gets q = y / scale with scale =
    max |y| / 448 of each row (scale [n, 1], group 0) or of each `group` columns (32, 64 or 128; scale [n, ceil(c / group)])."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x: [rows, columns] is required, got {tuple(shape)}")
    n, c = shape
    out8 = y.dtype is _F8
    if (scale is not None) != out8:
        raise ValueError("scale: required for 8-bit outputs and for them alone")
    head = _NORM_HEAD.pack(n, c, _code(x, "x"), _code(w, "w"), out8, group, eps, 0)
    parts = (n, -(-c // group) if group > 0 else 1)
    _call("seq_norm_fwd", _NORM_NAMES, stream, x, head, x, _TOKEN, shape, dtype, residual, _TOKEN, shape, dtype,
          y, _TOKEN, shape, _F8 if out8 else dtype, residual_out, _TOKEN, shape, dtype, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW,
          w, _DENSE, (c,), w.dtype, scale, _DENSE, parts, _F32, rstd, _DENSE, (n,), _F32, *_NONE, None, _WORKSPACE, None, None)
    return y


def rms_norm_workspace_bytes(n: int, c: int) -> int:
    return _bytes("seq_norm_workspace_bytes", n, c)


def rms_norm_workspace(x):
    """The backward pass's workspace for rows x [n, c]."""
    return _scratch(rms_norm_workspace_bytes(*x.shape), x.device)


def rms_norm_bwd(r, w, rstd, dy, dx, dw, *, dresidual=None, ws=None, stream=None):
    """Gradients of rms_norm_fwd from r (residual_out, or x without a residual) and rstd: dx [n, c] is the gradient of x and
    of residual alike, with `dresidual`, the gradient that arrives at residual_out, added (dx may be dresidual itself);
    dw [c] in fp32."""
    shape, dtype = r.shape, r.dtype
    if len(shape) != 2:
        raise ValueError(f"r: [rows, columns] is required, got {tuple(shape)}")
    n, c = shape
    head = _NORM_HEAD.pack(n, c, _code(r, "r"), _code(w, "w"), 0, 0, 0.0, 0)
    _call("seq_norm_bwd", _NORM_BWD_NAMES, stream, r, head, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, r, _TOKEN, shape, dtype,
          dy, _TOKEN, shape, dtype, dresidual, _TOKEN, shape, dtype, dx, _TOKEN, shape, dtype, w, _DENSE, (c,), w.dtype,
          *_NONE, rstd, _DENSE, (n,), _F32, dw, _DENSE, (c,), _F32, ws, _WORKSPACE, None, None)
    return dx, dw
