"""The sequence operators' binding without a GPU: stand-in tensors that say which device they are on, and entries that are
functions of this process in the library's place."""
import ctypes
import inspect
import os
import struct
import sysconfig
import threading
import time

import pytest
import torch

import implicit_gemm_convolution_nhwc_gb300 as cig
import test_seq_host as host
from implicit_gemm_convolution_nhwc_gb300 import _build, seq


class Stand:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self.like = torch.empty(shape, dtype=dtype, device="meta")
        self.on = device

    shape = property(lambda self: self.like.shape)
    dtype = property(lambda self: self.like.dtype)
    nbytes = property(lambda self: self.like.nbytes)
    is_cuda = property(lambda self: self.on >= 0)
    device = property(lambda self: torch.device("cuda", self.on) if self.on >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.on

    def stride(self):
        return self.like.stride()

    def data_ptr(self):
        return 1 << 20


N, L, C, W, S = 2, 4, 8, 4, 4


def _t(*shape, **kw):
    return Stand(*shape, **kw)


def tok():
    return _t(N, L, C)


def one():
    return _t(N, C)


def vec():
    return _t(C)


I32 = torch.int32
CALLS = {  # the binding's function: its arguments, every tensor among them
    "causal_conv_fwd": lambda: dict(x=tok(), w=_t(C, W), y=tok(), bias=vec(), state=_t(N, W - 1, C), state_out=_t(N, W - 1, C),
                                    lengths=_t(N, dtype=I32)),
    "causal_conv_bwd": lambda: dict(x=tok(), w=_t(C, W), dy=tok(), dx=tok(), dw=_t(C, W), bias=vec(), db=vec(),
                                    state=_t(N, W - 1, C), dstate_out=_t(N, W - 1, C), dstate=_t(N, W - 1, C),
                                    lengths=_t(N, dtype=I32), ws=_t(64, dtype=torch.uint8)),
    "causal_conv_step": lambda: dict(x=one(), w=_t(C, W), state=_t(5, W - 1, C), y=one(), bias=vec(), slots=_t(N, dtype=I32)),
    "scan_fwd": lambda: dict(x=tok(), dt=tok(), A=_t(C, S), B=_t(N, L, 1, S), C=_t(N, L, 1, S), y=tok(), D=vec(), z=tok(),
                             dt_bias=vec(), state=_t(N, C, S), state_out=_t(N, C, S), checkpoints=_t(N * C * S),
                             lengths=_t(N, dtype=I32), ws=_t(64)),
    "scan_bwd": lambda: dict(x=tok(), dt=tok(), A=_t(C, S), B=_t(N, L, 1, S), C=_t(N, L, 1, S), dy=tok(),
                             checkpoints=_t(N * C * S), dx=tok(), ddt=tok(), dA=_t(C, S), dB=_t(N, L, 1, S), dC=_t(N, L, 1, S),
                             D=vec(), dD=vec(), z=tok(), dz=tok(), dt_bias=vec(), ddt_bias=vec(), dstate_out=_t(N, C, S),
                             dstate=_t(N, C, S), lengths=_t(N, dtype=I32), ws=_t(64)),
    "scan_step": lambda: dict(x=one(), dt=one(), A=_t(C, S), B=_t(N, 1, S), C=_t(N, 1, S), state=_t(5, C, S), y=one(), D=vec(),
                              z=one(), dt_bias=vec(), slots=_t(N, dtype=I32)),
    "rms_norm_fwd": lambda: dict(x=one(), w=vec(), y=_t(N, C, dtype=torch.float8_e4m3fn), residual=one(), residual_out=one(),
                                 scale=_t(N, 1), rstd=_t(N)),
    "rms_norm_bwd": lambda: dict(r=one(), w=vec(), rstd=_t(N), dy=one(), dx=one(), dw=vec(), dresidual=one(), ws=_t(64)),
}
ENTRY = {"causal_conv": "seq_conv", "scan": "seq_scan", "rms_norm": "seq_norm"}


@pytest.fixture
def reached(monkeypatch):
    """The calls that reach the library, which is a function of this process here."""
    seen = []
    fn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)(lambda args, stream: seen.append(args) or 0)
    call, _ = seq._entry("seq_conv_fwd")
    for name in seq.EXPORTS:
        if "bytes" not in name:
            monkeypatch.setitem(seq._calls, name, (call, ctypes.cast(fn, ctypes.c_void_p).value))
    monkeypatch.setattr(seq, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(seq, "_raw_stream", lambda device: 0)
    yield seen
    del fn


@pytest.mark.parametrize("name", CALLS)
def test_calls_reach_the_library_on_the_current_device(name, reached):
    args = CALLS[name]()
    taken = [k for k, p in inspect.signature(getattr(seq, name)).parameters.items() if p.default is inspect.Parameter.empty]
    assert set(taken) <= set(args)
    getattr(seq, name)(**args)
    assert len(reached) == 1


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [1, -1])
def test_a_tensor_of_another_device_is_refused(name, device, reached):
    for which in CALLS[name]():
        args = CALLS[name]()
        args[which].on = device
        with pytest.raises(ValueError, match="on cuda:0|a CUDA tensor|current device"):
            getattr(seq, name)(**args)
        assert not reached, which


@pytest.mark.parametrize("name", CALLS)
def test_tensors_that_are_not_on_the_current_device_are_refused(name, reached):
    args = CALLS[name]()
    for t in args.values():
        t.on = 1
    with pytest.raises(ValueError, match="current device is cuda:0"):
        getattr(seq, name)(**args)
    assert not reached


def test_a_scan_workspace_is_sized_for_the_tensors_device(monkeypatch):
    monkeypatch.setattr(seq, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        seq.scan_workspace(_t(N, L, C, device=1), _t(N, L, 1, S, device=1))


def test_other_threads_run_while_the_library_is_called():
    """A launch may wait for room in the stream's queue, and a host function in front of it for the interpreter: the lock is
    not held meanwhile. nanosleep(const timespec*, timespec*) has the shape of an entry."""
    call, _ = seq._entry("seq_conv_fwd")
    sleep = ctypes.cast(ctypes.CDLL(None).nanosleep, ctypes.c_void_p).value
    ticks, done = [], threading.Event()

    def tick():
        while not done.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.005)

    other = threading.Thread(target=tick)
    other.start()
    try:
        begin = time.monotonic()
        assert call(sleep, 0, 0, struct.pack("qq", 0, 400_000_000)) == 0
        end = time.monotonic()
    finally:
        done.set()
        other.join()
    assert end - begin >= 0.4
    assert sum(begin + 0.1 < t < end - 0.1 for t in ticks) > 3


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    """A machine without a C compiler, on which the binding's module was never built."""
    cig.load()
    which = _build.shutil.which
    monkeypatch.setattr(_build.shutil, "which", lambda name, *a, **kw: None if name in ("cc", "gcc") else which(name, *a, **kw))
    monkeypatch.setattr(_build, "SEQCALL", str(tmp_path / "seqcall.so"))
    monkeypatch.setattr(seq, "_calls", {})


def test_the_library_needs_no_c_compiler(no_module):
    assert _build.up_to_date()
    assert _build.build() == _build.LIB
    assert cig.load(build_if_missing=False) is not None
    assert cig.output_dims(cig.Problem(n=1, h=8, w=8, c=4, k=4)) == (8, 8)


def test_the_sequence_operators_name_what_their_module_lacks(no_module):
    with pytest.raises(RuntimeError, match="C compiler"):
        seq._entry("seq_conv_fwd")


def test_the_module_belongs_to_this_interpreter():
    assert os.path.basename(_build.SEQCALL) == "seqcall" + sysconfig.get_config_var("EXT_SUFFIX")


@pytest.mark.parametrize("name", ["seq_conv_step", "seq_scan_step", "seq_conv_fwd"])
def test_strides_of_a_single_token_or_sequence_are_not_looked_at(name):
    """They have no meaning there, and the steps' are documented as not used. (What passes the checks fails at the launch
    here, where there is no GPU.)"""
    any_stride = host._Tensor(host.PTR, -1 if name == "seq_conv_fwd" else 16, 16 if name == "seq_conv_fwd" else -3)
    sizes = dict(n=1, l=2, c=16) if name == "seq_conv_fwd" else dict(n=2, l=1, c=16)
    make = host._conv if "conv" in name else host._scan
    views = ("x", "y") if "conv" in name else ("x", "dt", "z", "b", "cc", "y")
    args = make(**sizes, state_out=host.PTR, n_slots=2, **{k: any_stride for k in views})
    assert host._status(name, args) == cig.STATUS.index("CONV_ERR_CUDA")
