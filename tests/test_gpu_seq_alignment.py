"""Parameters of the sequence operators that stand where their element's alignment allows and no more: contiguous slices of
one flat buffer, as an optimiser keeps them, at every offset up to 16 bytes. Tolerances as in test_gpu_seq.py."""
import pytest
import torch

import seq_reference as ref
from implicit_gemm_convolution_nhwc_gb300 import seq
from test_gpu_seq import BF16, F16, F32, Gen, close, ws_nan

pytestmark = pytest.mark.gpu


def at_offset(t, offset):
    """t on the GPU, contiguous, from element `offset` of a 16-byte aligned buffer on."""
    buf = torch.empty(t.numel() + offset + 16, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and (not v.numel() or v.data_ptr() % 16 == offset * t.element_size() % 16)
    return v


CONV = [(dtype, wt, width, c) for dtype, wt in ((F32, F32), (BF16, F32), (F16, F32), (BF16, BF16)) for width, c in
        ((4, 16), (4, 7), (3, 16), (2, 24), (1, 8))]


@pytest.mark.parametrize("dtype, wt, width, c", CONV)
@pytest.mark.parametrize("offset", [1, 2, 3, 4])
def test_conv_filter_and_bias_at_odd_offsets(dtype, wt, width, c, offset):
    n, l = 2, 37
    g = Gen(width + c + offset)
    x, dy = g.normal(n, l, c, dtype=dtype), g.normal(n, l, c, dtype=dtype)
    w, b = g.normal(c, width, dtype=wt, scale=0.6), g.normal(c, dtype=wt)
    state = g.normal(n, width - 1, c, dtype=dtype)
    wd, bd, sd = at_offset(w, offset), at_offset(b, 4 - offset), at_offset(state, offset)
    y = torch.empty(n, l, c, dtype=dtype, device="cuda")
    kept = at_offset(torch.zeros_like(state), offset)
    seq.causal_conv_fwd(x.cuda(), wd, y, bd, silu=True, state=sd, state_out=kept)
    want, end, _ = ref.conv_fwd(x, w, b, True, state)
    mag = ref.conv_fwd(x.abs(), w.abs(), b.abs(), False, state.abs())[0]
    close(y, want, mag, 16, "y")
    assert torch.equal(kept.cpu().double(), end)

    dx = torch.empty_like(y)
    dw, db, dst = at_offset(torch.zeros(c, width), offset), at_offset(torch.zeros(c), 1), at_offset(torch.zeros_like(state), offset)
    seq.causal_conv_bwd(x.cuda(), wd, dy.cuda(), dx, dw, bd, db, silu=True, state=sd, dstate=dst,
                        ws=ws_nan(seq.causal_conv_workspace_bytes(n, l, c, width)))
    want = ref.conv_bwd(x, w, dy, b, True, state)
    mags = ref.conv_bwd(x, w, dy, b, False, state, mag=True)
    for name, got, e, m in zip(("dx", "dw", "db", "dstate"), (dx, dw, db, dst), want, mags):
        close(got, e, m * (2 + float(mag.max())), 16, name)

    pool = at_offset(state, offset)
    yt = torch.empty(n, c, dtype=dtype, device="cuda")
    seq.causal_conv_step(x[:, 0].cuda(), wd, pool, yt, bd, silu=True)
    one, moved, _ = ref.conv_fwd(x[:, :1], w, b, True, state)
    close(yt, one[:, 0], mag[:, 0], 16, "token's y")
    assert torch.equal(pool.cpu().double(), moved)


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("s", [4, 16, 5])
def test_scan_parameters_at_odd_offsets(s, offset):
    n, l, c = 2, 21, 16
    g = Gen(s + offset)
    x, dt, B, C = (g.normal(n, l, *k, dtype=F32) for k in ((c,), (c,), (1, s), (1, s)))
    A, D, bias = -g.uniform(0.3, 2.0, c, s), g.uniform(0.5, 1.5, c), g.uniform(-3.0, -1.0, c)
    Ad, Dd, bd = at_offset(A, offset), at_offset(D, offset), at_offset(bias, offset)
    kw = dict(D=Dd, dt_bias=bd, softplus=True)
    pos = [x.cuda(), dt.cuda(), Ad, B.cuda(), C.cuda()]
    y, end = torch.empty(n, l, c, device="cuda"), torch.zeros(n, c, s, device="cuda")
    kept = seq.scan_checkpoints(pos[0], pos[3])
    ws = ws_nan(seq.scan_workspace_bytes(n, l, c, s, 1, True))
    seq.scan_fwd(*pos, y, state_out=end, checkpoints=kept, ws=ws, **kw)
    rk = dict(D=D, dt_bias=bias, softplus=True)
    want, h, *_ = ref.scan_fwd(x, dt, A, B, C, **rk)
    my, mh, *_ = ref.scan_fwd(x, dt, A, B, C, **rk, mag=True)
    close(y, want, my, 16 + l, "y")
    close(end, h, mh, 16 + l, "state_out")
    dy = g.normal(n, l, c, dtype=F32)
    got = {k: torch.empty(n, l, c, device="cuda") for k in ("dx", "ddt")}
    got.update(dB=torch.empty_like(pos[3]), dC=torch.empty_like(pos[4]), dA=at_offset(torch.zeros(c, s), offset),
               dD=at_offset(torch.zeros(c), offset), ddt_bias=at_offset(torch.zeros(c), offset))
    seq.scan_bwd(*pos, dy.cuda(), kept, got["dx"], got["ddt"], got["dA"], got["dB"], got["dC"], dD=got["dD"],
                 ddt_bias=got["ddt_bias"], ws=ws, **kw)
    want = ref.scan_bwd(x, dt, A, B, C, dy, **rk)
    mag = ref.scan_bwd(x, dt, A, B, C, dy, **rk, mag=True)
    for k, v in got.items():
        close(v, want[k], mag[k], 16 + 2 * l, k)
    pool, yt = torch.zeros(n, c, s, device="cuda"), torch.empty(n, c, device="cuda")
    seq.scan_step(pos[0][:, 0], pos[1][:, 0], Ad, pos[3][:, 0], pos[4][:, 0], pool, yt, **kw)
    one, h, *_ = ref.scan_fwd(x[:, :1], dt[:, :1], A, B[:, :1], C[:, :1], **rk)
    close(yt, one[:, 0], my, 20, "token's y")
    close(pool, h, mh, 20, "token's state")


@pytest.mark.parametrize("dtype, wt", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("c", [64, 2048, 4104])
def test_norm_weights_at_odd_offsets(dtype, wt, c):
    n = 5
    g = Gen(c)
    x, w, dy = g.normal(n, c, dtype=dtype), g.normal(c, dtype=wt, scale=0.2, mean=1.0), g.normal(n, c, dtype=dtype)
    want, kept, rs = ref.norm_fwd(x, w, None, 1e-5)
    wx, ww = ref.norm_bwd(x, w, dy, None, 1e-5)
    hat = kept.abs() * rs[:, None]
    dh = (dy.double() * w.double()).abs()
    mx = rs[:, None] * (dh + hat * (dh * hat).mean(-1, keepdim=True))
    for offset in (1, 4):  # not a multiple of 16 bytes; of 16 but not of 32
        wd = at_offset(w, offset)
        y, dx = torch.empty(n, c, dtype=dtype, device="cuda"), torch.empty(n, c, dtype=dtype, device="cuda")
        rstd, dw = at_offset(torch.zeros(n), 1), at_offset(torch.zeros(c), 1)
        seq.rms_norm_fwd(x.cuda(), wd, y, rstd=rstd, eps=1e-5)
        close(y, want, want, 24, "y")
        seq.rms_norm_bwd(x.cuda(), wd, rstd, dy.cuda(), dx, dw, ws=ws_nan(seq.rms_norm_workspace_bytes(n, c)))
        close(dx, wx, mx, 24, "dx")
        close(dw, ww, (dy.double().abs() * hat).sum(0), 24, "dw")
