"""Past a sequence's length gradients are 0 whatever the weights, the states and their gradients hold: infinity times 0 does
not come through."""
import pytest
import torch

from implicit_gemm_convolution_nhwc_gb300 import seq
from test_gpu_seq import BF16, F32, Gen, ws_nan

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype, c", [(BF16, 64), (F32, 7)])
@pytest.mark.parametrize("l, lengths", [(21, [5, 0, 21, 2]), (300, [130, 0, 129, 1])])
def test_conv_gradients(dtype, c, l, lengths):
    n, width = len(lengths), 4
    g = Gen(l)
    x, dy = g.normal(n, l, c, dtype=dtype).cuda(), g.normal(n, l, c, dtype=dtype).cuda()
    w = g.normal(c, width, dtype=F32).cuda()
    w[1, 0], w[2, 1], w[3, 3] = INF, NAN, -INF
    kept = g.normal(n, width - 1, c, dtype=dtype).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for arriving in (None, kept):
        dx, dw, dst = torch.full_like(x, 3), torch.empty_like(w), torch.full_like(kept, 3)
        seq.causal_conv_bwd(x, w, dy, dx, dw, dstate=dst, dstate_out=arriving, lengths=lens,
                            ws=ws_nan(seq.causal_conv_workspace_bytes(n, l, c, width)))
        for i, ln in enumerate(lengths):
            assert bool((dx[i, ln:] == 0).all()), i
            if ln == 0:  # the state passes by
                assert torch.equal(dst[i], torch.zeros_like(dst[i]) if arriving is None else kept[i])
        plain = [k for k in range(c) if k not in (1, 2, 3)]
        assert bool(torch.isfinite(dx[..., plain]).all()) and bool(torch.isfinite(dw[plain]).all())


@pytest.mark.parametrize("dtype, c, s", [(BF16, 64, 16), (F32, 5, 3), (BF16, 16, 64)])
@pytest.mark.parametrize("l, lengths", [(21, [5, 0, 21]), (333, [130, 47, 0])])
def test_scan_gradients(dtype, c, s, l, lengths):
    n = len(lengths)
    g = Gen(l + s)
    x, dt, dy = (g.normal(n, l, c, dtype=dtype).cuda() for _ in range(3))
    B, C = (g.normal(n, l, 1, s, dtype=dtype).cuda() for _ in range(2))
    A = -g.uniform(0.3, 1.0, c, s).cuda()
    state, arriving = g.normal(n, c, s, dtype=F32).cuda(), g.normal(n, c, s, dtype=F32).cuda()
    state[:, 1, 0], arriving[:, 2, 1], arriving[:, 0, 2] = INF, -INF, NAN
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, end = torch.empty_like(x), torch.empty_like(state)
    kept = seq.scan_checkpoints(x, B)
    ws = ws_nan(seq.scan_workspace_bytes(n, l, c, s, 1, True))
    seq.scan_fwd(x, dt, A, B, C, y, softplus=True, state=state, state_out=end, checkpoints=kept, lengths=lens, ws=ws)
    dx, ddt, dB, dC = (torch.full_like(v, 3) for v in (x, dt, B, C))
    dA, dst = torch.empty_like(A), torch.empty_like(state)
    seq.scan_bwd(x, dt, A, B, C, dy, kept, dx, ddt, dA, dB, dC, softplus=True, dstate_out=arriving, dstate=dst, lengths=lens,
                 ws=ws)
    for i, ln in enumerate(lengths):
        for name, v in dict(y=y, dx=dx, ddt=ddt, dB=dB, dC=dC).items():
            assert bool((v[i, ln:] == 0).all()), (name, i)
        if ln == 0:
            assert torch.equal(end[i], state[i]) and torch.equal(dst[i].nan_to_num(), arriving[i].nan_to_num())
