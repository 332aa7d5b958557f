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
