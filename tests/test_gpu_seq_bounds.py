"""GPU parity of the sequence operators element by element: every element against 64 bits within its own bound on fp32's error
(seq_bounds.py), plus half a spacing of the output's type, twice for a value that rounds the other way."""
import pytest
import torch

import seq_bounds as bounds
import seq_reference as ref
from implicit_gemm_convolution_nhwc_gb300 import seq
from test_gpu_seq import BF16, F16, F32, HALF, Gen, ws_nan

pytestmark = pytest.mark.gpu
SUBNORMAL = {BF16: 0.0, F16: 2.0 ** -24, F32: 0.0}  # fp16's spacing near 0


def within(got, want, name):
    """got is as near to want.v as its bound says, in each element."""
    assert got.shape == want.v.shape, name
    d = got.double()
    assert bool(torch.isfinite(d).all()), f"{name}: not finite"
    limit = HALF[got.dtype] * want.v.abs() + SUBNORMAL[got.dtype] + bounds.U * want.err + 1e-30 * (1 + want.mag)
    over = (d - want.v).abs() - limit
    at = int(over.argmax())
    assert float(over.max()) <= 0, (f"{name}[{at}]: {float(d.flatten()[at]):.9g}, {float(want.v.flatten()[at]):.9g} within "
                                    f"{float(limit.expand_as(d).flatten()[at]):.3g}")


# n, l, c, s, g, dtype, softplus, lengths, decays; span: tokens whose deltas a cut time axis adds up
SCAN = [
    (2, 100, 32, 16, 1, F32, True, None, "spread", 100),
    (2, 100, 32, 16, 1, BF16, True, [100, 63], "spread", 100),
    (1, 333, 48, 16, 3, F32, True, None, "spread", 333),
    (1, 515, 24, 8, 1, F32, True, [515], "slow", 515),
    (1, 515, 24, 16, 1, F16, True, [500], "slow", 515),
    (1, 515, 24, 16, 1, F32, True, None, "fast", 515),
    (2, 333, 40, 64, 2, F32, True, [333, 1], "spread", 333),
    (2, 200, 40, 24, 1, BF16, False, None, "spread", 200),
    (1, 400, 9, 5, 1, F32, False, [399], "slow", 400),
    (3, 130, 700, 4, 7, F32, True, [130, 0, 77], "even", 130),
    # enough sequences that the time axis is not cut, in the forward and in the backward pass
    (160, 130, 130, 16, 1, F32, True, None, "spread", 0),
    (20, 200, 2048, 16, 1, BF16, True, None, "even", 0),
    (20, 97, 2048, 8, 2, F32, True, "some", "spread", 0),
    (40, 97, 1040, 32, 1, F16, True, "some", "even", 0),
]


def _decays(kind, c, s, g):
    if kind == "slow":   # states that live through all tokens
        return -g.uniform(1e-6, 1e-3, c, s)
    if kind == "fast":   # gone within a token, some wholly
        return -torch.logspace(1, 4, s).expand(c, s).contiguous()
    if kind == "spread":
        return -torch.logspace(-4, 3, s).expand(c, s).contiguous()
    return -g.uniform(0.3, 1.0, c, s) * torch.arange(1, s + 1).float()


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(str(v) for v in c if not isinstance(v, list)))
def test_scan(case):
    n, l, c, s, groups, dtype, softplus, lengths, kind, span = case
    g = Gen(l + s)
    if lengths == "some":
        lengths = torch.randint(0, l + 1, (n,), generator=g.g).tolist()
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    t = dict(x=g.normal(n, l, c, dtype=dtype),
             dt=g.normal(n, l, c, dtype=dtype, scale=0.5) if softplus else g.uniform(0.001, 0.1, n, l, c, dtype=dtype),
             A=_decays(kind, c, s, g), B=g.normal(n, l, groups, s, dtype=dtype), C=g.normal(n, l, groups, s, dtype=dtype),
             dy=g.normal(n, l, c, dtype=dtype), D=g.uniform(0.5, 1.5, c), z=g.normal(n, l, c, dtype=dtype, scale=2.0),
             dt_bias=g.uniform(-6.0, -2.0, c) if softplus else g.uniform(0.0, 0.01, c),
             state=g.normal(n, c, s, dtype=F32), dstate_out=g.normal(n, c, s, dtype=F32))
    t = {k: v.cuda() for k, v in t.items()}
    want = bounds.scan(**t, softplus=softplus, lengths=lens, span=span)
    y, end = torch.empty_like(t["x"]), torch.empty_like(t["state"])
    kept = seq.scan_checkpoints(t["x"], t["B"])
    kept.fill_(float("nan"))
    assert (seq.scan_workspace_bytes(n, l, c, s, groups) > 0) == (span > 0)
    ws = ws_nan(seq.scan_workspace_bytes(n, l, c, s, groups, True))
    pos = [t[k] for k in ("x", "dt", "A", "B", "C")]
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=softplus, lengths=lens, ws=ws)
    seq.scan_fwd(*pos, y, state=t["state"], state_out=end, checkpoints=kept, **kw)
    within(y, want["y"], "y")
    within(end, want["end"], "end")
    o = {k: torch.empty_like(t[v]) for k, v in dict(dx="x", ddt="dt", dA="A", dB="B", dC="C", dD="D", dz="z",
                                                    ddt_bias="dt_bias", dstate="state").items()}
    seq.scan_bwd(*pos, t["dy"], kept, o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], dD=o["dD"], dz=o["dz"],
                 ddt_bias=o["ddt_bias"], dstate_out=t["dstate_out"], dstate=o["dstate"], **kw)
    for k, v in o.items():
        within(v, want[k], k)


CONV = [  # n, l, c, width, dtype, w's type, silu, lengths
    (2, 70, 40, 4, F32, F32, True, [70, 3]), (3, 300, 257, 4, BF16, F32, True, None), (2, 500, 64, 3, F16, F16, True, [499, 0]),
    (1, 1000, 24, 2, F32, F32, False, None), (8, 700, 1024, 4, BF16, BF16, True, "some"), (5, 900, 516, 4, F32, F32, True, None),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_conv(case):
    n, l, c, width, dtype, wt, silu, lengths = case
    g = Gen(l + c)
    if lengths == "some":
        lengths = torch.randint(0, l + 1, (n,), generator=g.g).tolist()
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    x, dy = g.normal(n, l, c, dtype=dtype, scale=2.0).cuda(), g.normal(n, l, c, dtype=dtype).cuda()
    w, b = g.normal(c, width, dtype=wt, scale=0.6).cuda(), g.normal(c, dtype=wt).cuda()
    state, arriving = g.normal(n, width - 1, c, dtype=dtype).cuda(), g.normal(n, width - 1, c, dtype=dtype).cuda()
    want = bounds.conv(x, w, b, silu, dy, state, arriving, lens)
    y, dx, dst = torch.empty_like(x), torch.empty_like(x), torch.empty_like(state)
    dw, db = torch.empty(c, width, device="cuda"), torch.empty(c, device="cuda")
    seq.causal_conv_fwd(x, w, y, b, silu=silu, state=state, lengths=lens)
    within(y, want["y"], "y")
    seq.causal_conv_bwd(x, w, dy, dx, dw, b, db, silu=silu, state=state, dstate_out=arriving, dstate=dst, lengths=lens,
                        ws=ws_nan(seq.causal_conv_workspace_bytes(n, l, c, width)))
    for k, v in dict(dx=dx, dw=dw, db=db, dstate=dst).items():
        within(v, want[k], k)


# Rows enough that a CTA of the backward pass walks over more of them than its ring holds, with a remainder: n, c, dtype, w's type
NORM = [
    (5003, 2048, BF16, BF16), (30011, 256, BF16, F32), (6001, 256, F16, F32), (7301, 512, BF16, BF16), (9001, 1024, BF16, F32),
    (1501, 4096, BF16, BF16), (1501, 8192, F16, F16), (2003, 4096, F32, F32), (5003, 1024, F32, F32), (24321, 128, F32, F32),
    (7301, 1001, BF16, F32), (1201, 5000, F32, F32), (801, 16392, BF16, BF16),
]


@pytest.mark.parametrize("n, c, dtype, wt", NORM)
def test_norm_of_many_rows(n, c, dtype, wt):
    g = torch.Generator(device="cuda").manual_seed(c)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    x, res, dy, dr = ((rand(n, c) * k).to(dtype) for k in (1, 2, 1, 1))
    w = (rand(c) * 0.2 + 1).to(wt)
    y, r, dx, rstd, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(n, device="cuda"), \
        torch.empty(c, device="cuda")
    ws = ws_nan(seq.rms_norm_workspace_bytes(n, c))
    seq.rms_norm_fwd(x, w, y, residual=res, residual_out=r, rstd=rstd, eps=1e-5)
    want, kept, rs = ref.norm_fwd(x, w, res, 1e-5)
    assert torch.equal(r.double(), kept)
    within(rstd, bounds.Bounded(rs, rs, 24 * rs), "rstd")
    within(y, bounds.Bounded(want, want.abs(), 24 * want.abs()), "y")
    hat = kept.abs() * rs[:, None]
    dh = (dy.double() * w.double()).abs()
    mag = rs[:, None] * (dh + hat * (dh * hat).mean(-1, keepdim=True))
    mw = (dy.double().abs() * hat).sum(0)
    for extra in (None, dr):
        wx, ww = ref.norm_bwd(r, w, dy, extra, 1e-5)
        m = mag if extra is None else mag + extra.double().abs()
        seq.rms_norm_bwd(r, w, rstd, dy, dx, dw, dresidual=extra, ws=ws)
        within(dx, bounds.Bounded(wx, m, 24 * m), "dx")
        within(dw, bounds.Bounded(ww, mw, 24 * mw), "dw")
    inplace, dw2 = dr.clone(), torch.empty_like(dw)
    seq.rms_norm_bwd(r, w, rstd, dy, inplace, dw2, dresidual=inplace, ws=ws)
    assert torch.equal(inplace, dx) and torch.equal(dw2, dw)
