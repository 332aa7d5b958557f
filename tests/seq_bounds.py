"""The sequence operators in 64 bits with a bound on fp32's error for each element (test infrastructure). Sequences are
computed side by side, on whatever device the inputs are on.

Each value comes with `mag`, the sum of its terms' absolute values, and `err`, a bound on the error of a computation in 32
bits, in units of U = 2^-21. What an operation may add, in U:

  sum, product                  1/8 of its result (2^-24)
  exp2 of the special unit      1/2, and the argument's own error: for exp(delta A) that is |delta A| times the relative error
                                of delta and of A log2 e (1/8), and half a unit to round it
  reciprocal                    1/4
  sigmoid(v)                    1.5 + |v| / 4: exp2 and reciprocal, v log2 e rounded twice
  softplus(v)                   2 + |v| / 8: its own 1, and the rounding of v = dt + bias, which it magnifies by up to |v|
  softplus'(v)                  2 + |v| / 2
  silu(v), silu'(v)             1.75 + |v| / 4, 3 + |v| / 2 of the terms' absolute values; an error of v itself counts 1.1
                                and 0.6 times (the largest slopes)
  sums over many terms          1/8 for each addition that lies one after another

`span` is the tokens whose deltas are added up in 32 bits for the decay over a part of the time axis (0: the axis is not cut);
the sum's error is up to span / 8 of it."""
import torch

U = 2.0 ** -21


def _sig(v):
    return torch.sigmoid(v)


def _silu_grad(v):
    s = _sig(v)
    return s * (1 + v * (1 - s))


def _silu_grad_mag(v):
    s = _sig(v)
    return s * (1 + v.abs() * (1 - s))


class Bounded:
    """A value, its terms' absolute sum and its error bound."""

    def __init__(self, v, mag, err):
        self.v, self.mag, self.err = v, mag, err


def _live(lengths, n, l, device):
    lens = torch.full((n,), l, device=device) if lengths is None else lengths.to(device).long().clamp(0, l)
    return torch.arange(l, device=device)[None, :, None] < lens[:, None, None]


def scan(x, dt, A, B, C, dy=None, D=None, z=None, dt_bias=None, softplus=False, state=None, dstate_out=None, lengths=None,
         span=0):
    """A dict of Bounded: y, end and, with dy, dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate."""
    n, l, c = x.shape
    g, s = B.shape[2:]
    dev = x.device
    live = _live(lengths, n, l, dev)
    f = lambda t: torch.where(live, t.double(), 0)  # noqa: E731
    x, raw = f(x), f(dt.double() + (0 if dt_bias is None else dt_bias.double()))
    B, C = (torch.where(live[..., None], t.double(), 0) for t in (B, C))
    A = A.double()
    D = torch.zeros(c, dtype=torch.float64, device=dev) if D is None else D.double()
    delta = torch.where(live, torch.nn.functional.softplus(raw, threshold=200) if softplus else raw, 0)
    e_d = 2 + raw.abs() / 8
    e_u = e_d + 0.25
    u = delta * x
    if z is not None:
        z = f(z)
    gate = 1 if z is None else z * _sig(z)
    e_gate = 0.0 if z is None else 1.75 + z.abs() / 4
    rows = lambda t, i: t[:, i].repeat_interleave(c // g, 1)  # [n, c, s]  # noqa: E731

    def decay(i):
        dA = delta[:, i, :, None] * A
        return torch.exp(dA), dA.abs() * (e_d[:, i, :, None] + 0.75 + span / 8) + 1

    h = torch.zeros(n, c, s, dtype=torch.float64, device=dev) if state is None else state.double()
    mag, err = h.abs(), torch.zeros_like(h)
    hs = [(h, mag, err)]
    y = Bounded(torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x))
    for i in range(l):
        a, e_a = decay(i)
        b, cc, on = rows(B, i), rows(C, i), live[:, i, :, None]
        new = a * h + u[:, i, :, None] * b
        new_mag = a * mag + (u[:, i, :, None] * b).abs()
        new_err = a * err + a * mag * (e_a + 0.25) + (u[:, i, :, None] * b).abs() * (e_u[:, i, :, None] + 0.5) + new_mag / 8
        h, mag, err = (torch.where(on, p, q) for p, q in ((new, h), (new_mag, mag), (new_err, err)))
        hs.append((h, mag, err))
        dx_ = D * x[:, i]
        y.v[:, i] = (cc * h).sum(-1) + dx_
        y.mag[:, i] = (cc.abs() * mag).sum(-1) + dx_.abs()
        y.err[:, i] = (cc.abs() * (err + 3 * mag)).sum(-1) + dx_.abs()
    gm = 1 if z is None else gate.abs()
    r = dict(y=Bounded(y.v * gate * live, y.mag * gm, gm * (y.err + y.mag * (e_gate + 0.25))), end=Bounded(h, mag, err))
    if dy is None:
        return r
    dyo = f(dy)
    d = dyo * gate
    e_dy = e_gate + 0.25 if z is not None else torch.zeros_like(d)
    zero = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=dev)  # noqa: E731
    for k, shape in dict(dx=x.shape, ddt=x.shape, dA=A.shape, dB=B.shape, dC=C.shape).items():
        r[k] = Bounded(zero(*shape), zero(*shape), zero(*shape))
    if z is not None:
        sm = dyo.abs() * _silu_grad_mag(z)
        r["dz"] = Bounded(dyo * y.v * _silu_grad(z), sm * y.mag, sm * (y.err + y.mag * (3 + z.abs() / 2)))
    aG = zero(n, c, s) if dstate_out is None else dstate_out.double()
    amag, aerr = aG.abs(), torch.zeros_like(aG)
    by_group = lambda t: t.reshape(n, g, c // g, s).sum(2)  # noqa: E731
    for i in reversed(range(l)):
        on = live[:, i, :, None]
        b, cc, di, ui, xi = rows(B, i), rows(C, i), d[:, i, :, None], u[:, i, :, None], x[:, i]
        h, mag, err = hs[i + 1]
        G = cc * di + aG
        Gmag = (cc * di).abs() + amag
        Gerr = aerr + (cc * di).abs() * (e_dy[:, i, :, None] + 0.25) + Gmag / 8
        r["dC"].v[:, i], r["dC"].mag[:, i] = by_group(di * h), by_group(di.abs() * mag)
        r["dC"].err[:, i] = by_group(di.abs() * (err + mag * (e_dy[:, i, :, None] + 6)))
        r["dB"].v[:, i], r["dB"].mag[:, i] = by_group(G * ui), by_group(Gmag * ui.abs())
        r["dB"].err[:, i] = by_group(ui.abs() * (Gerr + Gmag * (e_u[:, i, :, None] + 6)))
        gb, gb_mag, gb_err = (G * b).sum(-1), (Gmag * b.abs()).sum(-1), ((Gerr + Gmag) * b.abs()).sum(-1)
        dl = delta[:, i].abs()
        r["dx"].v[:, i] = delta[:, i] * gb + D * d[:, i]
        r["dx"].mag[:, i] = dl * gb_mag + (D * d[:, i]).abs()
        r["dx"].err[:, i] = dl * (gb_err + gb_mag * (e_d[:, i] + 0.5)) + (D * d[:, i]).abs() * (e_dy[:, i] + 0.5)
        a, e_a = decay(i)
        new, nmag = a * G, a * Gmag
        nerr = a * Gerr + a * Gmag * (e_a + 0.25)
        p, pmag, perr = hs[i]
        Gp, Gpm = new * p, nmag * pmag
        Gpe = nerr * pmag + nmag * perr + Gpm / 8
        out = (Gp * A).sum(-1) + gb * xi
        omag = (Gpm * A.abs()).sum(-1) + gb_mag * xi.abs()
        oerr = ((Gpe + 1.5 * Gpm) * A.abs()).sum(-1) + (gb_err + gb_mag) * xi.abs()
        sg = _sig(raw[:, i]) if softplus else torch.ones_like(out)
        e_sg = 2 + raw[:, i].abs() / 2 if softplus else 0.25
        on2 = live[:, i]
        r["ddt"].v[:, i], r["ddt"].mag[:, i] = out * sg * on2, omag * sg * on2
        r["ddt"].err[:, i] = (oerr + omag * e_sg) * sg * on2
        dl3 = delta[:, i, :, None]
        r["dA"].v += torch.where(on, Gp * dl3, 0).sum(0)
        r["dA"].mag += torch.where(on, Gpm * dl3.abs(), 0).sum(0)
        r["dA"].err += torch.where(on, dl3.abs() * (Gpe + Gpm * (e_d[:, i, :, None] + 0.25)), 0).sum(0)
        aG, amag, aerr = (torch.where(on, q, o) for q, o in ((new, aG), (nmag, amag), (nerr, aerr)))
    many = 4 + l / 32 + n / 8
    r["dA"].err += many * r["dA"].mag
    t = d * x
    r["dD"] = Bounded(t.sum((0, 1)), t.abs().sum((0, 1)), (t.abs() * (e_dy + 0.25 + many)).sum((0, 1)))
    q = r["ddt"]
    r["ddt_bias"] = Bounded(q.v.sum((0, 1)), q.mag.sum((0, 1)), (q.err + many * q.mag).sum((0, 1)))
    r["dstate"] = Bounded(aG, amag, aerr)
    for k in ("dx", "dB", "dC"):
        m = live if r[k].v.dim() == 3 else live[..., None]
        r[k].v = r[k].v * m
    return r


def conv(x, w, bias=None, silu=False, dy=None, state=None, dstate_out=None, lengths=None):
    """A dict of Bounded: y and, with dy, dx, dw, db, dstate."""
    n, l, c = x.shape
    width = w.shape[1]
    dev = x.device
    live = _live(lengths, n, l, dev)
    past = torch.zeros(n, width - 1, c, dtype=torch.float64, device=dev) if state is None else state.double()
    line = torch.cat([past, torch.where(live, x.double(), 0)], 1)
    w = w.double()
    b = torch.zeros(c, dtype=torch.float64, device=dev) if bias is None else bias.double()
    win = line.unfold(1, width, 1)  # [n, l, c, width]
    v, vm = (win * w).sum(-1) + b, (win.abs() * w.abs()).sum(-1) + b.abs()
    ve = vm * (width + 1) / 8
    s = v * _sig(v) if silu else v
    r = dict(y=Bounded(s * live, vm, 1.1 * ve + s.abs() * (1.75 + v.abs() / 4) if silu else ve))
    if dy is None:
        return r
    dy = torch.where(live, dy.double(), 0)
    slope, smag = (_silu_grad(v), _silu_grad_mag(v)) if silu else (torch.ones_like(v), torch.ones_like(v))
    dv, dvm = dy * slope, dy.abs() * smag
    dve = dy.abs() * (0.6 * ve + smag * (3 + v.abs() / 2)) if silu else torch.zeros_like(dv)
    dl, dlm, dle = (torch.zeros_like(line) for _ in range(3))
    for j in range(width):
        dl[:, j:j + l] += w[:, j] * dv
        dlm[:, j:j + l] += w[:, j].abs() * dvm
        dle[:, j:j + l] += w[:, j].abs() * dve
    if dstate_out is not None:
        lens = live.sum(1)[:, 0]
        at = (lens[:, None] + torch.arange(width - 1, device=dev))[..., None].expand(-1, -1, c)
        dl.scatter_add_(1, at, dstate_out.double())
        dlm.scatter_add_(1, at, dstate_out.double().abs())
    dle += dlm * (width + 1) / 8
    k = width - 1
    r["dstate"], r["dx"] = (Bounded(*(t[:, a:e] for t in (dl, dlm, dle))) for a, e in ((0, k), (k, k + l)))
    r["dx"].v = r["dx"].v * live
    many = 24 + n / 8  # 128 tokens of a strip, 8 strips of a CTA, the slabs by 8 chains
    r["dw"] = Bounded((win * dv[..., None]).sum((0, 1)), (win.abs() * dvm[..., None]).sum((0, 1)),
                      (win.abs() * (dve + many * dvm)[..., None]).sum((0, 1)))
    r["db"] = Bounded(dv.sum((0, 1)), dvm.sum((0, 1)), (dve + many * dvm).sum((0, 1)))
    return r
