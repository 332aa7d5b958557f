"""The references with error bounds against the token-by-token ones."""
import pytest
import torch

import seq_bounds as bounds
import seq_reference as ref


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("softplus, lengths", [(True, None), (False, [5, 3]), (True, [0, 9])])
def test_scan(softplus, lengths):
    g = torch.Generator().manual_seed(1)
    n, l, c, s, gr = 2, 6, 4, 3, 2
    x, dt, z, dy = (_rand(g, n, l, c) for _ in range(4))
    B, C = _rand(g, n, l, gr, s), _rand(g, n, l, gr, s)
    A, D, bias = -_rand(g, c, s).abs(), _rand(g, c), _rand(g, c)
    state, arriving = _rand(g, n, c, s), _rand(g, n, c, s)
    lens = None if lengths is None else torch.tensor(lengths)
    got = bounds.scan(x, dt, A, B, C, dy, D, z, bias, softplus, state, arriving, lens)
    y, end, *_ = ref.scan_fwd(x, dt, A, B, C, D, z, bias, softplus, state, lengths)
    want = ref.scan_bwd(x, dt, A, B, C, dy, D, z, bias, softplus, state, arriving, lengths)
    want.update(y=y, end=end)
    assert want.keys() == got.keys()
    for k, v in want.items():
        assert torch.allclose(got[k].v, v, rtol=1e-10, atol=1e-12), k
        assert bool((got[k].mag >= got[k].v.abs() - 1e-12).all()) and bool((got[k].err >= 0).all()), k


@pytest.mark.parametrize("silu, lengths", [(True, None), (False, [5, 3]), (True, [0, 1])])
@pytest.mark.parametrize("width", [1, 4])
def test_conv(silu, lengths, width):
    g = torch.Generator().manual_seed(2)
    n, l, c = 2, 6, 3
    x, dy, w, b = _rand(g, n, l, c), _rand(g, n, l, c), _rand(g, c, width), _rand(g, c)
    state, arriving = _rand(g, n, width - 1, c), _rand(g, n, width - 1, c)
    got = bounds.conv(x, w, b, silu, dy, state, arriving, None if lengths is None else torch.tensor(lengths))
    want = dict(zip(("dx", "dw", "db", "dstate"), ref.conv_bwd(x, w, dy, b, silu, state, arriving, lengths)))
    want["y"] = ref.conv_fwd(x, w, b, silu, state, lengths)[0]
    assert want.keys() == got.keys()
    for k, v in want.items():
        assert torch.allclose(got[k].v, v, rtol=1e-10, atol=1e-12), k
        assert bool((got[k].mag >= got[k].v.abs() - 1e-12).all()) and bool((got[k].err >= 0).all()), k
