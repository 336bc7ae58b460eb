"""The 64-bit references of the sequence-model operators (seq_ref.py) against
differences: each gradient formula is compared with (f(x + e) - f(x - e)) / 2e along
random directions. Runs on the CPU; the kernels' gradients are then tested
against these formulas."""
import pytest
import torch

import seq_ref as R

F64 = torch.float64
E = 1e-6  # central differences: error O(E^2) of third derivatives, and 1e-16 / E of rounding


def rand(g, *shape):
    return torch.randn(shape, generator=g, dtype=F64)


def check(f, at, grads, g):
    """The derivative of f along a random direction of each input against its gradient."""
    for name, x in at.items():
        v = rand(g, *x.shape)
        up, down = f(**{**at, name: x + E * v}), f(**{**at, name: x - E * v})
        diff = (up - down) / (2 * E)
        want = (grads[name] * v).sum()
        assert abs(diff - want) <= 1e-7 * (1 + abs(want)) + 1e-7 * (grads[name] * v).abs().sum(), (name, diff, want)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("width", [1, 2, 4])
def test_conv_gradient_against_differences(width, silu):
    g = torch.Generator().manual_seed(width)
    x, w, bias, before = rand(g, 2, 6, 3), rand(g, 3, width), rand(g, 3), rand(g, 2, width - 1, 3)
    dout = rand(g, 2, 6, 3)
    mask = R.live_mask(torch.tensor([6, 4]), 2, 6)
    x = R.zeroed(x, mask)

    def f(x, w, bias, before):
        x = torch.where(mask[..., None], x, 0.0)
        return (R.conv(x, w, bias, silu, before, mask)[0] * dout).sum()

    dx, dw, db, ds = R.conv_grad(x, w, bias, silu, before, mask, dout)
    check(f, dict(x=x, w=w, bias=bias, before=before), dict(x=dx, w=dw, bias=db, before=ds), g)


@pytest.mark.parametrize("use_softplus", [True, False])
@pytest.mark.parametrize("groups", [1, 2])
def test_scan_gradient_against_differences(groups, use_softplus):
    g = torch.Generator().manual_seed(5 + groups)
    b, length, d, n = 2, 5, 4, 3
    lens = torch.tensor([5, 3], dtype=torch.int32)
    at = dict(u=rand(g, b, length, d), delta=rand(g, b, length, d) if use_softplus else rand(g, b, length, d).abs() * 0.3,
              A=-rand(g, d, n).abs(), B=rand(g, b, length, groups, n), C=rand(g, b, length, groups, n), D=rand(g, d),
              z=rand(g, b, length, d), delta_bias=rand(g, d) * 0.1, h0=rand(g, b, d, n))
    dout, dfinal = rand(g, b, length, d), rand(g, b, d, n)

    def f(**x):
        out, last = R.ScanCase(use_softplus=use_softplus, lens=lens, **x).forward()
        return (out * dout).sum() + (last * dfinal).sum()

    got = R.ScanCase(use_softplus=use_softplus, lens=lens, **at).grad(dout, dfinal)
    grads = {k: got["dinit" if k == "h0" else "d" + k] for k in at}
    check(f, at, grads, g)


def test_step_by_step_is_the_prompt():
    """The state after a prompt and the next token's result are those of the longer prompt."""
    g = torch.Generator().manual_seed(9)
    b, length, d, n = 1, 7, 3, 2
    x = dict(u=rand(g, b, length, d), delta=rand(g, b, length, d), B=rand(g, b, length, 1, n), C=rand(g, b, length, 1, n),
             z=rand(g, b, length, d))
    A = -rand(g, d, n).abs()
    whole, last = R.ScanCase(A=A, **x).forward()
    h = None
    for t in range(length):
        out, h = R.ScanCase(A=A, h0=h, **{k: v[:, t:t + 1] for k, v in x.items()}).forward()
        assert torch.allclose(out[:, 0], whole[:, t], rtol=1e-13, atol=1e-14)
    assert torch.allclose(h, last, rtol=1e-13, atol=1e-14)
