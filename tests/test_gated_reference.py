"""The 64-bit reference of the gated scan against differences, and of the selection against cases by hand."""
import pytest
import torch

import gated_ref as G

F64 = torch.float64


@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("gates", [(False, False), (True, True)])
def test_gradients_agree_with_differences(rate, gates):
    g = torch.Generator().manual_seed(3)
    b, t, d = 3, 6, 4
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    lens = torch.tensor([6, 0, 4])
    p = dict(x=r(b, t, d), r=r(b, t, d), h0=r(b, d))
    if gates[0]:
        p["i"] = r(b, t, d)
    if gates[1]:
        p["z"] = r(b, t, d)
    if rate:
        p["rate"] = torch.rand(d, generator=g, dtype=F64) + 0.05
    dout, dfinal = r(b, t, d), r(b, d)
    got = G.GatedCase(**p, lens=lens).gradient(dout, dfinal)

    def value():
        out, final = G.GatedCase(**p, lens=lens).forward()
        return float((out.v * dout).sum() + (final.v * dfinal).sum())

    for name, key in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("rate", "drate"), ("h0", "dinit")):
        if name not in p:
            continue
        flat, want = p[name].view(-1), got[key].v.reshape(-1)
        for n in range(0, flat.numel(), 5):
            keep, eps = float(flat[n]), 1e-6
            flat[n] = keep + eps
            up = value()
            flat[n] = keep - eps
            down = value()
            flat[n] = keep
            assert abs((up - down) / (2 * eps) - float(want[n])) < 1e-6 * (1 + abs(float(want[n]))), (key, n)


def test_states_pass_what_is_behind_a_sequence():
    x = torch.ones(1, 5, 2)
    x[:, 3:] = float("nan")
    out, final = G.GatedCase(x, x, lens=torch.tensor([3])).forward()
    assert torch.isfinite(out.v).all() and (out.v[:, 3:] == 0).all() and torch.equal(final.v, out.v[:, 2])


def test_selection_by_hand():
    ninf = float("-inf")
    x = torch.tensor([[[0.0, 1.0, 1.0], [2.0, ninf, ninf]]])
    r = G.beam_select(x, 3)
    # beam 1's only token has probability 1; beam 0's tokens 1 and 2 are equal, the lower comes first
    assert r["parents"].tolist() == [[1, 0, 0]] and r["tokens"].tolist() == [[0, 1, 2]]
    r = G.beam_select(x, 3, prior=torch.tensor([[ninf, 0.0]]))
    assert r["parents"].tolist() == [[1, 0, 0]] and r["tokens"].tolist() == [[0, 0, 1]]
    r = G.beam_select(x, 3, finished=torch.tensor([[1, 0]]), eos=2, prior=torch.tensor([[-0.5, -1.0]]),
                      slots=torch.tensor([[7, 4, 9]]))
    assert r["parents"].tolist() == [[0, 1, 0]] and r["tokens"].tolist() == [[2, 0, 0]] and r["finished"].tolist() == [[1, 0, 1]]
    assert r["slots"].tolist() == [[7, 4, 9]] and r["src"].tolist() == [[-1, -1, 7]] and r["dst"].tolist() == [[-1, -1, 9]]
