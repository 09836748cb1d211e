"""The float64 reference of the gated linear recurrence, pinned: a closed form for a
constant decay, an explicit sum, and the gradients against central differences."""
import pytest
import torch

import linrecref as R


def test_constant_decay_is_a_geometric_sum():
    T, D = 12, 3
    g = torch.full((1, T, D), -0.25, dtype=torch.float64)
    x = torch.ones(1, T, D, dtype=torch.float64)
    h, _ = R.states_and_bounds(x, g, None, None)
    a = torch.tensor(-0.25, dtype=torch.float64).exp()
    want = (1 - a ** torch.arange(1, T + 1, dtype=torch.float64)) / (1 - a)
    assert torch.allclose(h[0, 1:, 0], want, rtol=1e-14, atol=0)


def test_states_are_the_decayed_sum_of_writes():
    x, g, b, h0, _, _ = R.inputs(2, 9, 4, torch.float64, seed=1, device="cpu")
    h0 = h0.double()
    h, _ = R.states_and_bounds(x, g, b, h0)
    for t in range(9):
        want = g[:, :t + 1].sum(1).exp() * h0
        for j in range(t + 1):
            want = want + g[:, j + 1:t + 1].sum(1).exp() * b[:, j] * x[:, j]
        assert torch.allclose(h[:, t + 1], want, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("with_beta", [True, False])
def test_gradients_match_central_differences(with_beta):
    x, g, b, h0, dO, dhT = R.inputs(2, 7, 3, torch.float64, beta=with_beta, seed=2, device="cpu")
    h0, dhT = h0.double(), dhT.double()

    def loss(x, g, b, h0):
        h, _ = R.states_and_bounds(x, g, b, h0)
        return float((h[:, 1:] * dO).sum() + (h[:, -1] * dhT).sum())

    gr = R.grads_and_bounds(x, g, b, h0, dO, dhT)
    args = dict(x=x, g=g, b=b, h0=h0)
    eps = 1e-6
    for name, grad in (("x", "dx"), ("g", "dg"), ("b", "dbeta"), ("h0", "dh0")):
        if args[name] is None:
            assert grad not in gr
            continue
        flat = args[name].reshape(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + eps
            up = loss(**args)
            flat[i] = keep - eps
            down = loss(**args)
            flat[i] = keep
            # the loss is of order 100: differences of it carry 1e-14 * 100 / eps
            assert abs((up - down) / (2 * eps) - float(gr[grad][0].reshape(-1)[i])) < 1e-5, (name, i)
