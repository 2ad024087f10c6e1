"""The 64-bit definitions of tests/training_ref.py against the formulas of include/moe.h and
against finite differences, on the CPU."""
import pytest
import torch

from tests import training_ref as R


def case(router, seed=0, T=13, E=10, K=3):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, dtype=torch.float64, generator=g)
    s = R.affinity(logits, router)
    idx = torch.topk(s, K, dim=1).indices.int()
    dw = torch.randn(T, K, dtype=torch.float64, generator=g)
    return logits, s, idx, dw


OFFSETS = [0, 5, 5, 11]


@pytest.mark.parametrize("router", [0, 1])
def test_formula_is_the_gradient(router):
    logits, s, idx, dw = case(router)
    T, E, K, alpha = *s.shape, idx.shape[1], 0.3
    n = R.counts(idx, OFFSETS, E)
    dl = torch.tensor([2.0, 3.0, 5.0], dtype=torch.float64)
    x = logits.clone().requires_grad_()
    got = torch.autograd.grad(R.router_goal(R.affinity(x, router), idx, dw, OFFSETS, n, dl, alpha),
                              x)[0]
    ds = torch.zeros_like(s)
    for q, (lo, hi) in enumerate(R.spans(OFFSETS, T)):
        N = hi - lo
        for t in range(lo, hi):
            S = s[t].sum()
            p = s[t] / S
            ds[t] += dl[q] * alpha * E / (K * N * N) * (n[q] - (n[q] * p).sum()) / S
    for t in range(T):
        Z = s[t, idx[t].long()].sum()
        w = s[t, idx[t].long()] / Z
        ds[t, idx[t].long()] += (dw[t] - (dw[t] * w).sum()) / Z
    slope = (1 - torch.exp(-s * s)) / (2 * s) if router else s * (1 - s)
    assert torch.allclose(got, ds * slope, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("router", [0, 1])
def test_gradient_is_the_difference_quotient(router):
    logits, s, idx, dw = case(router, seed=1, T=6, E=5, K=2)
    offs, alpha = [0, 4, 6], 0.7
    n = R.counts(idx, offs, 5)
    dl = torch.tensor([1.5, -2.0], dtype=torch.float64)

    def goal(v):
        return R.router_goal(R.affinity(v, router), idx, dw, offs, n, dl, alpha)

    x = logits.clone().requires_grad_()
    grad = torch.autograd.grad(goal(x), x)[0]
    h = 1e-5  # truncation h^2 f'''/6 ~ 1e-10, cancellation 1e-16 / h ~ 1e-11
    for t in range(6):
        for i in range(5):
            e = torch.zeros_like(logits)
            e[t, i] = h
            assert abs((goal(logits + e) - goal(logits - e)) / (2 * h) - grad[t, i]) < 1e-8


def test_logits_of_inverts_the_affinity():
    x = torch.linspace(-6, 6, 41, dtype=torch.float64)
    for router in (0, 1):
        assert torch.allclose(R.logits_of(R.affinity(x, router), router), x, atol=1e-10)
