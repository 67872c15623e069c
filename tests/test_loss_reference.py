"""The 64-bit reference of the linear head's losses itself: hand-worked values
and its gradients against differences (CPU only)."""
import math

import pytest
import torch

from loss_reference import problem, reference


def test_hand_worked_cross_entropy():
    # logits (0, log 3): p = (1/4, 3/4)
    X = torch.tensor([[1.0] + [0.0] * 7]).bfloat16()
    W = torch.zeros(4, 8, dtype=torch.bfloat16)
    W[2, 0] = 1.0
    lab = torch.tensor([2])
    r = reference(X, W, labels=lab, dloss=torch.ones(1), scale=math.log(3.0))
    assert abs(float(r["lse"][0]) - math.log(6.0)) < 1e-12
    assert abs(float(r["loss"][0]) - math.log(2.0)) < 1e-12
    # dz = (1/6, 1/6, -1/2, 1/6)
    assert abs(float(r["dX"][0, 0]) - math.log(3.0) * -0.5) < 1e-12
    assert abs(float(r["dW"][0, 0]) - math.log(3.0) / 6.0) < 1e-12


def test_hand_worked_distillation():
    X = torch.zeros(2, 8, dtype=torch.bfloat16)
    W = torch.ones(4, 8, dtype=torch.bfloat16)
    idx = torch.tensor([[1, 3, -1], [-1, -1, -1]])
    te = torch.tensor([[math.log(3.0), 0.0, 5.0], [1.0, 2.0, 3.0]])
    r = reference(X, W, index=idx, teacher=te, dloss=torch.ones(2))
    # q = (3/4, 1/4), p = 1/4 everywhere
    want = 0.75 * math.log(3.0) + 0.25 * math.log(1.0)
    assert abs(float(r["loss"][0]) - want) < 1e-7 and float(r["loss"][1]) == 0.0
    assert float(r["lse"][1]) == 0.0 and float(r["logp"][1].abs().sum()) == 0.0


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_gradients_against_differences(kind):
    T, V, D = 5, 11, 8
    X, W, lead = problem(T, V, D, 3, device="cpu")
    g = torch.Generator().manual_seed(9)
    dl = torch.rand(T, generator=g) + 0.5
    if kind == "ce":
        lab = lead.clone()
        lab[1] = -100
        kw = dict(labels=lab, z_loss=1e-2, scale=0.7)
    else:
        idx = torch.randint(-1, V, (T, 4), generator=g)
        idx[:, 0] = lead
        idx[2, 1] = idx[2, 0]                 # one column twice
        idx[3] = -1
        kw = dict(index=idx, teacher=torch.randn(T, 4, generator=g), scale=0.7)
    r = reference(X, W, dloss=dl, **kw)

    def total(x, w):
        return float((reference(x, w, **kw)["loss"] * dl.double()).sum())

    h = 1e-6
    Xd, Wd = X.double(), W.double()
    for M, grad, f in ((Xd, r["dX"], lambda m: total(m, Wd)), (Wd, r["dW"], lambda m: total(Xd, m))):
        for _ in range(6):
            u = torch.randn(M.shape, generator=g, dtype=torch.float64)
            num = (f(M + h * u) - f(M - h * u)) / (2 * h)
            ana = float((grad * u).sum())
            # central differences: h^2 third derivatives and 2^-53 |loss| / h
            assert abs(num - ana) < 1e-7 * (1 + abs(ana)) + 1e-8 * (1 + abs(total(Xd, Wd)))
