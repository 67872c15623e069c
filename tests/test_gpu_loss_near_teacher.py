"""Distillation of a student that is near its teacher: every p - q is small,
and one or two columns still make up a whole row of dX."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from loss_reference import check, reference
from test_gpu_loss_rounding import _dloss, _held_once, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,D,k", [(1, 3000, 512, 2), (40, 4000, 512, 2), (128, 3000, 264, 3), (129, 3000, 264, 3),
                                     (600, 4000, 512, 4), (300, 2000, 1032, 64)])
def test_small_differences_are_rounded_once(T, V, D, k):
    g = torch.Generator().manual_seed(T + k)
    W = (torch.randn(V, D, generator=g) * (2.0 / D ** 0.5)).bfloat16()
    idx = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(T)])
    # two columns of probability near 1/2 each, the others' together below 1 %
    X = (4.0 * (W[idx[:, 0]].float() + W[idx[:, 1]].float()) + 0.5 * torch.randn(T, D, generator=g)).bfloat16()
    z = X.double() @ W.double().t()
    te = z.gather(1, idx)
    te[:, :2] += 0.03 * torch.randn(T, 2, generator=g, dtype=torch.float64)
    X, W, idx, te = X.cuda(), W.cuda(), idx.cuda(), te.float().cuda()
    dl = _dloss(T, 3)
    p = torch.softmax(z.cuda(), 1).gather(1, idx)
    q = torch.softmax(te.double(), 1)
    assert float((p - q).abs().max()) < 0.0625         # the inputs are what they are meant to be
    got = _run(X, W, None, idx, te, dl)
    ref = reference(X, W, index=idx, teacher=te, dloss=dl)
    check(got, ref, f"near the teacher {T}x{V}x{D} k={k}")
    _held_once(f"near the teacher {T}x{V}x{D} k={k}", got, ref, X, W, None, idx, te, dl)
