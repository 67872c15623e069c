"""A batch without rows in the linear head's losses: no call is refused for the
pointers of tensors that hold nothing (CPU; on a GPU through the binding too)."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from test_loss_abi import E, OK, ce_grad, di_grad


@pytest.mark.parametrize("call,kw", [(ce_grad, dict(labels=None, loss=None)),
                                     (di_grad, dict(index=None, teacher=None, logp=None))])
def test_a_frozen_head_without_rows(call, kw):
    # dX [0, D] of a caching allocator is a null pointer, dW is not asked for
    empty = dict(T=0, X=None, lse=None, dloss=None, dX=None, dW=None, ws=None, nbytes=0, **kw)
    assert call(**empty) == OK
    assert call(**{**empty, "W": None}) == E
    # with rows, a call that asks for nothing stays an error
    assert call(dX=None, dW=None) == E


@pytest.mark.gpu
def test_a_frozen_head_without_rows_through_the_binding():
    X = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((50, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(0, device="cuda")
    lab = torch.zeros(0, dtype=torch.int64, device="cuda")
    dX, dW = dg.linear_cross_entropy_grad(X, W, lab, v, v, v, need_dW=False)
    assert dX.shape == (0, 64) and dW is None
    idx, te = torch.zeros((0, 3), dtype=torch.int64, device="cuda"), torch.zeros((0, 3), device="cuda")
    dX, dW = dg.linear_distillation_grad(X, W, idx, te, v, te, v, need_dW=False)
    assert dX.shape == (0, 64) and dW is None
    _, dW = dg.linear_distillation_grad(X, W, idx, te, v, te, v)
    assert float(dW.abs().sum()) == 0.0
