"""Few rows of the linear head's losses over vocabularies of one and several
pieces (the gradient's two halves fill 256 MiB, or a piece 2^21 columns)."""
import math

import pytest
import torch

import dense_gemm_linear_amd as dg
from loss_reference import check, problem, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,D,k", [(1, 600001, 8, 0), (3, 600001, 16, 0), (3, 600001, 8, 3),
                                     (128, 530003, 8, 0), (128, 530003, 8, 2), (40, (1 << 21) + 3001, 8, 0),
                                     (2, (1 << 21) + 3001, 8, 0), (2, (1 << 21) + 3001, 8, 5)])
@pytest.mark.parametrize("keep", [0.6, 1.0])
def test_few_rows_of_wide_vocabularies(T, V, D, k, keep):
    print(f"[wide {T} {V} {D} {k} {keep}]", flush=True)
    X, W, lab = problem(T, V, D, T + k)
    g = torch.Generator().manual_seed(T)
    lab[0], lab[T // 2] = V - 1, 530000 % V              # the last column, and one past most pieces
    if keep < 1.0 and T > 2:
        gone = (torch.rand(T, generator=g) >= keep).cuda()
        gone[0] = gone[T // 2] = False
        lab[gone] = -100
    dl = ((torch.rand(T, generator=g) + 0.5) / T).cuda()
    nbytes = dg.linear_loss_workspace_bytes(T, V, D, k, backward=True)
    # the workspace and what lies behind it
    buf = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = buf[:nbytes]
    if k:
        idx = torch.randint(0, V, (T, k), generator=g).cuda()
        idx[:, 0] = lab.clamp(min=-1)
        te = torch.randn(T, k, generator=g).cuda()
        loss, lse, logp = dg.linear_distillation(X, W, idx, te, workspace=ws)
        ws.fill_(0xFF)
        dX, dW = dg.linear_distillation_grad(X, W, idx, te, lse, logp, dl, workspace=ws)
        got = dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW)
        ref = reference(X, W, index=idx, teacher=te, dloss=dl)
    else:
        loss, lse = dg.linear_cross_entropy(X, W, lab, workspace=ws)
        ws.fill_(0xFF)
        dX, dW = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, workspace=ws)
        got = dict(loss=loss, lse=lse, dX=dX, dW=dW)
        ref = reference(X, W, labels=lab, dloss=dl)
    torch.cuda.synchronize()
    check(got, ref, f"{T}x{V}x{D} k={k}")
    assert bool((buf[nbytes:] == 0xFF).all()), "wrote past the workspace"
    assert math.isfinite(float(got["loss"].sum()))
