"""Roundings of the logits' gradient to bf16 in the linear head's losses: what
they may leave in dX and dW beside the one rounding of the result.

A rounding to nearest bf16 of x is off by at most h(x) = 2^(e - 8), e the
exponent of x (2^e <= |x| < 2^(e + 1)), evenly: h(x) / sqrt(3) root mean
square.  At some columns the logits' gradient is carried to more bits than bf16
holds (see _held_once), so a result's error has two parts: the rounding of the
result, and those of the other columns, which are independent.  The square of
its norm is the sum of their squares.  5 % on top: fp32 sums, and the targets that may be
left out, which together hold at most 1/16 of the square of their row's largest
(sqrt(1 + 1/16) = 1.031)."""
import math

import pytest
import torch

import dense_gemm_linear_amd as dg
from loss_reference import check, problem, reference

pytestmark = pytest.mark.gpu


def _half_step(x):
    """h(x) of the module's comment."""
    return torch.where(x == 0, 0.0, torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-300))) - 8))


def _dloss(T, seed):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(T, generator=g) + 0.5) / T).cuda()


def _run(X, W, lab, idx, te, dl, **kw):
    if idx is None:
        loss, lse = dg.linear_cross_entropy(X, W, lab)
        dX, dW = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, **kw)
        out = dict(loss=loss, lse=lse, dX=dX, dW=dW)
    else:
        loss, lse, logp = dg.linear_distillation(X, W, idx, te)
        dX, dW = dg.linear_distillation_grad(X, W, idx, te, lse, logp, dl, **kw)
        out = dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW)
    torch.cuda.synchronize()
    return out


def _held_once(what, got, ref, X, W, lab, idx, te, dl):
    """Error norms of dX and dW against one rounding of the result and those of
    the columns whose rounding is not made good: for dX all but the targets, for
    dW of up to 128 rows none, of more all but the row's label or, of a teacher's
    columns, those in the 256 columns of the one of the largest |p - q|."""
    z = X.double() @ W.double().t()
    dz = torch.softmax(z, 1)
    at = lab[:, None] if idx is None else idx
    keep = (at >= 0).any(1)
    cols = at.clamp(min=0)
    if idx is not None:
        q = torch.softmax(torch.where(idx >= 0, te.double(), -math.inf), 1).nan_to_num(0.0)
        dz = dz.scatter_add(1, cols, -q)
    dz = torch.where(keep[:, None], dz * dl.double()[:, None], 0.0)
    lead = cols.gather(1, dz.gather(1, cols).abs().argmax(1, keepdim=True))
    near = torch.where(cols // 256 == lead // 256, cols, lead)
    for name, made_good in (("dX", cols), ("dW", near)):
        if got[name] is None:
            continue
        h2 = _half_step(dz).square_().scatter_(1, made_good, 0.0)
        if name == "dW" and X.shape[0] <= 128:
            h2.zero_()
        left = h2 @ (W.double() ** 2) if name == "dX" else h2.t() @ (X.double() ** 2)
        bound = math.sqrt(float((_half_step(ref[name]) ** 2).sum()) + float(left.sum())) / math.sqrt(3.0)
        err = float((got[name].double() - ref[name]).norm())
        print(f"[{what} {name}: error norm {err:.3e}, bound {bound:.3e}, ratio {err / bound:.3f}]",
              flush=True)
        assert err <= 1.05 * bound, f"{what} {name}: {err:.3e} against {bound:.3e}"


def _targets(T, V, k, lab, seed):
    if not k:
        return None, None
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, V, (T, k), generator=g).cuda()
    idx[:, 0] = lab
    return idx, torch.randn(T, k, generator=g).cuda() * 2


# one row past the few-row kernels, each tile shape of dW and the launch it
# shares with dX, rows looked at in one and several passes, pieces of the vocabulary
@pytest.mark.parametrize("T,V,D,k", [(129, 3000, 256, 0), (129, 3000, 72, 3), (300, 2005, 136, 0),
                                     (600, 5003, 264, 4), (1100, 11001, 520, 0), (1100, 11001, 520, 5),
                                     (1000, 23001, 1032, 0), (4600, 3001, 264, 0), (4600, 3001, 264, 2),
                                     (9000, 17001, 136, 0), (9000, 17001, 136, 3)])
def test_gradients_of_many_rows_are_rounded_once(T, V, D, k):
    X, W, lab = problem(T, V, D, T + k, pull=4.0)
    idx, te = _targets(T, V, k, lab, k)
    dl = _dloss(T, 5)
    got = _run(X, W, lab, idx, te, dl)
    kw = dict(labels=lab) if idx is None else dict(index=idx, teacher=te)
    ref = reference(X, W, dloss=dl, **kw)
    _held_once(f"{T}x{V}x{D} k={k}", got, ref, X, W, lab, idx, te, dl)
    check(got, ref, f"{T}x{V}x{D} k={k}")


def test_more_groups_of_columns_than_one_workgroup_counts():
    """2^12 groups of 256 columns and more, rows in two chunks, few of them kept."""
    T, V, D = 4300, (1 << 20) + 70001, 8
    X, W, lab = problem(T, V, D, 9)
    out = torch.ones(T, dtype=torch.bool, device="cuda")
    out[::71] = False
    out[-1] = False
    lab[-1], lab[71], lab[142] = V - 1, 1 << 20, (1 << 20) - 1
    lab[out] = -100
    dl = _dloss(T, 7)
    check(_run(X, W, lab, None, None, dl), reference(X, W, labels=lab, dloss=dl), "many groups")


# few columns hold most of the targets: tiles with as many target rows as rows,
# tiles with none
@pytest.mark.parametrize("T,V,D,k,hot", [(700, 5003, 136, 0, 1), (700, 5003, 136, 6, 3), (5000, 3001, 264, 0, 2),
                                         (2500, 700, 520, 0, 700), (2500, 700, 520, 130, 700),
                                         (4300, 20001, 72, 9, 40)])
@pytest.mark.parametrize("alone", [False, True])
def test_common_targets(T, V, D, k, hot, alone):
    g = torch.Generator().manual_seed(T + k)
    X, W, _ = problem(T, V, D, T + k)
    cols = torch.randperm(V, generator=g)[:hot]
    lab = cols[torch.randint(0, hot, (T,), generator=g)].cuda()
    lab[::5] = -100
    idx = te = None
    if k:
        idx = cols[torch.randint(0, hot, (T, k), generator=g)].cuda()
        idx[::5] = -1
        te = torch.randn(T, k, generator=g).cuda() * 2
    dl = _dloss(T, 6)
    got = _run(X, W, lab, idx, te, dl, need_dX=not alone)
    kw = dict(labels=lab) if idx is None else dict(index=idx, teacher=te)
    ref = reference(X, W, dloss=dl, **kw)
    check(got, ref, "common targets")
    _held_once("common targets", got, ref, X, W, lab, idx, te, dl)
    again = _run(X, W, lab, idx, te, dl, need_dX=not alone)
    assert torch.equal(got["dW"], again["dW"])
