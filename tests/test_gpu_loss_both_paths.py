"""The linear head's losses on both sides of 128 rows, which take other kernels
(rows not selected, labels read where they are needed, the join among the picks,
G in two halves; and rows in the order of their targets), and what one side alone
was tested with: signs of the scale, bad targets, used workspaces, replays, repeats,
pieces of the vocabulary, wide heads, long pitches."""
import math

import pytest
import torch

import dense_gemm_linear_amd as dg
from loss_reference import check, problem, reference

pytestmark = pytest.mark.gpu


def _dloss(T, seed):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(T, generator=g) + 0.5) / T).cuda()


def _slots(T, V, k, lead, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, V, (T, k), generator=g)
    idx[:, 0] = lead.cpu()
    idx[torch.rand(T, k, generator=g) < 0.15] = -1
    return idx.cuda(), (torch.randn(T, k, generator=g) * 2).cuda()


def _run(X, W, tg, dl, ws=None, **kw):
    """tg: labels, or (index, teacher)."""
    if isinstance(tg, tuple):
        loss, lse, logp = dg.linear_distillation(X, W, *tg, workspace=ws, **kw)
        dX, dW = dg.linear_distillation_grad(X, W, *tg, lse, logp, dl, workspace=ws, **kw)
        return dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW)
    loss, lse = dg.linear_cross_entropy(X, W, tg, workspace=ws, **kw)
    dX, dW = dg.linear_cross_entropy_grad(X, W, tg, loss, lse, dl, workspace=ws, **kw)
    return dict(loss=loss, lse=lse, dX=dX, dW=dW)


def _ref(X, W, tg, dl, **kw):
    t = dict(index=tg[0], teacher=tg[1]) if isinstance(tg, tuple) else dict(labels=tg)
    return reference(X, W, dloss=dl, **t, **kw)


@pytest.mark.parametrize("T", [1, 30, 48, 100, 130, 300])
@pytest.mark.parametrize("scale,z_loss", [(-1.0, 0.0), (0.0, 0.0), (-0.3, 1e-2), (1.7, -1e-3)])
@pytest.mark.parametrize("k", [0, 5])
def test_scales(T, scale, z_loss, k):
    V, D = 1003, 136
    X, W, lab = problem(T, V, D, T + k)
    dl = _dloss(T, 1)
    tg = _slots(T, V, k, lab, 2) if k else lab
    kw = dict(scale=scale) if k else dict(scale=scale, z_loss=z_loss)
    check(_run(X, W, tg, dl, **kw), _ref(X, W, tg, dl, **kw), f"T {T} scale {scale} k {k}")


@pytest.mark.parametrize("T", [5, 40, 70, 300, 5000])
def test_targets_outside_the_vocabulary(T):
    V, D = 300, 64
    X, W, lab = problem(T, V, D, T)
    dl = _dloss(T, 3)
    bad = lab.clone()
    bad[1], bad[3], bad[4] = V, -7, 1 << 40
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[1] = mask[3] = mask[4] = True
    got = _run(X, W, bad, dl)
    assert bool(torch.isnan(got["loss"][mask]).all()) and bool(torch.isnan(got["dX"][mask]).all())
    assert bool(torch.isnan(got["dW"]).all())
    ref = _ref(X, W, torch.where(mask, -100, lab), dl)
    for name in ("loss", "lse", "dX"):
        err = (got[name].double() - ref[name]).abs()[~mask]
        assert bool((err <= ref[name + "_tol"][~mask] + 1e-37).all()), name
    idx, te = _slots(T, V, 4, lab, 4)
    idx[:5] = lab[:5, None]
    idx[1, 1], te[3, 2], te[4, 0] = V + 1, math.nan, math.inf
    got = _run(X, W, (idx, te), dl)
    assert bool(torch.isnan(got["loss"][mask]).all()) and bool(torch.isnan(got["dX"][mask]).all())
    clean = idx.clone()
    clean[mask] = -1
    ref = _ref(X, W, (clean, te.nan_to_num(0.0, 0.0)), dl)
    for name in ("loss", "lse", "logp", "dX"):
        err = (got[name].double() - ref[name]).abs()[~mask]
        assert bool((err <= ref[name + "_tol"][~mask] + 1e-37).all()), name


@pytest.mark.parametrize("T", [1, 48, 128, 4500])
@pytest.mark.parametrize("k", [0, 6])
def test_used_workspaces_repeats_and_replays(T, k):
    V, D = 3001, 136
    X, W, lab = problem(T, V, D, T)
    dl = _dloss(T, 5)
    lab[::3] = -100
    lab[0] = 7
    tg = _slots(T, V, k, lab, 6) if k else lab
    ws = torch.full((dg.linear_loss_workspace_bytes(T, V, D, k, backward=True),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    want = _run(X, W, tg, dl)
    check(want, _ref(X, W, tg, dl), f"T {T} k {k}")
    for fill in (0xFF, 0x7F, 0x00):
        ws.fill_(fill)
        got = _run(X, W, tg, dl, ws)
        assert all(torch.equal(got[n], want[n]) for n in want), f"workspace of {fill:#x}"
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = _run(X, W, tg, dl, ws)
    for i in range(4):
        X2, W2, lab2 = problem(T, V, D, 50 + i)
        X.copy_(X2)
        W.copy_(W2)
        if k:
            tg2 = _slots(T, V, k, lab2, 60 + i)
            tg[0].copy_(tg2[0])
            tg[1].copy_(tg2[1])
        else:
            tg.copy_(torch.where(torch.arange(T, device="cuda") % (i + 2) == 1, -100, lab2))
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in res.items()}
        want = _run(X, W, tg, dl)                   # eager work between the replays
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), f"replay {i}: {n}"


# several pieces of the vocabulary with heads wider than a tile: dX is added up
# over them, each gradient alone and both
@pytest.mark.parametrize("T,V,D,k", [(8192, 20001, 520, 0), (6000, 25003, 264, 3)])
@pytest.mark.parametrize("keep", [0.4, 1.0])
def test_gradients_over_pieces(T, V, D, k, keep):
    X, W, lab = problem(T, V, D, T + k)
    g = torch.Generator().manual_seed(8)
    lab = torch.where((torch.rand(T, generator=g) < keep).cuda(), lab, -100)
    tg = lab
    if k:
        idx, te = _slots(T, V, k, torch.where(lab >= 0, lab, -1), 9)
        idx[lab < 0] = -1
        tg = (idx, te)
    dl = _dloss(T, 7)
    ref = _ref(X, W, tg, dl)
    got = _run(X, W, tg, dl)
    check(got, ref, "pieces")
    if k:
        fn, args = dg.linear_distillation_grad, (X, W, *tg, got["lse"], got["logp"], dl)
    else:
        fn, args = dg.linear_cross_entropy_grad, (X, W, tg, got["loss"], got["lse"], dl)
    check(dict(dX=fn(*args, need_dW=False)[0], dW=fn(*args, need_dX=False)[1]), ref, "pieces, alone")


@pytest.mark.parametrize("T,V,D,k", [(5, 300, 65536, 0), (150, 300, 65536, 2), (40, 2003, 8200, 3), (300, 2003, 8192, 0)])
def test_wide_heads(T, V, D, k):
    X, W, lab = problem(T, V, D, T)
    tg = _slots(T, V, k, lab, 3) if k else lab
    dl = _dloss(T, 4)
    check(_run(X, W, tg, dl), _ref(X, W, tg, dl), f"{T}x{V}x{D}")


@pytest.mark.parametrize("T", [3, 140])
def test_the_longest_pitches(T):
    """Rows 2^21 elements apart; what lies between the rows of dX and dW stays."""
    V, D, P = 260, 72, 1 << 21
    X, W, lab = problem(T, V, D, T)
    big = torch.full((V, P), 3.0, dtype=torch.bfloat16, device="cuda")
    Wp, Xp = big[:, :D], torch.empty((T, P), dtype=torch.bfloat16, device="cuda")[:, :D]
    Wp.copy_(W)
    Xp.copy_(X)
    dW = torch.full((V, P), -7.0, dtype=torch.bfloat16, device="cuda")
    dX = torch.full((T, P), -7.0, dtype=torch.bfloat16, device="cuda")
    dl = _dloss(T, 4)
    loss, lse = dg.linear_cross_entropy(Xp, Wp, lab)
    dg.linear_cross_entropy_grad(Xp, Wp, lab, loss, lse, dl, dX=dX[:, :D], dW=dW[:, :D])
    torch.cuda.synchronize()
    check(dict(loss=loss, lse=lse, dX=dX[:, :D], dW=dW[:, :D]), _ref(X, W, lab, dl), "long pitches")
    for t in (dX, dW):
        assert bool((t[:, D:] == -7.0).all())


@pytest.mark.parametrize("T", [3, 140])
def test_weights_past_4_gib(T):
    """W and dW of more than 2^32 bytes.  All rows but the first and last hundred
    are zero, so the rest of the log-sum-exp is their number, and the rest of
    dW is one vector."""
    V, D, R = 530003, 4104, 100
    X, Wr, lab = problem(T, 2 * R, D, T)
    W = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    W[:R], W[V - R:] = Wr[:R], Wr[R:]
    labels = torch.where(lab < R, lab, lab - 2 * R + V)
    labels[1] = -100
    dl = _dloss(T, 4)
    got = _run(X, W, labels, dl)
    torch.cuda.synchronize()
    keep = labels >= 0
    Xd = X.double()
    z = Xd @ Wr.double().t()
    lse = torch.logsumexp(torch.cat([z, torch.full((T, 1), math.log(V - 2 * R), device="cuda", dtype=torch.float64)], 1), 1)
    loss = lse - z.gather(1, lab[:, None])[:, 0]
    # as loss_reference bounds them: the sums of z, the tile columns, the exponentials
    u = 2.0 ** -24
    ez = (D + 3) * u * (Xd.abs() @ Wr.double().abs().t()).max(1).values
    rng = z.max(1).values.clamp(min=0) - z.min(1).values.clamp(max=0)
    e_lse = ez + (64 + V / 2048 + 4 * rng) * u + 4 * u * lse.abs()
    assert bool(((got["lse"].double() - lse).abs() <= e_lse)[keep].all())
    assert bool(((got["loss"].double() - loss).abs() <= (e_lse + ez + 8 * u * loss.abs()))[keep].all())
    g = dl.double() * keep
    dz = torch.exp(z - lse[:, None]).scatter_add(1, lab[:, None], -torch.ones_like(lse)[:, None]) * g[:, None]
    e_dz = (dz.abs() + 2 * g[:, None] * torch.exp(z - lse[:, None])) * (2 * e_lse + (16 + 4 * rng) * u)[:, None]
    h = 2.0 ** -8
    dW = dz.t() @ Xd
    tol = e_dz.t() @ Xd.abs() + h * 1.01 * (dz.abs().t() @ Xd.abs()) + h * dW.abs()
    at = torch.cat([torch.arange(R), torch.arange(V - R, V)]).cuda()
    assert bool(((got["dW"][at].double() - dW).abs() <= tol + 1e-37).all())
    flat = (g * torch.exp(-lse)) @ Xd
    tol = h * 2.1 * ((g * torch.exp(-lse)) @ Xd.abs()) * 1.01
    for r0 in range(R, V - R, 100000):
        r1 = min(r0 + 100000, V - R)
        assert bool(((got["dW"][r0:r1].double() - flat).abs() <= tol + 1e-37).all()), r0
    dX = dz @ Wr.double()
    tol = e_dz @ Wr.double().abs() + h * 1.01 * (dz.abs() @ Wr.double().abs()) + h * dX.abs() + \
        V * u * (dz.abs() @ Wr.double().abs())
    assert bool(((got["dX"].double() - dX).abs() <= tol + 1e-37).all())
