"""linear_adapters and the grouped products on tables whose first row is not 0: a
range of the groups with their part of the offsets, rows of no group in front."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import bf16, close, product, sorted_slots, make_ids
from test_gpu_group import _adapter_reference

pytestmark = pytest.mark.gpu

MARK = 1234.0


# T, groups, N, K, R: one token; few rows in slices; whole products of few ranks and of
# more, with inner values of a row a workgroup (its rows' groups counted) and of tiles
SIZES = [(1, 3, 136, 264, 16), (1, 3, 40, 8200, 16), (48, 6, 300, 264, 16), (130, 5, 257, 520, 32),
         (3, 2, 140003, 72, 16), (600, 9, 2056, 72, 64), (2500, 7, 264, 136, 24)]


@pytest.mark.parametrize("T,groups,N,K,R", SIZES)
def test_adapters_of_a_range(T, groups, N, K, R):
    """Rows of groups before and behind the range take the projection alone."""
    print("[range", T, groups, N, K, R, "]", flush=True)
    ids = make_ids(T, 1, groups, T, none=0.2 if T > 1 else 0.0)
    ids[0, 0] = 0                                  # at least one row in front
    off, order, _ = sorted_slots(ids, groups)
    X, W = bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5)
    A, B = bf16(groups, R, K, seed=3, scale=K ** -0.5), bf16(groups, N, R, seed=4, scale=0.3)
    scale = 0.5 + torch.rand(groups, generator=torch.Generator().manual_seed(5))
    Xd, Wd, Ad, Bd, sd, offd, orderd = (t.cuda() for t in (X, W, A, B, scale, off, order))
    for g0, g1 in ((1, groups), (1, groups - 1), (groups - 1, groups)):
        if g0 >= g1:
            continue
        got = dg.linear_adapters(Xd, Wd, Ad[g0:g1], Bd[g0:g1], offd[g0:g1 + 1], orderd, scale=sd[g0:g1])
        want, err = _adapter_reference(X, W, A[g0:g1], B[g0:g1], scale[g0:g1], off[g0:g1 + 1], order)
        close(got, want, err, f"Y of groups {g0} to {g1}")


@pytest.mark.parametrize("T,N,K,R", [(1, 40, 72, 8), (48, 300, 264, 16), (600, 2056, 72, 64)])
def test_adapters_of_rows_in_front(T, N, K, R):
    """Every row stands before the first group's: none has an adapter."""
    X, W = bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5)
    A, B = bf16(2, R, K, seed=3), bf16(2, N, R, seed=4)
    off, order = torch.full((3,), T, dtype=torch.int32).cuda(), torch.arange(T, dtype=torch.int32).cuda()
    close(dg.linear_adapters(X.cuda(), W.cuda(), A.cuda(), B.cuda(), off, order), *product(X, W), "Y")


@pytest.mark.parametrize("T,k,groups,N,K", [(60, 2, 6, 136, 72), (900, 2, 5, 264, 136)])
def test_products_of_a_range(T, k, groups, N, K):
    """A range of the groups gives their rows and weights, and the rows before and behind
    stay as they are."""
    off, order, _ = sorted_slots(make_ids(T, k, groups, T), groups)
    X, W, dY = bf16(T, K, seed=1), bf16(groups, N, K, seed=2), bf16(T * k, N, seed=3)
    g0, g1 = 2, groups - 1
    part = (W[g0:g1].cuda(), off.cuda()[g0:g1 + 1], order.cuda())
    Y, dX = torch.full((T * k, N), MARK).bfloat16().cuda(), torch.full((T * k, K), MARK).bfloat16().cuda()
    dg.group_linear(X.cuda(), *part, slots=k, out=Y)
    _, dW = dg.group_linear_grad(dY.cuda(), X.cuda(), *part, slots=k, dX=dX)
    for g in range(g0, g1):
        a, b = int(off[g]), int(off[g + 1])
        x = X[order[a:b].long() // k]
        close(Y[a:b], *product(x, W[g]), f"Y of group {g}")
        close(dX[a:b], *product(dY[a:b], W[g].t()), f"dX of group {g}")
        close(dW[g - g0], *product(dY[a:b].t(), x.t()), f"dW of group {g}")
    a, b = int(off[g0]), int(off[g1])
    for t in (Y, dX):
        assert bool((t[:a] == MARK).all()) and bool((t[b:] == MARK).all())


def test_gradients_of_far_rows():
    """group_linear_grad with an order takes rows of X past 2 GiB; linear_adapters takes
    them in pieces."""
    T, G, N, K, tail = (1 << 20) - 8, 3, 24, 1032, 300
    ids = torch.full((T, 1), -1)
    ids[-tail:] = make_ids(tail, 1, G, 1)
    off, order, _ = dg.group_sort(ids.cuda(), G)
    n = int(off[-1])
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    rows, W, dYn = bf16(tail, K, seed=1), bf16(G, N, K, seed=2), bf16(n, N, seed=3)
    X[-tail:] = rows.cuda()
    dY = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    dY[:n] = dYn.cuda()
    dX, dW = dg.group_linear_grad(dY, X, W.cuda(), off, order)
    at = order[:n].cpu().long() - (T - tail)
    for g in range(G):
        a, b = int(off[g]), int(off[g + 1])
        close(dX[a:b], *product(dYn[a:b], W[g].t()), f"dX of group {g}")
        close(dW[g], *product(dYn[a:b].t(), rows[at[a:b]].t()), f"dW of group {g}")
    del dX, dY
    A, B, Wd = bf16(G, 8, K, seed=4, scale=K ** -0.5), bf16(G, N, 8, seed=5), bf16(N, K, seed=6, scale=K ** -0.5)
    dev = Wd.cuda(), A.cuda(), B.cuda()
    with pytest.raises(dg.GemmError):
        dg.linear_adapters(X, *dev, off, order)
    half = X[T // 2:]
    off, order, _ = dg.group_sort(ids[T // 2:].cuda(), G)
    Y = dg.linear_adapters(half, *dev, off, order)[-tail:]
    o, p, _ = sorted_slots(ids[-tail:], G)
    close(Y, *_adapter_reference(rows, Wd, A, B, None, o, p), "Y")
