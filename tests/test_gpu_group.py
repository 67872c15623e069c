"""Rows sorted by group, their products and gradients, and adapters on the GPU,
against their definitions in 64 bits (tests/group_reference.py states the bounds)."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import UBF, U32, activation, bf16, close, make_ids, product, sorted_slots

pytestmark = pytest.mark.gpu

MARK = 1234.0                  # what rows that are not written must keep


def _say(*a):
    print("[" + " ".join(str(x) for x in a) + "]", flush=True)


# T, k, groups, kind: one slot, sizes around 64, 1024 and 8192 (a wave's step, a
# workgroup's, where chunks begin), one group, all of 512, empty groups
SORTS = [(1, 1, 1, "random"), (1, 8, 64, "distinct"), (63, 1, 3, "random"), (65, 3, 512, "random"),
         (341, 3, 7, "distinct"), (1025, 1, 512, "random"), (8192, 1, 8, "one"), (4097, 2, 8, "distinct"),
         (4096, 1, 12, "random"), (4097, 1, 512, "random"), (8193, 1, 512, "random"), (3000, 64, 100, "random"), (300001, 4, 130, "random"), (140001, 2, 512, "distinct"), (5000, 1, 9, "runs")]


@pytest.mark.parametrize("T,k,groups,kind", SORTS)
def test_sort(T, k, groups, kind):
    _say("sort", T, k, groups, kind)
    ids = make_ids(T, k, groups, T + k, kind=kind)
    want = sorted_slots(ids, groups)
    got = dg.group_sort(ids.cuda(), groups)
    for g, w, name in zip(got, want, ("offsets", "order", "place")):
        assert torch.equal(g.cpu(), w), name


def test_sort_pitch_and_none():
    ids = make_ids(700, 5, 33, 1)
    wide = torch.full((700, 9), 2).cuda()
    wide[:, :5] = ids.cuda()
    for g, w in zip(dg.group_sort(wide[:, :5], 33), sorted_slots(ids, 33)):
        assert torch.equal(g.cpu(), w)
    one = make_ids(300, 1, 4, 2)
    wide = torch.full((300, 3), 1).cuda()
    wide[:, 0] = one[:, 0].cuda()
    for g, w in zip(dg.group_sort(wide[:, :1], 4), sorted_slots(one, 4)):
        assert torch.equal(g.cpu(), w)
    # extreme ids, and a batch in which no slot takes part
    ids = torch.tensor([[-(1 << 62)], [(1 << 62)], [1 << 32], [-1]]).cuda()
    off, order, place = dg.group_sort(ids, 5)
    assert off.tolist() == [0] * 6 and order.tolist() == [0, 1, 2, 3] and place.flatten().tolist() == [-1] * 4
    off, order, place = dg.group_sort(torch.empty(0, 2, dtype=torch.int64).cuda(), 5)
    assert off.tolist() == [0] * 6 and order.numel() == 0 and place.shape == (0, 2)


# T, k, groups, D: rows shorter than a piece, odd ones, one and several pieces a thread
ROWS = [(1, 1, 1, 1), (1, 8, 64, 2048), (5, 2, 3, 7), (9, 3, 4, 9), (130, 2, 8, 520), (597, 4, 60, 1031),
        (33, 64, 40, 8), (257, 8, 16, 4100)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8, torch.float32])
@pytest.mark.parametrize("T,k,groups,D", ROWS)
def test_gather(T, k, groups, D, dtype):
    _say("gather", T, k, groups, D, dtype)
    ids = make_ids(T, k, groups, T)
    off, order, place = sorted_slots(ids, groups)
    g = torch.Generator().manual_seed(D)
    X = torch.randint(0, 256, (T, D), generator=g).to(dtype)
    n = int(off[-1])
    want = X[order[:n].long() // k]
    for pad in (0, 3):
        Xd = torch.zeros(T, D + pad, dtype=dtype).cuda()
        Xd[:, :D] = X.cuda()
        out = torch.full((T * k, D + pad), 77, dtype=dtype).cuda()
        dg.group_gather(Xd[:, :D], place.cuda(), out=out[:, :D])
        out = out.cpu()
        assert torch.equal(out[:n, :D], want)
        assert bool((out[n:] == 77).all()) and bool((out[:, D:] == 77).all())


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,groups,D", ROWS)
def test_combine(T, k, groups, D, weighted):
    _say("combine", T, k, groups, D, weighted)
    ids = make_ids(T, k, groups, T, none=0.3)
    off, order, place = sorted_slots(ids, groups)
    n = int(off[-1])
    Y = bf16(T * k, D + 1, seed=1)[:, :D]
    Y[n:] = float("nan")                                    # never read
    w = torch.rand(T, k + 2, generator=torch.Generator().manual_seed(3))[:, 1:k + 1] if weighted else None
    got = torch.full((T, D + 1), MARK).bfloat16().cuda()
    dg.group_combine(Y.cuda(), place.cuda(), w.cuda() if weighted else None, out=got[:, :D])
    live = (place >= 0)[:, :, None]
    terms = torch.where(live, Y[place.clamp(min=0).long()].double(), 0.0)
    if weighted:
        terms = terms * w.double()[:, :, None]
    want = terms.sum(1)
    close(got[:, :D], want, UBF * want.abs() + k * U32 * terms.abs().sum(1), "out")
    assert bool((got[:, D] == MARK).all())


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,groups,D", ROWS)
def test_combine_grad(T, k, groups, D, weighted):
    _say("combine_grad", T, k, groups, D, weighted)
    ids = make_ids(T, k, groups, T, none=0.3)
    off, order, place = sorted_slots(ids, groups)
    n = int(off[-1])
    Y, dout = bf16(T * k, D, seed=1), bf16(T, D, seed=2)
    Y[n:] = float("nan")
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(3)) if weighted else torch.ones(T, k)
    dY = torch.full((T * k, D), MARK).bfloat16().cuda()
    wd = w.cuda() if weighted else None
    _, dw = dg.group_combine_grad(dout.cuda(), Y.cuda(), place.cuda(), wd, dY=dY)
    slots = order[:n].long()
    want = dout[slots // k].double() * w.reshape(-1)[slots].double()[:, None]
    close(dY[:n], want, UBF * want.abs() + U32 * want.abs(), "dY")
    assert bool((dY[n:] == MARK).all())
    live = (place >= 0)[:, :, None]
    terms = torch.where(live, Y[place.clamp(min=0).long()].double(), 0.0) * dout.double()[:, None, :]
    close(dw, terms.sum(2), (D + 2) * U32 * terms.abs().sum(2), "dweights")
    # one at a time, and in place of Y
    only, none = dg.group_combine_grad(dout.cuda(), None, place.cuda(), wd, need_dweights=False)
    assert none is None and torch.equal(only[:n], dY[:n])
    none, dw2 = dg.group_combine_grad(dout.cuda(), Y.cuda(), place.cuda(), wd, need_dY=False)
    assert none is None and torch.equal(dw, dw2)
    own = Y.cuda()
    _, dw2 = dg.group_combine_grad(dout.cuda(), own, place.cuda(), wd, dY=own)
    assert torch.equal(dw, dw2) and torch.equal(own[:n], dY[:n])


# T, k, groups, N, K, kind: from one row to several tiles a group; sizes around the
# tiles' 16, 32, 64, 128, 256 and the k-tiles' 32 and 64; empty groups; 512 groups
PRODUCTS = [(1, 1, 1, 8, 8, "random"), (1, 2, 8, 520, 136, "distinct"), (3, 1, 5, 33, 24, "random"),
            (40, 4, 64, 264, 200, "distinct"), (64, 8, 64, 1024, 264, "distinct"), (100, 1, 512, 72, 40, "random"),
            (90, 2, 6, 129, 72, "random"), (200, 2, 8, 384, 520, "distinct"), (257, 1, 1, 257, 64, "one"),
            (700, 2, 3, 1000, 136, "random"), (700, 2, 40, 1000, 72, "runs"), (1500, 2, 4, 2056, 520, "distinct"),
            (2100, 4, 6, 4104, 328, "random"), (300, 1, 2, 20008, 96, "random"), (33, 1, 2, 8200, 1032, "random"),
            (120, 1, 4, 520, 2056, "random")]


def _problem(T, k, groups, N, K, kind, sort=False):
    ids = make_ids(T, k, groups, T + N, kind=kind)
    off, order, place = sorted_slots(ids, groups)
    X, W = bf16(T, K, seed=1), bf16(groups, N, K, seed=2, scale=K ** -0.5)
    return off, order, place, X, W


def _per_group(off, order, k, X):
    rows = X[order.long() // k]
    for g in range(len(off) - 1):
        a, b = int(off[g]), int(off[g + 1])
        if b > a:
            yield g, a, b, rows[a:b]


@pytest.mark.parametrize("T,k,groups,N,K,kind", PRODUCTS)
def test_linear(T, k, groups, N, K, kind):
    _say("linear", T, k, groups, N, K, kind)
    off, order, place, X, W = _problem(T, k, groups, N, K, kind)
    S, n = T * k, int(off[-1])
    Xd, Wd, offd, orderd = X.cuda(), W.cuda(), off.cuda(), order.cuda()
    out = torch.full((S, N + 1), MARK).bfloat16().cuda()
    dg.group_linear(Xd, Wd, offd, orderd, slots=k, out=out[:, :N])
    want, err = torch.zeros(S, N, dtype=torch.float64), torch.zeros(S, N, dtype=torch.float64)
    for g, a, b, x in _per_group(off, order, k, X):
        want[a:b], err[a:b] = product(x, W[g])
    close(out[:n, :N], want[:n], err[:n], "Y")
    assert bool((out[n:] == MARK).all()) and bool((out[:, N] == MARK).all())
    # sorted rows, an aligned output: the same bits
    Xs = dg.group_gather(Xd, place.cuda())
    Y = dg.group_linear(Xs, Wd, offd)
    assert torch.equal(Y[:n], out[:n, :N].contiguous())


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,k,groups,N,K,kind", [PRODUCTS[i] for i in (2, 4, 6, 9, 11)])
def test_linear_gated(T, k, groups, N, K, kind, act):
    _say("gated", T, k, groups, N, K, act)
    off, order, place, X, W = _problem(T, k, groups, N, K, kind)
    S, n = T * k, int(off[-1])
    W = W * 2
    mul = bf16(S, N, seed=3)
    want, err = torch.zeros(S, N, dtype=torch.float64), torch.zeros(S, N, dtype=torch.float64)
    for g, a, b, x in _per_group(off, order, k, X):
        v, e = product(x, W[g])
        e = e - UBF * v.abs()
        f = activation(act, v)
        # slopes of the activations stay below 1.2; their own error: exponential
        # and reciprocal of fp32, an erf of absolute error 1.5e-7
        f_err = 1.2 * e + 2.0 ** -20 * (v.abs() + f.abs()) * (act is not None)
        want[a:b] = f * mul[a:b].double()
        err[a:b] = mul[a:b].double().abs() * f_err + UBF * want[a:b].abs() + U32 * want[a:b].abs()
    args = (X.cuda(), W.cuda(), off.cuda(), order.cuda())
    got = dg.group_linear(*args, slots=k, activation=act, mul=mul.cuda())
    close(got[:n], want[:n], err[:n], "Y")
    own = mul.cuda()
    dg.group_linear(*args, slots=k, activation=act, mul=own, out=own)
    assert torch.equal(own[:n], got[:n]) and torch.equal(own[n:].cpu(), mul[n:])
    if act:
        plain = dg.group_linear(*args, slots=k, activation=act)
        ones = dg.group_linear(*args, slots=k, activation=act, mul=torch.ones_like(own))
        assert torch.equal(plain[:n], ones[:n])
    odd = torch.zeros(S, N + 3).bfloat16().cuda()
    odd[:, 1:N + 1] = mul.cuda()
    got2 = torch.empty(S, N + 1).bfloat16().cuda()
    dg.group_linear(*args, slots=k, activation=act, mul=odd[:, 1:N + 1], out=got2[:, :N])
    assert torch.equal(got2[:n, :N], got[:n])


GRADS = [(T, k, G, (N + 7) // 8 * 8, K, kind) for T, k, G, N, K, kind in PRODUCTS]


@pytest.mark.parametrize("T,k,groups,N,K,kind", GRADS)
def test_linear_grad(T, k, groups, N, K, kind):
    _say("grad", T, k, groups, N, K, kind)
    off, order, place, X, W = _problem(T, k, groups, N, K, kind)
    S, n = T * k, int(off[-1])
    dY = bf16(S, N, seed=4)
    dY[n:] = float("nan")
    args = (dY.cuda(), X.cuda(), W.cuda(), off.cuda(), order.cuda())
    dX = torch.full((S, K + 1), MARK).bfloat16().cuda()
    dW = torch.full((groups, N, K), MARK).bfloat16().cuda()
    dg.group_linear_grad(*args, slots=k, dX=dX[:, :K], dW=dW)
    seen = set()
    for g, a, b, x in _per_group(off, order, k, X):
        seen.add(g)
        close(dX[a:b, :K], *product(dY[a:b], W[g].t()), f"dX of group {g}")
        close(dW[g], *product(dY[a:b].t(), x.t()), f"dW of group {g}")
    for g in set(range(groups)) - seen:
        assert not bool(dW[g].any()), g
    assert bool((dX[n:] == MARK).all()) and bool((dX[:, K] == MARK).all())
    only, none = dg.group_linear_grad(*args, slots=k, need_dW=False)
    assert none is None and torch.equal(only[:n], dX[:n, :K].contiguous())
    none, only = dg.group_linear_grad(*args, slots=k, need_dX=False)
    assert none is None and torch.equal(only, dW)
    Xs = torch.full((S, K), float("nan")).bfloat16().cuda()
    dg.group_gather(args[1], place.cuda(), out=Xs)
    dX2, dW2 = dg.group_linear_grad(args[0], Xs, args[2], args[3])
    assert torch.equal(dX2[:n], only.new_empty(0) if n == 0 else dX[:n, :K].contiguous()) and torch.equal(dW2, dW)


# T, groups, N, K, R, kind
ADAPTERS = [(1, 1, 8, 8, 8, "one"), (1, 4, 520, 264, 16, "one"), (1, 512, 4099, 2056, 72, "random"),
            (1, 3, 20011, 5000, 256, "one"), (1, 2, 9000, 40, 24, "random"), (2, 3, 1000, 4104, 16, "random"), (3, 2, 33, 24, 8, "random"),
            (16, 16, 136, 72, 40, "random"), (48, 64, 1032, 264, 16, "random"), (64, 512, 200, 136, 24, "random"),
            (130, 3, 257, 520, 32, "random"), (597, 16, 1000, 136, 32, "runs"), (700, 9, 2056, 264, 64, "random"),
            (2050, 30, 4104, 136, 128, "random"), (2050, 5, 4096, 72, 256, "runs"), (300, 2, 20008, 96, 8, "random"),
            (40, 3, 8200, 2056, 16, "random"), (700, 512, 640, 40, 8, "random")]


def _adapter_reference(X, W, A, B, scale, off, order):
    want, err = product(X, W)
    err = err - UBF * want.abs()
    for g, a, b, x in _per_group(off, order, 1, X):
        rows = order[a:b].long()
        s = 1.0 if scale is None else float(scale[g])
        u = x.double() @ A[g].double().t() * s
        # u in fp32 (its scale one rounding more), then in two bf16 halves
        u_err = (X.shape[1] + 3) * U32 * abs(s) * (x.double().abs() @ A[g].double().abs().t()) + UBF ** 2 * u.abs()
        Bg = B[g].double()
        want[rows] += u @ Bg.t()
        err[rows] += u_err @ Bg.abs().t() + (X.shape[1] + 2 * A.shape[1] + 2) * U32 * 1.01 * (u.abs() @ Bg.abs().t())
    # the sums of the shared part go on through the adapters' terms
    err = err + 2 * A.shape[1] * U32 * (X.double().abs() @ W.double().abs().t())
    return want, err + UBF * want.abs()


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("T,groups,N,K,R,kind", ADAPTERS)
def test_adapters(T, groups, N, K, R, kind, scaled):
    _say("adapters", T, groups, N, K, R, kind, scaled)
    ids = make_ids(T, 1, groups, T, none=0.0 if T == 1 else 0.2, kind=kind)
    off, order, place = sorted_slots(ids, groups)
    X, W = bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5)
    A, B = bf16(groups, R, K, seed=3, scale=K ** -0.5), bf16(groups, N, R, seed=4, scale=0.3)
    scale = 0.5 + torch.rand(groups, generator=torch.Generator().manual_seed(5)) if scaled else None
    dev = [t.cuda() for t in (X, W, A, B, off, order)]
    out = torch.full((T, N + 1), MARK).bfloat16().cuda()
    dg.linear_adapters(*dev, scale=None if scale is None else scale.cuda(), out=out[:, :N])
    close(out[:, :N], *_adapter_reference(X, W, A, B, scale, off, order), "Y")
    assert bool((out[:, N] == MARK).all())
    Y = dg.linear_adapters(*dev, scale=None if scale is None else scale.cuda())
    assert torch.equal(Y, out[:, :N].contiguous())


@pytest.mark.parametrize("T,groups,N,K,R", [(2, 2, 40, 64, 8), (48, 5, 300, 264, 16), (200, 4, 520, 136, 24),
                                            (600, 3, 2056, 72, 64)])
def test_adapters_keep_apart(T, groups, N, K, R):
    """An adapter with infinities and NaN, a row with them, and the memory of rows
    without an adapter reach no other row."""
    ids = make_ids(T, 1, groups, T, none=0.2)
    ids[0], ids[1] = 1, 0
    off, order, place = sorted_slots(ids, groups)
    X, W = bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5)
    A, B = bf16(groups, R, K, seed=3, scale=K ** -0.5), bf16(groups, N, R, seed=4, scale=0.3)
    ws = torch.full((dg.linear_adapters_workspace_bytes(T, R, groups),), 0xFF, dtype=torch.uint8).cuda()
    offd, orderd = off.cuda(), order.cuda()
    good = dg.linear_adapters(X.cuda(), W.cuda(), A.cuda(), B.cuda(), offd, orderd, workspace=ws).cpu()
    assert bool(torch.isfinite(good).all())
    B2, A2, X2 = B.clone(), A.clone(), X.clone()
    B2[1, ::3] = float("inf")
    B2[1, 1] = float("nan")
    A2[1, 2] = float("nan")
    rest = (ids[:, 0] != 1) | (torch.arange(T) == T)
    got = dg.linear_adapters(X.cuda(), W.cuda(), A2.cuda(), B2.cuda(), offd, orderd, workspace=ws).cpu()
    assert torch.equal(got[rest], good[rest]) and not bool(torch.isfinite(got[0]).any())
    X2[0] = float("nan")
    got = dg.linear_adapters(X2.cuda(), W.cuda(), A.cuda(), B.cuda(), offd, orderd, workspace=ws).cpu()
    assert torch.equal(got[1:], good[1:]) and bool(torch.isnan(got[0]).all())


@pytest.mark.parametrize("T,k,groups,N,K", [(40, 2, 4, 136, 72), (700, 2, 3, 520, 136)])
def test_linear_keeps_apart(T, k, groups, N, K):
    """NaN in one group's weight, in one token's row and behind the last row reach
    nothing else."""
    off, order, place, X, W = _problem(T, k, groups, N, K, "random")
    n, S = int(off[-1]), T * k
    args = (off.cuda(), order.cuda())
    good = dg.group_linear(X.cuda(), W.cuda(), *args, slots=k)[:n].cpu()
    W2, X2 = W.clone(), X.clone()
    W2[1] = float("nan")
    got = dg.group_linear(X.cuda(), W2.cuda(), *args, slots=k)[:n].cpu()
    a, b = int(off[1]), int(off[2])
    assert torch.equal(got[:a], good[:a]) and torch.equal(got[b:], good[b:]) and bool(torch.isnan(got[a:b]).all())
    X2[5] = float("inf")
    got = dg.group_linear(X2.cuda(), W.cuda(), *args, slots=k)[:n].cpu()
    other = (order[:n] // k) != 5
    assert torch.equal(got[other], good[other])
    # a group's NaN gradient rows stay in its own dX and dW
    dY = bf16(S, N, seed=4)
    dX, dW = dg.group_linear_grad(dY.cuda(), X.cuda(), W.cuda(), *args, slots=k)
    dY[a:b] = float("nan")
    dX2, dW2 = dg.group_linear_grad(dY.cuda(), X.cuda(), W.cuda(), *args, slots=k)
    keep = torch.ones(n, dtype=torch.bool)
    keep[a:b] = False
    assert torch.equal(dX2[:n].cpu()[keep], dX[:n].cpu()[keep])
    assert torch.equal(dW2[0], dW[0]) and torch.equal(dW2[2:], dW[2:]) and bool(torch.isnan(dW2[1]).all())
