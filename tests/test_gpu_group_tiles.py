"""Every instance of the grouped rows' products against the definitions in 64 bits, at
the sizes of group_tiles.py, with what is to keep apart on each."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import UBF, U32, activation, bf16, close, make_ids, product, sorted_slots
from group_tiles import ADAPTER_SIZES, DWS, DXS, FORWARDS
from test_gpu_group import _adapter_reference

pytestmark = pytest.mark.gpu

MARK = 1234.0


def _say(*a):
    print("[" + " ".join(str(x) for x in a) + "]", flush=True)


def _groups(off, order, k, X):
    """(group, first row, end, its rows of X)"""
    for g in range(len(off) - 1):
        a, b = int(off[g]), int(off[g + 1])
        if b > a:
            yield g, a, b, X[order[a:b].long() // k]


def _within(got, want_err, what):
    """close() with a reference on the device."""
    close(got, *(t.cpu() for t in want_err), what)


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("tile,T,k,groups,N,K", FORWARDS)
def test_forward(tile, T, k, groups, N, K):
    _say("forward", tile, T, k, groups, N, K)
    ids = make_ids(T, k, groups, T, kind="distinct" if k > 1 else "random")
    ids[T - 1, 0], ids[0, 0] = 0, groups - 1          # two groups that have rows
    off, order, place = (t.cuda() for t in sorted_slots(ids, groups))
    S, n = T * k, int(off[-1])
    X, W = bf16(T, K, seed=1).cuda(), bf16(groups, N, K, seed=2, scale=2 * K ** -0.5).cuda()
    mul = bf16(S, N, seed=3).cuda()
    Y, Z = (torch.full((S, N), MARK).bfloat16().cuda() for _ in range(2))
    dg.group_linear(X, W, off, order, slots=k, out=Y)
    dg.group_linear(X, W, off, order, slots=k, activation="silu", mul=mul, out=Z)
    for g, a, b, x in _groups(off, order, k, X):
        v, e = product(x, W[g])
        _within(Y[a:b], (v, e), f"Y of group {g}")
        # as for the gate's own test: slopes of SiLU below 1.2, its error 2^-20
        f, m = activation("silu", v), mul[a:b].double()
        want = f * m
        err = m.abs() * (1.2 * (e - UBF * v.abs()) + 2.0 ** -20 * (v.abs() + f.abs())) + (UBF + U32) * want.abs()
        _within(Z[a:b], (want, err), f"gated Y of group {g}")
    assert bool((Y[n:] == MARK).all()) and bool((Z[n:] == MARK).all())
    # the multiplier as output; views: the same bits, nothing between the rows touched
    own = mul.clone()
    dg.group_linear(X, W, off, order, slots=k, activation="silu", mul=own, out=own)
    assert _same(own[:n], Z[:n]) and _same(own[n:], mul[n:])
    wide = torch.full((S, N + 16), MARK).bfloat16().cuda()
    Xv = torch.full((T, K + 8), float("nan")).bfloat16().cuda()[:, :K]
    Xv.copy_(X)
    for lead in (8, 3):
        dg.group_linear(Xv, W, off, order, slots=k, out=wide[:, lead:lead + N])
        assert _same(wide[:n, lead:lead + N].contiguous(), Y[:n])
        wide[:n, lead:lead + N] = MARK
        assert bool((wide == MARK).all())
    # NaN and infinities of one group's weight and of one token stay where they are
    bad = W.clone()
    bad[0, ::2], bad[0, 1::2] = float("nan"), float("inf")
    got = dg.group_linear(X, bad, off, order, slots=k)
    a = int(off[1])
    assert _same(got[a:n], Y[a:n]) and not bool(torch.isfinite(got[:a]).any())
    x = X.clone()
    x[T - 1] = float("nan")
    got = dg.group_linear(x, W, off, order, slots=k, activation="silu", mul=mul)
    its = order[:n].long() // k == T - 1
    assert _same(got[:n][~its], Z[:n][~its]) and bool(torch.isnan(got[:n][its]).all())


@pytest.mark.parametrize("tile,T,k,groups,N,K", DXS + DWS)
def test_gradients(tile, T, k, groups, N, K):
    _say("gradients", tile, T, k, groups, N, K)
    ids = make_ids(T, k, groups, T, kind="distinct" if k > 1 else "random")
    off, order, place = (t.cuda() for t in sorted_slots(ids, groups))
    S, n = T * k, int(off[-1])
    X, W, dY = (t.cuda() for t in (bf16(T, K, seed=1), bf16(groups, N, K, seed=2), bf16(S, N, seed=4)))
    dY[n:] = float("nan")
    dX = torch.full((S, K + 1), MARK).bfloat16().cuda()
    dW = torch.full((groups, N, K), MARK).bfloat16().cuda()
    dg.group_linear_grad(dY, X, W, off, order, slots=k, dX=dX[:, :K], dW=dW)
    seen = set()
    for g, a, b, x in _groups(off, order, k, X):
        seen.add(g)
        _within(dX[a:b, :K], product(dY[a:b], W[g].t()), f"dX of group {g}")
        _within(dW[g], product(dY[a:b].t(), x.t()), f"dW of group {g}")
    for g in set(range(groups)) - seen:
        assert not bool(dW[g].any()), g
    assert bool((dX[n:] == MARK).all()) and bool((dX[:, K] == MARK).all())
    # a group's NaN stays in its own rows and weight
    last = max(seen)
    a, b = int(off[last]), int(off[last + 1])
    dY[a:b] = float("nan")
    dX2, dW2 = dg.group_linear_grad(dY, X, W, off, order, slots=k)
    assert _same(dX2[:a], dX[:a, :K].contiguous()) and _same(dW2[:last], dW[:last])
    assert bool(torch.isnan(dX2[a:b]).all()) and bool(torch.isnan(dW2[last]).all())


def _adapters(T, groups, N, K, R, none=0.2):
    ids = make_ids(T, 1, groups, T, none=none if T > 2 else 0.0, kind="runs" if T % 2 else "random")
    ids[T - 1], ids[0] = 0, groups - 1
    off, order, _ = (t.cuda() for t in sorted_slots(ids, groups))
    return (ids.cuda(), off, order) + tuple(t.cuda() for t in (
        bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5), bf16(groups, R, K, seed=3, scale=K ** -0.5),
        bf16(groups, N, R, seed=4, scale=0.3), 0.5 + torch.rand(groups, generator=torch.Generator().manual_seed(5))))


@pytest.mark.parametrize("form,T,groups,N,K,R", ADAPTER_SIZES)
def test_adapters(form, T, groups, N, K, R):
    _say("adapters", form, T, groups, N, K, R)
    ids, off, order, X, W, A, B, scale = _adapters(T, groups, N, K, R)
    ws = torch.full((dg.linear_adapters_workspace_bytes(T, R, groups),), 0xFF, dtype=torch.uint8).cuda()
    out = torch.full((T, N + 1), MARK).bfloat16().cuda()
    dg.linear_adapters(X, W, A, B, off, order, scale=scale, out=out[:, :N], workspace=ws)
    _within(out[:, :N], _adapter_reference(X, W, A, B, scale, off, order), "Y")
    assert bool((out[:, N] == MARK).all())
    good = dg.linear_adapters(X, W, A, B, off, order, scale=scale, workspace=ws)
    assert _same(good, out[:, :N].contiguous())
    # an adapter's and a row's NaN and infinities reach no other row
    A2, B2, X2 = A.clone(), B.clone(), X.clone()
    last = int(ids[T - 1])
    A2[last, R // 2] = float("nan")
    B2[last, ::3] = float("inf")
    rest = ids[:, 0] != last
    got = dg.linear_adapters(X, W, A2, B2, off, order, scale=scale, workspace=ws)
    assert _same(got[rest], good[rest]) and not bool(torch.isfinite(got[T - 1]).any())
    X2[T - 1] = float("nan")
    got = dg.linear_adapters(X2, W, A, B, off, order, scale=scale, workspace=ws)
    assert _same(got[:T - 1], good[:T - 1]) and bool(torch.isnan(got[T - 1]).all())


@pytest.mark.parametrize("form,T,groups,N,K,R", [s for s in ADAPTER_SIZES if s[0].startswith("whole")])
def test_adapters_without_rows(form, T, groups, N, K, R):
    """No row has an adapter."""
    _say("no rows", form, T, groups, N, K, R)
    ids, off, order, X, W, A, B, scale = _adapters(T, groups, N, K, R)
    off.zero_()
    _within(dg.linear_adapters(X, W, A, B, off, order), product(X, W), "Y")


@pytest.mark.parametrize("T,groups,N,K,R", [(2438, 3, 9, 264, 24), (294, 4, 9, 552, 208), (620, 3, 193, 536, 224),
                                            (4758, 3, 793, 264, 64), (2708, 3, 3049, 264, 136)])
def test_adapters_past_2_gib(T, groups, N, K, R):
    """Adapters so far apart that 32-bit offsets into B do not reach them: a k-tile of
    the ranks is of one adapter."""
    _say("apart", T, groups, N, K, R)
    ids, off, order, X, W, A, B, scale = _adapters(T, groups, N, K, R)
    far = (1 << 30) + 64                                     # elements
    room = torch.zeros((groups - 1) * far + N * R, dtype=torch.bfloat16, device="cuda")
    Bf = room.as_strided((groups, N, R), (far, R, 1))
    Bf.copy_(B)
    got = dg.linear_adapters(X, W, A, Bf, off, order, scale=scale)
    _within(got, _adapter_reference(X, W, A, B, scale, off, order), "Y")


@pytest.mark.parametrize("T,groups,N,K,R", [(2438, 6, 9, 72, 24), (294, 70, 9, 552, 208), (3420, 6, 133, 72, 248),
                                            (4758, 70, 793, 264, 64), (2708, 6, 3049, 264, 136)])
def test_adapter_tables_that_are_none(T, groups, N, K, R):
    """Offsets and orders that no sort wrote, in whole products: nothing outside the
    buffers is written (the checks are the kernels' own)."""
    ids, off, order, X, W, A, B, scale = _adapters(T, groups, N, K, R)
    big = 2 ** 31 - 1
    some = ([0, T], [T, 0], [-5, 9, big, -big, 40, big], [big], [-big], [T // 2, T, 0])
    for numbers in some:
        off = torch.tensor((numbers * (groups + 1))[:groups + 1], dtype=torch.int32).cuda()
        for order in (torch.arange(T, dtype=torch.int32), torch.full((T,), -1, dtype=torch.int32),
                      torch.full((T,), T, dtype=torch.int32), torch.full((T,), big, dtype=torch.int32)):
            _say("tables", T, N, R, numbers, int(order[0]))
            Y = torch.full((T + 64, N), MARK).bfloat16().cuda()
            dg.linear_adapters(X, W, A, B, off, order.cuda(), scale=scale, out=Y[:T])
            torch.cuda.synchronize()
            assert bool((Y[T:] == MARK).all())
