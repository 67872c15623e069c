"""The grouped rows' operators on the host (CPU only): workspace sizes, and every
refusal of the C ABI and of the binding, before any device call."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import make_ids, sorted_slots

OK, E, U = dg.GEMM_OK, dg.GEMM_ERR_INVALID_VALUE, dg.GEMM_ERR_UNSUPPORTED
# fake device addresses: a call that is refused never looks at them
P = 0x10000
BIG = 1 << 40


def sort(ids=P, ld=2, T=8, k=2, groups=4, off=P, order=P, place=P, ws=P, nbytes=BIG):
    return dg.lib.group_sort(ids, ld, T, k, groups, off, order, place, ws, nbytes, None)


def gather(X=P, ldx=64, place=P, T=8, k=2, D=64, e=2, Xs=P, ldxs=64):
    return dg.lib.group_gather(X, ldx, place, T, k, D, e, Xs, ldxs, None)


def combine(Y=P, ldy=64, place=P, w=P, ldw=2, T=8, k=2, D=64, out=P, ldo=64):
    return dg.lib.group_combine(Y, ldy, place, w, ldw, T, k, D, out, ldo, None)


def combine_grad(dout=P, ldd=64, Y=P, ldy=64, place=P, w=P, ldw=2, T=8, k=2, D=64, dY=P, lddy=64, dw=P):
    return dg.lib.group_combine_grad(dout, ldd, Y, ldy, place, w, ldw, T, k, D, dY, lddy, dw, None)


def linear(X=P, ldx=64, W=P, ldw=64, stride=64 * 32, off=P, order=P, T=8, k=2, groups=4, N=32, K=64, act=0,
           mul=P, ldm=32, Y=P, ldy=32):
    return dg.lib.group_linear(X, ldx, W, ldw, stride, off, order, T, k, groups, N, K, act, mul, ldm, Y, ldy, None)


def linear_grad(dY=P, lddy=32, X=P, ldx=64, W=P, ldw=64, stride=64 * 32, off=P, order=P, T=8, k=2, groups=4,
                N=32, K=64, dX=P, lddx=64, dW=P, lddw=64, dstride=64 * 32, ws=P, nbytes=BIG):
    return dg.lib.group_linear_grad(dY, lddy, X, ldx, W, ldw, stride, off, order, T, k, groups, N, K, dX, lddx,
                                    dW, lddw, dstride, ws, nbytes, None)


def adapters(X=P, ldx=64, W=P, ldw=64, A=P, lda=64, sa=64 * 16, B=P, ldb=16, sb=16 * 32, scale=P, off=P,
             order=P, T=8, N=32, K=64, R=16, groups=4, Y=P, ldy=32, ws=P, nbytes=BIG):
    return dg.lib.linear_adapters(X, ldx, W, ldw, A, lda, sa, B, ldb, sb, scale, off, order, T, N, K, R, groups,
                                  Y, ldy, ws, nbytes, None)


LONG = (1 << 21) + 8
CASES = [
    (sort, [(dict(T=-1), E), (dict(k=0), E), (dict(groups=0), E), (dict(groups=513), U), (dict(k=65, ld=65), U),
            (dict(T=(1 << 24) + 1, k=1, ld=1), U), (dict(T=1 << 20, k=32, ld=32), U), (dict(ids=None), E),
            (dict(ids=P + 4), E), (dict(ld=1), E), (dict(off=None), E), (dict(off=P + 2), E), (dict(order=None), E),
            (dict(order=P + 1), E), (dict(place=None), E), (dict(T=4097, ws=None), E),
            (dict(T=4097, ws=P + 8), E), (dict(T=4097, nbytes=16), E)]),
    (gather, [(dict(T=-1), E), (dict(k=0), E), (dict(D=0), E), (dict(e=3), E), (dict(e=8), E), (dict(X=None), E),
              (dict(X=P + 1), E), (dict(ldx=63), E), (dict(place=None), E), (dict(place=P + 2), E),
              (dict(Xs=None), E), (dict(Xs=P + 1), E), (dict(ldxs=63), E), (dict(k=65), U),
              (dict(D=(1 << 20) + 1, ldx=BIG, ldxs=BIG), U)]),
    (combine, [(dict(T=-1), E), (dict(k=0), E), (dict(D=0), E), (dict(Y=None), E), (dict(Y=P + 1), E),
               (dict(ldy=63), E), (dict(place=None), E), (dict(w=P + 2), E), (dict(ldw=1), E), (dict(out=None), E),
               (dict(out=P + 1), E), (dict(ldo=63), E), (dict(k=65, ldw=65), U)]),
    (combine_grad, [(dict(T=-1), E), (dict(D=0), E), (dict(dout=None), E), (dict(ldd=63), E), (dict(Y=None), E),
                    (dict(ldy=63), E), (dict(place=None), E), (dict(w=P + 2), E), (dict(ldw=1), E),
                    (dict(dY=None, dw=None), E), (dict(dY=P + 1), E), (dict(lddy=63), E), (dict(dw=P + 2), E)]),
    (linear, [(dict(T=-1), E), (dict(k=0), E), (dict(groups=0), E), (dict(groups=513), U), (dict(N=0), E),
              (dict(K=0), E), (dict(K=60), U), (dict(K=1 << 17, ldx=1 << 17, ldw=1 << 17, stride=BIG), U),
              (dict(N=(1 << 20) + 1, stride=BIG), U), (dict(order=None), E), (dict(order=P + 2), E),
              (dict(off=None), E), (dict(off=P + 1), E), (dict(X=None), E), (dict(X=P + 8), E), (dict(ldx=56), E),
              (dict(ldx=68), E), (dict(ldx=LONG), U), (dict(W=None), E), (dict(W=P + 2), E), (dict(ldw=65), E),
              (dict(ldw=LONG, stride=BIG), U), (dict(stride=64), E), (dict(stride=64 * 32 + 4), E),
              (dict(stride=(1 << 40) + 8), U), (dict(act=5), E), (dict(act=-1), E), (dict(mul=P + 1), E),
              (dict(ldm=31), E), (dict(Y=None), E), (dict(Y=P + 1), E), (dict(ldy=31), E),
              # rows picked up by an order span less than 2 GiB
              (dict(T=1 << 19, k=1, ldx=1 << 12), U)]),
    (linear_grad, [(dict(T=-1), E), (dict(N=30), U), (dict(K=60), U), (dict(N=1 << 17, stride=BIG, dstride=BIG,
                                                                              lddy=1 << 17), U),
                   (dict(dY=None), E), (dict(dY=P + 8), E), (dict(lddy=36), E), (dict(lddy=24), E),
                   (dict(order=None), E), (dict(dX=None, dW=None), E), (dict(dX=P + 1), E), (dict(lddx=63), E),
                   (dict(dW=P + 1), E), (dict(lddw=63), E), (dict(dstride=64), E), (dict(ws=None), E),
                   (dict(ws=P + 16), E), (dict(nbytes=64), E), (dict(X=None), E), (dict(W=None), E),
                   (dict(T=0, dW=P + 1), E)]),
    (adapters, [(dict(T=-1), E), (dict(T=(1 << 20) + 1), U), (dict(R=0), E), (dict(R=12), U), (dict(R=264), U),
                (dict(K=60), U), (dict(N=0), E), (dict(groups=0), E), (dict(groups=513), U), (dict(A=None), E),
                (dict(A=P + 2), E), (dict(lda=56), E), (dict(sa=64), E), (dict(B=None), E), (dict(ldb=8), E),
                (dict(ldb=20), E), (dict(sb=16), E), (dict(scale=P + 2), E), (dict(off=None), E),
                (dict(order=None), E), (dict(Y=None), E), (dict(ldy=31), E), (dict(ws=None), E),
                (dict(ws=P + 128), E), (dict(nbytes=8), E), (dict(X=None), E), (dict(W=P + 8), E)]),
]


@pytest.mark.parametrize("call,bad,status", [(c, b, s) for c, cases in CASES for b, s in cases])
def test_c_refusals(call, bad, status):
    assert call(**bad) == status


def test_nothing_to_do():
    assert gather(T=0, X=None, place=None, Xs=None) == OK
    assert combine(T=0, Y=None, place=None, out=None) == OK
    assert combine_grad(T=0, dout=None, place=None) == OK
    assert linear(T=0, k=1, X=None, off=None, order=None, Y=None) == OK
    assert linear_grad(T=0, dY=None, X=None, dW=None) == OK
    assert adapters(T=0, X=None, Y=None, ws=None) == OK


def test_workspaces():
    assert dg.group_sort_workspace_bytes(4096, 1, 512) == 0
    assert dg.group_sort_workspace_bytes(4097, 1, 512) > 0
    assert dg.group_sort_workspace_bytes(-1, 1, 4) == 0 == dg.group_sort_workspace_bytes(8, 2, 513)
    assert dg.group_linear_grad_workspace_bytes(100, 3, 64) == 100 * 3 * 64 * 2
    assert dg.group_linear_grad_workspace_bytes(100, 3, 60) == 0
    # the inner values, and for few rows sums over slices of K
    assert dg.linear_adapters_workspace_bytes(1, 16, 4) >= 16 * 4
    assert dg.linear_adapters_workspace_bytes(2049, 16, 4) == 513 * 256
    assert dg.linear_adapters_workspace_bytes(100, 16, 4) > 100 * 16 * 4
    assert dg.linear_adapters_workspace_bytes(100, 12, 4) == 0 == dg.linear_adapters_workspace_bytes(1, 16, 0)


def _b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


X, W, PL, OFF, ORD = _b(8, 64), _b(4, 32, 64), _i(8, 2), _i(5), _i(16)
BINDING = [
    (lambda: dg.group_sort(torch.zeros(8, 2, dtype=torch.int32), 4), "int64"),
    (lambda: dg.group_sort(torch.zeros(8, 2, 2, dtype=torch.int64), 4), "contiguous rows"),
    (lambda: dg.group_sort([1, 2], 4), "int64"),
    (lambda: dg.group_gather(X.double(), PL), "1-, 2- or 4-byte"),
    (lambda: dg.group_gather(X, PL[:7]), "place"),
    (lambda: dg.group_gather(X, PL.long()), "int32"),
    (lambda: dg.group_gather(X, torch.zeros(8, 4, dtype=torch.int32)[:, :2]), "contiguous"),
    (lambda: dg.group_gather(X, PL, out=_b(15, 64)), "out"),
    (lambda: dg.group_gather(X.t(), PL), "contiguous rows"),
    (lambda: dg.group_combine(_b(15, 64), PL), "Y"),
    (lambda: dg.group_combine(_b(16, 64).float(), PL), "bfloat16"),
    (lambda: dg.group_combine(_b(16, 64), PL, torch.zeros(8, 3)), "weights"),
    (lambda: dg.group_combine(_b(16, 64), PL, _b(8, 2)), "float32"),
    (lambda: dg.group_combine(_b(16, 64), PL, out=_b(8, 63)), "out"),
    (lambda: dg.group_combine_grad(_b(7, 64), _b(16, 64), PL), "dout"),
    (lambda: dg.group_combine_grad(X, None, PL), "Y"),
    (lambda: dg.group_combine_grad(X, _b(16, 64), PL, need_dY=False, need_dweights=False), "neither"),
    (lambda: dg.group_combine_grad(X, _b(16, 64), PL, need_dY=False, dY=_b(16, 64)), "need_dY"),
    (lambda: dg.group_linear(X, _b(4, 32, 56), OFF, ORD, slots=2), "W"),
    (lambda: dg.group_linear(X, W, _i(4), ORD, slots=2), "offsets"),
    (lambda: dg.group_linear(X, W, OFF.long(), ORD, slots=2), "int32"),
    (lambda: dg.group_linear(X, W, OFF, ORD), "order"),
    (lambda: dg.group_linear(X, W, OFF, slots=2), "slots"),
    (lambda: dg.group_linear(X, W, OFF, ORD, slots=0), "slots"),
    (lambda: dg.group_linear(X, W, OFF, ORD, slots=2, mul=_b(15, 32)), "mul"),
    (lambda: dg.group_linear(X, W, OFF, ORD, slots=2, out=_b(16, 31)), "out"),
    (lambda: dg.group_linear(X.half(), W, OFF), "bfloat16"),
    (lambda: dg.group_linear(X, W.transpose(1, 2).contiguous().transpose(1, 2), OFF), "W"),
    (lambda: dg.group_linear_grad(_b(15, 32), X, W, OFF, ORD, slots=2), "dY"),
    (lambda: dg.group_linear_grad(_b(8, 32), X, W, OFF, need_dX=False, need_dW=False), "neither"),
    (lambda: dg.group_linear_grad(_b(8, 32), X, W, OFF, need_dW=False, dW=W), "need_dW"),
    (lambda: dg.linear_adapters(X, _b(32, 56), _b(4, 16, 64), _b(4, 32, 16), OFF, _i(8)), "W"),
    (lambda: dg.linear_adapters(X, _b(32, 64), _b(4, 16, 64), _b(4, 32, 8), OFF, _i(8)), "B"),
    (lambda: dg.linear_adapters(X, _b(32, 64), _b(4, 16, 64), _b(4, 32, 16), OFF, _i(7)), "order"),
    (lambda: dg.linear_adapters(X, _b(32, 64), _b(4, 16, 64), _b(4, 32, 16), OFF, _i(8), scale=torch.zeros(3)),
     "scale"),
    # everything in order, but not on a device
    (lambda: dg.group_sort(torch.zeros(8, 2, dtype=torch.int64), 4), "device"),
    (lambda: dg.group_gather(X, PL), "device"),
    (lambda: dg.group_combine(_b(16, 64), PL), "device"),
    (lambda: dg.group_combine_grad(X, _b(16, 64), PL), "device"),
    (lambda: dg.group_linear(X, W, OFF, ORD, slots=2), "device"),
    (lambda: dg.group_linear_grad(_b(8, 32), X, W, OFF), "device"),
    (lambda: dg.linear_adapters(X, _b(32, 64), _b(4, 16, 64), _b(4, 32, 16), OFF, _i(8)), "device"),
]


@pytest.mark.parametrize("call,word", BINDING)
def test_binding_refusals(call, word):
    with pytest.raises(ValueError, match=word):
        call()


@pytest.mark.parametrize("T,k,groups", [(1, 1, 1), (7, 3, 4), (40, 2, 9)])
def test_reference_sort(T, k, groups):
    """The reference's sort has the properties that define it."""
    ids = make_ids(T, k, groups, T)
    off, order, place = sorted_slots(ids, groups)
    flat = ids.reshape(-1)
    assert sorted(order.tolist()) == list(range(T * k))
    for g in range(groups):
        rows = order[int(off[g]):int(off[g + 1])].tolist()
        assert rows == sorted(rows) and all(int(flat[s]) == g for s in rows)
        assert all(int(place.reshape(-1)[s]) == int(off[g]) + i for i, s in enumerate(rows))
    n = int(off[-1])
    assert n == int(((flat >= 0) & (flat < groups)).sum())
    assert all(int(place.reshape(-1)[s]) == -1 for s in order[n:].tolist())
