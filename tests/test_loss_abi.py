"""The linear head's losses on the host (CPU only): workspace sizes, and every
refusal of the C ABI and of the binding, before any device call."""
import pytest
import torch

import dense_gemm_linear_amd as dg

OK, E, U = dg.GEMM_OK, dg.GEMM_ERR_INVALID_VALUE, dg.GEMM_ERR_UNSUPPORTED
# fake device addresses: a call that is refused never looks at them
PX, PW, PL, PI, PT, PO, PS = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000
BIG = 1 << 40
INF, NAN = float("inf"), float("nan")


def ce(X=PX, ldx=64, W=PW, ldw=64, labels=PL, T=8, V=100, D=64, scale=1.0, z=0.0, ignore=-100,
       loss=PO, lse=PO, ws=PS, nbytes=BIG):
    return dg.lib.linear_cross_entropy(X, ldx, W, ldw, labels, T, V, D, scale, z, ignore, loss, lse,
                                       ws, nbytes, None)


def ce_grad(X=PX, ldx=64, W=PW, ldw=64, labels=PL, T=8, V=100, D=64, scale=1.0, z=0.0, ignore=-100,
            loss=PO, lse=PO, dloss=PO, count=8, dX=PO, lddx=64, dW=PO, lddw=64, ws=PS, nbytes=BIG):
    return dg.lib.linear_cross_entropy_grad(X, ldx, W, ldw, labels, T, V, D, scale, z, ignore, loss,
                                            lse, dloss, count, dX, lddx, dW, lddw, ws, nbytes, None)


def di(X=PX, ldx=64, W=PW, ldw=64, index=PI, ldi=4, teacher=PT, ldt=4, T=8, V=100, D=64, k=4,
       scale=1.0, loss=PO, lse=PO, logp=PO, ws=PS, nbytes=BIG):
    return dg.lib.linear_distillation(X, ldx, W, ldw, index, ldi, teacher, ldt, T, V, D, k, scale,
                                      loss, lse, logp, ws, nbytes, None)


def di_grad(X=PX, ldx=64, W=PW, ldw=64, index=PI, ldi=4, teacher=PT, ldt=4, T=8, V=100, D=64, k=4,
            scale=1.0, lse=PO, logp=PO, dloss=PO, count=8, dX=PO, lddx=64, dW=PO, lddw=64, ws=PS,
            nbytes=BIG):
    return dg.lib.linear_distillation_grad(X, ldx, W, ldw, index, ldi, teacher, ldt, T, V, D, k,
                                           scale, lse, logp, dloss, count, dX, lddx, dW, lddw, ws,
                                           nbytes, None)


COMMON = [
    (dict(T=-1), E), (dict(V=0), E), (dict(D=0), E), (dict(D=-8), E),
    (dict(D=60, ldx=64, ldw=64), U), (dict(D=1 << 17, ldx=1 << 17, ldw=1 << 17), U),
    (dict(T=(1 << 20) + 1), U), (dict(V=(1 << 24) + 1), U),
    (dict(X=None), E), (dict(W=None), E), (dict(X=PX + 2), E), (dict(W=PW + 8), E),
    (dict(ldx=56), E), (dict(ldw=56), E), (dict(ldx=65), E), (dict(ldw=68), E),
    (dict(ldx=(1 << 21) + 8), U), (dict(ldw=(1 << 21) + 8), U),
    (dict(scale=INF), E), (dict(scale=NAN), E),
    (dict(ws=None), E), (dict(ws=PS + 16), E), (dict(nbytes=1), E),
]
GRAD = [
    (dict(dX=None, dW=None), E), (dict(dX=PO + 1), E), (dict(dW=PO + 1), E), (dict(lddx=63), E),
    (dict(lddw=63), E), (dict(lddw=(1 << 21) + 8), U), (dict(dloss=None), E), (dict(count=2), E),
    (dict(count=0), E), (dict(lse=None), E), (dict(lse=PO + 2), E),
]


@pytest.mark.parametrize("bad,status", COMMON)
@pytest.mark.parametrize("call", [ce, ce_grad, di, di_grad])
def test_common_refusals(call, bad, status):
    kw = dict(bad)
    if call in (ce_grad, di_grad) and "T" in kw:
        kw["count"] = 1
    if call in (ce_grad, di_grad) and kw.get("D", 0) > 64:
        kw.update(lddx=kw["D"], lddw=kw["D"])
    assert call(**kw) == status


@pytest.mark.parametrize("bad,status", GRAD)
@pytest.mark.parametrize("call", [ce_grad, di_grad])
def test_gradient_refusals(call, bad, status):
    assert call(**bad) == status


@pytest.mark.parametrize("call,bad,status", [
    (ce, dict(labels=None), E), (ce, dict(labels=PL + 4), E), (ce, dict(loss=None), E),
    (ce, dict(lse=None), E), (ce, dict(z=INF), E), (ce, dict(z=NAN), E),
    (ce_grad, dict(labels=None), E), (ce_grad, dict(loss=None), E), (ce_grad, dict(z=INF), E),
    (di, dict(index=None), E), (di, dict(teacher=None), E), (di, dict(index=PI + 4), E),
    (di, dict(teacher=PT + 2), E), (di, dict(k=0), E), (di, dict(k=257, ldi=300, ldt=300), U),
    (di, dict(ldi=3), E), (di, dict(ldt=3), E), (di, dict(logp=None), E), (di, dict(loss=None), E),
    (di_grad, dict(index=None), E), (di_grad, dict(logp=None), E), (di_grad, dict(k=-1), E),
    (di_grad, dict(ldt=3), E),
])
def test_target_refusals(call, bad, status):
    assert call(**bad) == status


def test_no_rows_is_no_work():
    assert ce(T=0, X=None, labels=None, loss=None, lse=None, ws=None, nbytes=0) == OK
    assert di(T=0, X=None, index=None, teacher=None, loss=None, lse=None, logp=None, ws=None,
              nbytes=0) == OK
    assert ce_grad(T=0, X=None, labels=None, loss=None, lse=None, dloss=None, dX=PO, dW=None,
                   ws=None, nbytes=0) == OK
    assert di_grad(T=0, X=None, index=None, teacher=None, lse=None, logp=None, dloss=None, dX=PO,
                   dW=None, ws=None, nbytes=0) == OK


def test_workspace_bytes():
    f = dg.linear_loss_workspace_bytes
    for bad in ((0, 100, 64), (8, 0, 64), (8, 100, 0), (8, 100, 60), (-1, 100, 64)):
        assert f(*bad) == 0
    assert f(8, 100, 64, -1) == 0 and f(8, 100, 64, 257) == 0
    for T, V, D, k in ((1, 50257, 512, 0), (1024, 50257, 512, 0), (8192, 131072, 4096, 64)):
        fwd, bwd = f(T, V, D, k), f(T, V, D, k, backward=True)
        assert 0 < fwd <= bwd
        # far below the logits of a long batch: the point of the operators
        if T == 8192:
            assert fwd < T * V * 2 // 4
        assert bwd < T * D * 2 + 64 * T * D * 4 + (260 << 20) + 64 * T * max(k, 1) + T * V // 8
    # one byte less than needed is refused
    need = f(8, 100, 64)
    assert ce(nbytes=need - 1) == E
    need = f(8, 100, 64, 4, True)
    assert di_grad(nbytes=need - 1) == E


def _x(T=4, D=16, dt=torch.bfloat16):
    return torch.zeros((T, D), dtype=dt)


def test_binding_checks_types_and_shapes():
    lab = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="X must be a bfloat16"):
        dg.linear_cross_entropy(_x(dt=torch.float16), _x(10), lab)
    with pytest.raises(ValueError, match="W must be a bfloat16"):
        dg.linear_cross_entropy(_x(), _x(10, dt=torch.float32), lab)
    with pytest.raises(ValueError, match="labels must be a torch.int64"):
        dg.linear_cross_entropy(_x(), _x(10), lab.int())
    with pytest.raises(ValueError, match="columns"):
        dg.linear_cross_entropy(_x(), _x(10, 24), lab)
    with pytest.raises(ValueError, match="vector of 4"):
        dg.linear_cross_entropy(_x(), _x(10), lab[:3])
    with pytest.raises(ValueError, match="vector of 4"):
        dg.linear_cross_entropy(_x(), _x(10), torch.zeros(8, dtype=torch.int64)[::2])
    with pytest.raises(ValueError, match="contiguous rows"):
        dg.linear_cross_entropy(_x(16, 4).t(), _x(10), lab)
    with pytest.raises(ValueError, match="device"):
        dg.linear_cross_entropy(_x(), _x(10), lab)
    idx, te = torch.zeros((4, 3), dtype=torch.int64), torch.zeros((4, 3))
    with pytest.raises(ValueError, match="index must be a torch.int64"):
        dg.linear_distillation(_x(), _x(10), idx.int(), te)
    with pytest.raises(ValueError, match="teacher must be a torch.float32"):
        dg.linear_distillation(_x(), _x(10), idx, te.bfloat16())
    with pytest.raises(ValueError, match="slots"):
        dg.linear_distillation(_x(), _x(10), idx, te[:, :2])
    with pytest.raises(ValueError, match="slots"):
        dg.linear_distillation(_x(), _x(10), idx[:3], te)
    with pytest.raises(ValueError, match="device"):
        dg.linear_distillation(_x(), _x(10), idx, te)
    v = torch.zeros(4)
    with pytest.raises(ValueError, match="loss must be a torch.float32"):
        dg.linear_cross_entropy_grad(_x(), _x(10), lab, v.double(), v, v)
    with pytest.raises(ValueError, match="logp must be a torch.float32"):
        dg.linear_distillation_grad(_x(), _x(10), idx, te, v, te.double(), v)
