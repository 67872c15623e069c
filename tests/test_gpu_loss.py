"""The linear head's losses on the GPU against their definitions in 64 bits
(tests/loss_reference.py states the error bounds)."""
import math

import pytest
import torch

import dense_gemm_linear_amd as dg
from loss_reference import check, problem, reference

pytestmark = pytest.mark.gpu

# T, V, D: one of everything, odd sizes around the tiles (32, 128, 256 rows;
# 128, 256 columns; 32, 64 values of K), one and several pieces of the vocabulary
SHAPES = [(1, 1, 8), (1, 50257, 64), (3, 7, 24), (17, 130, 64), (32, 1000, 136), (33, 257, 72),
          (130, 1003, 520), (257, 129, 40), (600, 5003, 136)]
LARGE = [(48, 3001, 136), (64, 700, 64), (128, 900, 200),   # one tile of rows
         (1, 40000, 264), (20, 33000, 72), (60, 40000, 72), (100, 17000, 200), (110, 40000, 72),  # one tile of rows
         (215, 9904, 264),        # 128 x 128 tiles of whole lines
         (3, 70001, 1000), (40, 131072, 1032),    # dW and W past half and all of the Infinity Cache
         (600, 11008, 72),        # the 256 x 256 tiles
         (400, 11007, 136), (300, 30011, 72),     # 128 x 192 tiles
         (600, 23001, 520),       # whole rounds of them, and the rest apart
         (1100, 11001, 520),      # and for dX
         (8192, 5003, 64), (20000, 7001, 16)]     # rows counted in chunks, two pieces of the vocabulary


def _say(*a):
    print("[" + " ".join(str(x) for x in a) + "]", flush=True)


def _dloss(T, seed):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(T, generator=g) + 0.5) / T).cuda()


def _run_ce(X, W, lab, dl, **kw):
    loss, lse = dg.linear_cross_entropy(X, W, lab, **kw)
    dX, dW = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, **kw)
    torch.cuda.synchronize()
    return dict(loss=loss, lse=lse, dX=dX, dW=dW)


def _run_di(X, W, idx, te, dl, **kw):
    loss, lse, logp = dg.linear_distillation(X, W, idx, te, **kw)
    dX, dW = dg.linear_distillation_grad(X, W, idx, te, lse, logp, dl, **kw)
    torch.cuda.synchronize()
    return dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW)


def _slots(T, V, k, lead, seed, empty=0.2):
    """Slots with the lead first, some empty, some naming a column twice."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, V, (T, k), generator=g)
    idx[:, 0] = lead.cpu()
    if k > 2:
        twice = torch.rand(T, generator=g) < 0.3
        idx[twice, 2] = idx[twice, 1]
    gone = torch.rand(T, k, generator=g) < empty
    gone[:, 0] &= torch.rand(T, generator=g) < 0.3
    te = torch.randn(T, k, generator=g).sort(dim=1, descending=True).values * 2
    idx[gone] = -1
    minus = torch.rand(T, k, generator=g) < 0.05
    te[minus] = -math.inf
    return idx.cuda(), te.cuda()


@pytest.mark.parametrize("T,V,D", SHAPES + LARGE)
def test_cross_entropy(T, V, D):
    _say("ce", T, V, D)
    X, W, lab = problem(T, V, D, T + V + D)
    dl = _dloss(T, 1)
    check(_run_ce(X, W, lab, dl), reference(X, W, labels=lab, dloss=dl), f"ce {T}x{V}x{D}")


@pytest.mark.parametrize("T,V,D,k", [(1, 1, 8, 1), (1, 5000, 64, 1), (3, 7, 24, 3), (33, 257, 72, 5),
                                     (130, 1003, 520, 64), (257, 129, 40, 65), (600, 5003, 136, 17),
                                     (40, 3000, 64, 256), (1100, 11001, 520, 9), (8192, 5003, 64, 4),
                                     (20000, 7001, 16, 2)])
def test_distillation(T, V, D, k):
    _say("distill", T, V, D, k)
    X, W, lead = problem(T, V, D, T + V + D + k)
    idx, te = _slots(T, V, k, lead, k)
    dl = _dloss(T, 2)
    check(_run_di(X, W, idx, te, dl, scale=0.5),
          reference(X, W, index=idx, teacher=te, dloss=dl, scale=0.5), f"distill {T}x{V}x{D} k={k}")


@pytest.mark.parametrize("scale,z_loss", [(1.0, 1e-4), (0.25, 0.0), (-1.0, 0.0), (1.7, 1e-2), (0.0, 0.0)])
def test_scale_and_z_loss(scale, z_loss):
    T, V, D = 130, 1003, 136
    X, W, lab = problem(T, V, D, 5)
    dl = _dloss(T, 3)
    check(_run_ce(X, W, lab, dl, scale=scale, z_loss=z_loss),
          reference(X, W, labels=lab, dloss=dl, scale=scale, z_loss=z_loss), f"scale {scale} z {z_loss}")


@pytest.mark.parametrize("T,V,D", [(30, 500, 72), (64, 500, 72), (127, 500, 72), (130, 1003, 136), (600, 11008, 72),
                                   (3000, 5003, 264)])
@pytest.mark.parametrize("keep", [0.0, 0.03, 0.5])
@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_rows_out(T, V, D, keep, kind):
    """Rows that are out: zeros, whatever their X holds, and the others' results
    as if they were not there."""
    _say("rows out", T, V, D, keep, kind)
    X, W, lead = problem(T, V, D, 6)
    g = torch.Generator().manual_seed(7)
    gone = (torch.rand(T, generator=g) >= keep).cuda()
    dl = _dloss(T, 4)
    Xp = X.clone()
    Xp[gone] = math.nan
    Xp[gone, 0] = math.inf
    if kind == "ce":
        lab = torch.where(gone, 11, torch.where(lead == 11, 12, lead))      # 11: a padding id
        got = _run_ce(Xp, W, lab, dl, ignore_index=11)
        ref = reference(X, W, labels=lab, dloss=dl, ignore_index=11)
    else:
        idx, te = _slots(T, V, 5, lead, 8, empty=0.0)
        idx[gone & (lead % 2 == 0)] = -1
        te[gone & (lead % 2 == 1)] = -math.inf
        got = _run_di(Xp, W, idx, te, dl)
        ref = reference(X, W, index=idx, teacher=te, dloss=dl)
    check(got, ref, f"{kind} keep {keep}")
    for name in ("loss", "lse", "logp", "dX"):
        if name in got:
            assert float(got[name][gone].abs().sum()) == 0.0, name


def test_confident_rows_keep_their_digits():
    """Labels of probability 1 - 1e-6: the loss and the gradient are small
    numbers with full relative accuracy (a difference lse - z would leave
    fp32's rounding of z, 20 % of them)."""
    V, D = 999, 64
    X = torch.zeros(4, D, device="cuda")
    W = torch.zeros(V, D, device="cuda")
    X[:, 0] = torch.tensor([20.0, 21.0, 22.0, 23.0])
    W[5, 0] = 1.0
    X, W = X.bfloat16(), W.bfloat16()
    lab = torch.full((4,), 5, device="cuda")
    loss, lse = dg.linear_cross_entropy(X, W, lab)
    want = torch.log1p((V - 1) * torch.exp(-X[:, 0].double()))
    assert bool(((loss.double() - want).abs() <= 2.0 ** -18 * want).all())
    # one row: dX = -(1 - p) W[5], one bf16 rounding of dz and one of dX
    dX, _ = dg.linear_cross_entropy_grad(X[:1], W, lab[:1], loss[:1], lse[:1],
                                         torch.ones(1, device="cuda"))
    gone = -torch.expm1(-want[0])
    assert abs(float(dX[0, 0]) + float(gone)) <= 2.02 * 2.0 ** -8 * float(gone)
    # distillation onto one column: the same loss
    idx, te = lab[:, None].contiguous(), torch.zeros(4, 1, device="cuda")
    l2, _, logp = dg.linear_distillation(X, W, idx, te)
    assert bool(((l2.double() - want).abs() <= 2.0 ** -18 * want).all())
    assert bool(((logp[:, 0].double() + want).abs() <= 2.0 ** -18 * want).all())


@pytest.mark.parametrize("T,V,D,k", [(1, 4000, 256, 0), (6, 9001, 136, 0), (100, 2000, 512, 0),
                                     (3, 4000, 256, 2), (128, 3000, 72, 5), (600, 3000, 256, 0),
                                     (600, 3000, 256, 4)])
def test_gradients_of_few_targets_are_rounded_once(T, V, D, k):
    """Where one target makes up a row of dX, or a few rows make up dW, the
    rounding of the logits' gradient to bf16 would show beside that of the
    result.  A rounding to nearest of a value of mantissa m in [1, 2) is off by
    at most 2^-8 / m, evenly: 2^-8 / (sqrt(3) m) root mean square, at most
    2^-8 / sqrt(3).  dX: one such rounding, and those of the columns that are no
    targets (independent, so the sum of their squares); dW of up to 128 rows:
    one, the rest of G going into a second half."""
    X, W, lab = problem(T, V, D, T + k, pull=8.0)
    dl = _dloss(T, 5)
    if k:
        g = torch.Generator().manual_seed(k)
        idx = torch.randint(0, V, (T, k), generator=g).cuda()
        idx[:, 0] = lab
        te = torch.randn(T, k, generator=g).cuda() * 3
        got, ref = _run_di(X, W, idx, te, dl), reference(X, W, index=idx, teacher=te, dloss=dl)
    else:
        idx = lab[:, None]
        got, ref = _run_ce(X, W, lab, dl), reference(X, W, labels=lab, dloss=dl)
    z = X.double() @ W.double().t()
    rest = torch.softmax(z, 1) * dl.double()[:, None]
    rest = rest.scatter(1, idx, 0.0)
    others = float(((rest * rest) @ (W.double() ** 2)).sum()) ** 0.5
    once = 2.0 ** -8 / math.sqrt(3.0)
    worst = {"dX": once * math.hypot(float(ref["dX"].norm()), others)}
    if T <= 128:
        worst["dW"] = once * float(ref["dW"].norm())
    for name, bound in worst.items():
        err = float((got[name].double() - ref[name]).norm())
        # 5 %: fp32 sums, and targets below 1/16
        assert err <= 1.05 * bound, f"{name}: {err:.3e} against {bound:.3e}"


def test_large_logits_do_not_overflow():
    T, V, D = 33, 700, 64
    X, W, lab = problem(T, V, D, 10, spread=60.0)
    dl = _dloss(T, 5)
    check(_run_ce(X, W, lab, dl), reference(X, W, labels=lab, dloss=dl), "large logits")


def test_targets_outside_the_vocabulary_are_loud():
    T, V, D = 70, 300, 64
    X, W, lab = problem(T, V, D, 11)
    dl = _dloss(T, 6)
    bad = lab.clone()
    bad[3], bad[40] = V, -7
    got = _run_ce(X, W, bad, dl)
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[3] = mask[40] = True
    assert bool(torch.isnan(got["loss"][mask]).all()) and bool(torch.isnan(got["dX"][mask]).all())
    assert bool(torch.isnan(got["dW"]).all())
    clean = lab.clone()
    clean[mask] = -100
    ref = reference(X, W, labels=clean, dloss=dl)
    for name in ("loss", "lse", "dX"):
        err = (got[name].double() - ref[name]).abs()[~mask]
        assert bool((err <= ref[name + "_tol"][~mask] + 1e-37).all()), name
    idx, te = _slots(T, V, 4, lab, 12, empty=0.0)
    te.clamp_(min=-5)
    idx[5, 1], te[6, 2], te[7, 0] = V + 1, math.nan, math.inf
    got = _run_di(X, W, idx, te, dl)
    for r in (5, 6, 7):
        assert math.isnan(float(got["loss"][r])) and bool(torch.isnan(got["dX"][r]).all()), r
    rest = [r for r in range(T) if r not in (5, 6, 7)]
    assert bool(torch.isfinite(got["loss"][rest]).all()) and bool(torch.isfinite(got["dX"][rest]).all())


@pytest.mark.parametrize("T,V,D,px,pw,pdx,pdw", [(70, 301, 72, 8, 16, 3, 5), (1, 40, 8, 0, 8, 1, 0),
                                                 (600, 11001, 72, 24, 8, 8, 8)])
def test_pitches_and_untouched_padding(T, V, D, px, pw, pdx, pdw):
    """Operands and outputs as column ranges of wider buffers: nothing outside
    the outputs' region is written."""
    _say("pitches", T, V, D)
    X, W, lab = problem(T, V, D, 13)
    Xw = torch.full((T, D + px), math.nan, dtype=torch.bfloat16, device="cuda")
    Ww = torch.full((V, D + pw), math.nan, dtype=torch.bfloat16, device="cuda")
    Xw[:, :D], Ww[:, :D] = X, W
    s = -7.0
    bx = torch.full((T + 2, D + pdx), s, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V + 2, D + pdw), s, dtype=torch.bfloat16, device="cuda")
    dl = _dloss(T, 7)
    Xv, Wv = Xw[:, :D], Ww[:, :D]
    loss, lse = dg.linear_cross_entropy(Xv, Wv, lab)
    dX, dW = dg.linear_cross_entropy_grad(Xv, Wv, lab, loss, lse, dl, dX=bx[1:T + 1, :D],
                                          dW=bw[1:V + 1, :D])
    torch.cuda.synchronize()
    check(dict(loss=loss, lse=lse, dX=dX, dW=dW), reference(X, W, labels=lab, dloss=dl), "pitches")
    for b, n in ((bx, T), (bw, V)):
        b[1:n + 1, :D] = s
        assert bool((b == s).all()), "wrote outside the output"


@pytest.mark.parametrize("T,V,D", [(100, 3001, 136), (20, 5003, 264),      # one tile of rows, in
                                   (100, 40000, 520),        # one launch and in two
                                   (400, 11007, 136), (1100, 11001, 520),  # dX and dW in one launch
                                   (300, 60001, 264), (8192, 5003, 64)])   # in two, in pieces
@pytest.mark.parametrize("keep", [0.0, 0.3, 1.0])
def test_each_gradient_alone(T, V, D, keep):
    """Each gradient within its bounds when asked for alone and together."""
    _say("alone", T, V, D, keep)
    X, W, lab = problem(T, V, D, 16)
    g = torch.Generator().manual_seed(17)
    lab = torch.where((torch.rand(T, generator=g) < keep).cuda(), lab, -100)
    dl = _dloss(T, 18)
    ref = reference(X, W, labels=lab, dloss=dl)
    loss, lse = dg.linear_cross_entropy(X, W, lab)
    dX, _ = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, need_dW=False)
    _, dW = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, need_dX=False)
    check(dict(dX=dX, dW=dW), ref, "alone")
    dX, dW = dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl)
    check(dict(dX=dX, dW=dW), ref, "together")


def test_one_gradient_one_weight_and_workspace_reuse():
    T, V, D, k = 130, 1003, 136, 6
    X, W, lead = problem(T, V, D, 14)
    idx, te = _slots(T, V, k, lead, 15)
    one = torch.full((1,), 0.125, device="cuda")
    ref = reference(X, W, index=idx, teacher=te, dloss=one)
    nbytes = dg.linear_loss_workspace_bytes(T, V, D, k, backward=True)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse, logp = dg.linear_distillation(X, W, idx, te, workspace=ws)
    dX, none = dg.linear_distillation_grad(X, W, idx, te, lse, logp, one, need_dW=False, workspace=ws)
    assert none is None
    ws.fill_(0xFF)
    none, dW = dg.linear_distillation_grad(X, W, idx, te, lse, logp, one.expand(T), need_dX=False,
                                           workspace=ws)
    assert none is None
    check(dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW), ref, "one at a time")
    with pytest.raises(ValueError, match="needed"):
        dg.linear_distillation(X, W, idx, te, workspace=ws[:64])
    with pytest.raises(ValueError, match="neither"):
        dg.linear_distillation_grad(X, W, idx, te, lse, logp, one, need_dX=False, need_dW=False)
    with pytest.raises(ValueError, match="dloss"):
        dg.linear_distillation_grad(X, W, idx, te, lse, logp, one.expand(3).contiguous())
    with pytest.raises(dg.GemmError):
        dg.linear_cross_entropy(X[:, :60], W[:, :60], lead)
    with pytest.raises(dg.GemmError):
        dg.linear_cross_entropy(X, W, lead, scale=math.nan)


def test_no_rows():
    X = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((50, 64), dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, device="cuda")
    lab = torch.zeros(0, dtype=torch.int64, device="cuda")
    got = _run_ce(X, W, lab, e)
    assert got["loss"].shape == (0,) and got["dX"].shape == (0, 64)
    assert got["dW"].shape == (50, 64) and float(got["dW"].abs().sum()) == 0.0


def test_most_rows():
    """2^20 rows, a third of them out, in chunks of the row count."""
    T, V, D = 1 << 20, 270, 8
    X, W, lab = problem(T, V, D, 24)
    lab[::3] = -100
    dl = torch.full((1,), 1.0, device="cuda")
    check(_run_ce(X, W, lab, dl), reference(X, W, labels=lab, dloss=dl), "2^20 rows")


def test_repeats_bitwise_and_on_another_stream():
    T, V, D, k = 600, 11008, 136, 8
    X, W, lead = problem(T, V, D, 16)
    idx, te = _slots(T, V, k, lead, 17)
    dl = _dloss(T, 8)
    a = _run_di(X, W, idx, te, dl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = _run_di(X, W, idx, te, dl)
    s.synchronize()
    c = _run_di(X, W, idx, te, dl)
    for name in a:
        assert torch.equal(a[name], b[name]) and torch.equal(a[name], c[name]), name


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, at the same time:
    the results of the calls one after the other."""
    problems = []
    for i, (T, V, D, k) in enumerate([(700, 9001, 264, 0), (300, 20011, 136, 7)]):
        X, W, lead = problem(T, V, D, 40 + i)
        tg = _slots(T, V, k, lead, 41) if k else (lead,)
        run = _run_di if k else _run_ce
        ws = torch.empty(dg.linear_loss_workspace_bytes(T, V, D, k, backward=True), dtype=torch.uint8,
                         device="cuda")
        dl = _dloss(T, 42)
        want = run(X, W, *tg, dl)
        problems.append((X, W, tg, dl, ws, bool(k), torch.cuda.Stream(), want))
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (X, W, tg, dl, ws, di, s, _want) in enumerate(problems):
            with torch.cuda.stream(s):
                if di:
                    loss, lse, logp = dg.linear_distillation(X, W, *tg, workspace=ws)
                    dX, dW = dg.linear_distillation_grad(X, W, *tg, lse, logp, dl, workspace=ws)
                    got[i] = dict(loss=loss, lse=lse, logp=logp, dX=dX, dW=dW)
                else:
                    loss, lse = dg.linear_cross_entropy(X, W, *tg, workspace=ws)
                    dX, dW = dg.linear_cross_entropy_grad(X, W, *tg, loss, lse, dl, workspace=ws)
                    got[i] = dict(loss=loss, lse=lse, dX=dX, dW=dW)
    torch.cuda.synchronize()
    for g, (*_rest, want) in zip(got, problems):
        for name in want:
            assert torch.equal(g[name], want[name]), name


def test_captured_and_replayed():
    """Forward and gradients of both losses in one graph, on one workspace;
    replays on new inputs give the eager results on them."""
    T, V, D, k = 200, 1003, 136, 4
    X, W, lab = problem(T, V, D, 18)
    idx, te = _slots(T, V, k, lab, 19)
    lab[::3] = -100
    dl = _dloss(T, 9)
    nbytes = dg.linear_loss_workspace_bytes(T, V, D, k, backward=True)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(X if n[1] == "X" else W) for n in ("aX", "aW", "bX", "bW")}

    def step(w):
        loss, lse = dg.linear_cross_entropy(X, W, lab, workspace=w)
        dg.linear_cross_entropy_grad(X, W, lab, loss, lse, dl, dX=out["aX"], dW=out["aW"], workspace=w)
        l2, s2, logp = dg.linear_distillation(X, W, idx, te, workspace=w)
        dg.linear_distillation_grad(X, W, idx, te, s2, logp, dl, dX=out["bX"], dW=out["bW"],
                                    workspace=w)
        return loss, lse, l2, s2, logp

    step(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(ws)
    for i in range(4):
        X2, W2, lab2 = problem(T, V, D, 30 + i)
        X.copy_(X2)
        W.copy_(W2)
        lab.copy_(torch.where(torch.arange(T, device="cuda") % (i + 2) == 0, -100, lab2))
        for t in out.values():
            t.fill_(math.nan)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res] + [t.clone() for t in out.values()]
        for t in out.values():
            t.fill_(math.nan)
        want = list(step(None)) + list(out.values())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), f"replay {i}"


def test_a_run_of_steps():
    """Forward, gradients and plain updates of X and W together, some steps,
    each step against the reference on that step's values; then the directional
    derivative of the loss against the gradients."""
    T, V, D = 300, 2005, 136
    X, W, lab = problem(T, V, D, 20)
    lab[::7] = -100
    dl = torch.full((1,), 1.0 / T, device="cuda")
    for step in range(3):
        got = _run_ce(X, W, lab, dl, z_loss=1e-3)
        ref = reference(X, W, labels=lab, dloss=dl, z_loss=1e-3)
        check(got, ref, f"step {step}")
        X = (X.float() - 5.0 * got["dX"].float()).bfloat16()
        W = (W.float() - 5.0 * got["dW"].float()).bfloat16()
    idx, te = _slots(T, V, 6, torch.where(lab >= 0, lab, 0), 21)
    check(_run_di(X, W, idx, te, dl), reference(X, W, index=idx, teacher=te, dloss=dl), "distill after")


def test_head_next_to_the_gemm():
    """The losses agree with the library's own GEMM on the same head: rows of
    logits from gemm_bf16 (rounded to bf16) give lse within that rounding."""
    T, V, D = 96, 1000, 128
    X, W, lab = problem(T, V, D, 22)
    z = dg.gemm_bf16(X, dg.shuffle_b(W), V).double()
    loss, lse = dg.linear_cross_entropy(X, W, lab)
    # each z off by at most half a bf16 step, so is the log-sum-exp
    tol = 2.0 ** -8 * z.abs().max(dim=1).values + 1e-4
    assert bool(((torch.logsumexp(z, 1) - lse.double()).abs() <= tol).all())
