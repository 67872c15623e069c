"""The grouped rows' operators as a program uses them: a whole layer of experts with
its gradients, graphs, streams, views, tables from elsewhere, buffers past 2 and 4 GiB."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import UBF, U32, bf16, close, make_ids, product, sorted_slots
from test_gpu_group import _adapter_reference, test_adapters as check_adapters

pytestmark = pytest.mark.gpu

MARK = 1234.0


def _say(*a):
    print("[" + " ".join(str(x) for x in a) + "]", flush=True)


# ---- a layer of experts, out = sum_j w_j down(silu(gate x) * up x)

class Layer:
    """The layer and its gradients from the operators, every buffer made once."""

    def __init__(self, T, k, G, D, H):
        S, b, f = T * k, torch.bfloat16, "cuda"
        self.k, self.G = k, G
        new = lambda *shape: torch.zeros(*shape, dtype=b, device=f)
        self.up, self.h, self.dh = new(S, H), new(S, H), new(S, H)
        self.gate, self.act = new(S, H), new(S, H)
        self.y, self.dy, self.out = new(S, D), new(S, D), new(T, D)
        self.dxs, self.dxs2 = new(S, D), new(S, D)
        self.sort_ws = torch.zeros(max(1, dg.group_sort_workspace_bytes(T, k, G)), dtype=torch.uint8, device=f)
        self.ws = torch.zeros(dg.group_linear_grad_workspace_bytes(T, k, D), dtype=torch.uint8, device=f)

    def forward(self, X, ids, w, Wg, Wu, Wd):
        self.off, self.order, self.place = dg.group_sort(ids, self.G, workspace=self.sort_ws)
        args = (self.off, self.order)
        dg.group_linear(X, Wu, *args, slots=self.k, out=self.up)
        dg.group_linear(X, Wg, *args, slots=self.k, activation="silu", mul=self.up, out=self.h)
        dg.group_linear(self.h, Wd, self.off, out=self.y)
        return dg.group_combine(self.y, self.place, w, out=self.out)

    def backward(self, dout, X, w, Wg, Wu, Wd):
        _, dw = dg.group_combine_grad(dout, self.y, self.place, w, dY=self.dy)
        _, dWd = dg.group_linear_grad(self.dy, self.h, Wd, self.off, dX=self.dh)
        # the gate again, and its gradients by the formula
        dg.group_linear(X, Wg, self.off, self.order, slots=self.k, out=self.gate)
        g, u, d = self.gate.float(), self.up.float(), self.dh.float()
        s = torch.sigmoid(g)
        dgate = (d * u * (s + g * s * (1 - s))).bfloat16()
        dup = (d * g * s).bfloat16()
        dX1, dWg = dg.group_linear_grad(dgate, X, Wg, self.off, self.order, slots=self.k, dX=self.dxs,
                                        workspace=self.ws)
        dX2, dWu = dg.group_linear_grad(dup, X, Wu, self.off, self.order, slots=self.k, dX=self.dxs2,
                                        workspace=self.ws)
        dX = dg.group_combine(dX1, self.place).float() + dg.group_combine(dX2, self.place).float()
        return dX, dw, dWg, dWu, dWd


def _layer_inputs(T, k, G, D, H, seed=0):
    ids = make_ids(T, k, G, seed + T, kind="distinct")
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(seed + 9))
    X, dout = bf16(T, D, seed=seed + 1), bf16(T, D, seed=seed + 2)
    Wg, Wu = bf16(G, H, D, seed=seed + 3, scale=D ** -0.5), bf16(G, H, D, seed=seed + 4, scale=D ** -0.5)
    Wd = bf16(G, D, H, seed=seed + 5, scale=H ** -0.5)
    return X, ids, w, Wg, Wu, Wd, dout


@pytest.mark.parametrize("T,k,G,D,H", [(1, 2, 4, 64, 40), (60, 2, 6, 136, 72), (700, 4, 16, 264, 136)])
def test_layer_against_autograd(T, k, G, D, H):
    """The whole layer and all its gradients against autograd in 64 bits.  Values are
    rounded to bf16 between the operators; every error is carried on to first order by
    the operators' formulas on absolute values, in 64 bits, with 5 % for the second."""
    _say("layer", T, k, G, D, H)
    X, ids, w, Wg, Wu, Wd, dout = _layer_inputs(T, k, G, D, H)
    L = Layer(T, k, G, D, H)
    dev = [t.cuda() for t in (X, ids, w, Wg, Wu, Wd)]
    out = L.forward(*dev)
    dX, dw, dWg, dWu, dWd = L.backward(dout.cuda(), dev[0], *dev[2:])

    x64, w64, g64, u64, d64 = (t.double().requires_grad_() for t in (X, w, Wg, Wu, Wd))
    want = torch.zeros(T, D, dtype=torch.float64)
    o_err, dx_err, dw_err = torch.zeros(T, D).double(), torch.zeros(T, D).double(), torch.zeros(T, k).double()
    e_Wg, e_Wu, e_Wd = (torch.zeros_like(t, dtype=torch.float64) for t in (Wg, Wu, Wd))
    B = UBF
    for e in range(G):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        x = x64[t]
        gate, up = x @ g64[e].t(), x @ u64[e].t()
        h = gate * torch.sigmoid(gate) * up
        y = h @ d64[e].t()
        want = want.index_add(0, t, w64[t, j][:, None] * y)
        with torch.no_grad():
            aX, aD = x.abs(), d64[e].abs()
            sums = lambda a, b, K: (K + 2) * U32 * (a @ b)              # of fp32 sums
            e_g = sums(aX, g64[e].abs().t(), D)                          # before any rounding
            e_u = sums(aX, u64[e].abs().t(), D) + B * up.abs()
            s = torch.sigmoid(gate)
            silu = gate * s
            # |silu'| <= 1.1; its own error as for the operator alone
            e_s = 1.1 * e_g + 2.0 ** -20 * (gate.abs() + silu.abs())
            e_h = e_s * up.abs() + silu.abs() * e_u + (B + U32) * h.abs()
            e_y = e_h @ aD.t() + sums(h.abs(), aD.t(), H) + B * y.abs()
            wt = w64[t, j][:, None].abs()
            o_err.index_add_(0, t, wt * (e_y + k * U32 * y.abs()))
            do = dout[t].double()
            dw_err[t, j] = (do.abs() * e_y).sum(1) + (D + 2) * U32 * (do.abs() * y.abs()).sum(1)
            dy = w64[t, j][:, None] * do
            e_dy = (B + U32) * dy.abs()
            dh = dy @ d64[e]
            e_dh = e_dy @ aD + sums(dy.abs(), aD, D) + B * dh.abs()
            e_Wd[e] = e_dy.t() @ h.abs() + dy.abs().t() @ e_h + sums(dy.abs().t(), h.abs(), len(t)) + \
                B * (dy.t() @ h).abs()
            # silu' = s + g s (1 - s), |silu''| <= 1/2; the gate's value is rounded here
            e_gr = e_g + B * gate.abs()
            slope = (s + gate * s * (1 - s)).abs()
            f = 2.0 ** -20
            dga, dua = (dh * up).abs() * slope, (dh * silu).abs()
            e_dg = e_dh * up.abs() * slope + dh.abs() * e_u * slope + (dh * up).abs() * (0.5 * e_gr + f) + B * dga
            e_du = e_dh * silu.abs() + dh.abs() * (1.1 * e_gr + f * gate.abs()) + B * dua
            for err, a, W, e_W in ((e_dg, dga, g64[e].abs(), e_Wg), (e_du, dua, u64[e].abs(), e_Wu)):
                e_W[e] = err.t() @ aX + sums(a.t(), aX, len(t)) + B * (a.t() @ aX)
                # joined rows are rounded once more
                dx_err.index_add_(0, t, err @ W + sums(a, W, H) + 2.2 * B * (a @ W))
    (want * dout.double()).sum().backward()
    live = (ids >= 0) & (ids < G)
    err = lambda e, v: 1.05 * e + 1e-30
    close(out, want.detach(), err(o_err, want) + UBF * want.detach().abs(), "out")
    close(dw, torch.where(live, w64.grad, 0.0), err(dw_err, 0), "dweights")
    close(dX, x64.grad, err(dx_err, 0) + U32 * x64.grad.abs(), "dX")
    for got, ref, e, name in ((dWg, g64, e_Wg, "dWgate"), (dWu, u64, e_Wu, "dWup"), (dWd, d64, e_Wd, "dWdown")):
        close(got, ref.grad, err(e, 0), name)


@pytest.mark.parametrize("T,k,G,N,K", [(5, 2, 3, 8, 16), (90, 3, 7, 40, 56), (300, 2, 4, 136, 24)])
def test_gradients_against_differences(T, k, G, N, K):
    """Small integers: every product, sum and difference is exact, so that a step
    along any direction changes <dout, out> by exactly what the gradient says."""
    g = torch.Generator().manual_seed(T)
    ints = lambda *shape: torch.randint(-1, 2, shape, generator=g).bfloat16()
    ids = make_ids(T, k, G, T)
    off, order, place = (t.cuda() for t in sorted_slots(ids, G))
    X, W, dout = ints(T, K).cuda(), ints(G, N, K).cuda(), ints(T, N).cuda()
    w = torch.randint(1, 3, (T, k), generator=g).float().cuda()

    def run(X, W, w):
        Y = dg.group_linear(X, W, off, order, slots=k)
        out = dg.group_combine(Y, place, w)
        return Y, out, float((out.double() * dout.double()).sum())

    Y, out, base = run(X, W, w)
    assert float(out.abs().max()) < 256                    # integers that bf16 holds
    dY, dw = dg.group_combine_grad(dout, Y, place, w)
    dXs, dW = dg.group_linear_grad(dY, X, W, off, order, slots=k)
    dX = dg.group_combine(dXs, place)
    assert max(float(t.abs().max()) for t in (dW, dX, dXs)) < 256
    for _ in range(3):
        step = ints(T, K).cuda()
        assert run(X + step, W, w)[2] - base == float((step.double() * dX.double()).sum())
        step = ints(G, N, K).cuda()
        assert run(X, W + step, w)[2] - base == float((step.double() * dW.double()).sum())
        step = torch.randint(0, 2, (T, k), generator=g).float().cuda()
        assert run(X, W, w + step)[2] - base == float((step.double() * dw.double()).sum())


# ---- graphs and streams

@pytest.mark.parametrize("T,k,G,D,H", [(1, 2, 8, 136, 264), (48, 4, 16, 264, 136), (2100, 3, 20, 520, 264)])
def test_layer_in_a_graph(T, k, G, D, H):
    """Forward and backward captured once and replayed on other inputs, with eager
    runs between; every replay gives the eager bits.  The eager layer has leaves and
    buffers of its own and lives on."""
    _say("graph", T, k, G, D, H)
    first = [t.cuda() for t in _layer_inputs(T, k, G, D, H)]
    L, eager = Layer(T, k, G, D, H), Layer(T, k, G, D, H)
    X, ids, w, Wg, Wu, Wd, dout = (t.clone() for t in first)

    def run(layer, X, ids, w, Wg, Wu, Wd, dout):
        out = layer.forward(X, ids, w, Wg, Wu, Wd)
        return (out, *layer.backward(dout, X, w, Wg, Wu, Wd))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(L, X, ids, w, Wg, Wu, Wd, dout)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(L, X, ids, w, Wg, Wu, Wd, dout)
    for replay in range(4):
        inputs = [t.cuda() for t in _layer_inputs(T, k, G, D, H, seed=50 * replay)]
        for into, new in zip((X, ids, w, Wg, Wu, Wd, dout), inputs):
            into.copy_(new)
        graph.replay()
        want = run(eager, *inputs)
        torch.cuda.synchronize()
        for a, b, name in zip(got, want, ("out", "dX", "dw", "dWg", "dWu", "dWd")):
            assert torch.equal(a, b), (replay, name)


@pytest.mark.parametrize("T,G,N,K,R", [(1, 4, 520, 264, 16), (48, 16, 520, 264, 16), (48, 4, 520, 264, 64),
                                       (700, 8, 1032, 264, 32)])
def test_adapters_in_a_graph(T, G, N, K, R):
    X, W = bf16(T, K, seed=1).cuda(), bf16(N, K, seed=2, scale=K ** -0.5).cuda()
    A, B = bf16(G, R, K, seed=3, scale=K ** -0.5).cuda(), bf16(G, N, R, seed=4, scale=0.3).cuda()
    ids = make_ids(T, 1, G, 0).cuda()
    ws = torch.zeros(dg.linear_adapters_workspace_bytes(T, R, G), dtype=torch.uint8).cuda()
    sort_ws = torch.zeros(1, dtype=torch.uint8).cuda()
    out = torch.zeros(T, N, dtype=torch.bfloat16).cuda()

    def run(X, ids, ws, out):
        off, order, _ = dg.group_sort(ids, G, workspace=sort_ws)
        return dg.linear_adapters(X, W, A, B, off, order, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(X, ids, ws, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(X, ids, ws, out)
    for replay in range(4):
        x2, i2 = bf16(T, K, seed=10 + replay).cuda(), make_ids(T, 1, G, replay).cuda()
        X.copy_(x2)
        ids.copy_(i2)
        graph.replay()
        want = run(x2, i2, None, None)
        torch.cuda.synchronize()
        assert torch.equal(out, want), replay


def test_two_streams():
    """Two layers at once, each on a stream and with workspaces of its own, give the
    bits that each gives alone; and so does each run again."""
    size = (900, 4, 24, 264, 136)
    inputs = [[t.cuda() for t in _layer_inputs(*size, seed=s)] for s in (0, 70)]
    layers = [Layer(*size) for _ in inputs]

    def run(layer, X, ids, w, Wg, Wu, Wd, dout):
        out = layer.forward(X, ids, w, Wg, Wu, Wd).clone()
        return (out, *layer.backward(dout, X, w, Wg, Wu, Wd))

    alone = [run(L, *i) for L, i in zip(layers, inputs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(4):
        got = []
        for st, L, i in zip(streams, layers, inputs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(L, *i))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---- views, single rows, nothing to do

@pytest.mark.parametrize("T,k,G,N,K", [(60, 2, 5, 136, 72), (900, 2, 3, 264, 136)])
def test_views(T, k, G, N, K):
    """Pitches, starts inside a row and gaps between groups change no bit and what
    lies between is not touched."""
    ids = make_ids(T, k, G, T)
    off, order, place = sorted_slots(ids, G)
    S, n = T * k, int(off[-1])
    offd, orderd = off.cuda(), order.cuda()
    X, W, dY = bf16(T, K, seed=1).cuda(), bf16(G, N, K, seed=2).cuda(), bf16(S, N, seed=3).cuda()
    Y = dg.group_linear(X, W, offd, orderd, slots=k)
    dX, dW = dg.group_linear_grad(dY, X, W, offd, orderd, slots=k)
    nan = lambda *shape: torch.full(shape, float("nan")).bfloat16().cuda()
    Xv, Wv, dYv = nan(T, K + 24)[:, 8:K + 8], nan(G, N + 3, K + 16)[:, 2:N + 2, 8:K + 8], nan(S, N + 16)[:, 16:]
    for v, t in ((Xv, X), (Wv, W), (dYv, dY)):
        v.copy_(t)
    for lead in (1, 8):
        big = torch.full((S, N + 17), MARK).bfloat16().cuda()
        v = big[:, lead:lead + N]
        dg.group_linear(Xv, Wv, offd, orderd, slots=k, out=v)
        assert torch.equal(v[:n], Y[:n])
        big[:n, lead:lead + N] = MARK
        assert bool((big == MARK).all())
        bx = torch.full((S, K + 24), MARK).bfloat16().cuda()
        bw = torch.full((G, N + 2, K + 24), MARK).bfloat16().cuda()
        vx, vw = bx[:, lead:lead + K], bw[:, 1:N + 1, lead:lead + K]
        dg.group_linear_grad(dYv, Xv, Wv, offd, orderd, slots=k, dX=vx, dW=vw)
        assert torch.equal(vx[:n], dX[:n]) and torch.equal(vw, dW)
        bx[:n, lead:lead + K] = MARK
        vw.fill_(MARK)
        assert bool((bx == MARK).all()) and bool((bw == MARK).all())


def test_one_row_of_any_pitch():
    """A single row's pitch says nothing, through the C ABI too: one of 0 or of 1
    gives the row alone."""
    N, K, G = 40, 24, 3
    X, W = bf16(1, K, seed=1).cuda(), bf16(G, N, K, seed=2).cuda()
    off = torch.tensor([0, 0, 1, 1], dtype=torch.int32).cuda()
    order = torch.zeros(1, dtype=torch.int32).cuda()
    want, err = product(X.cpu(), W[1].cpu())
    stream = torch.cuda.current_stream().cuda_stream
    for pitch in (0, 1):
        out = torch.full((N + 8,), MARK).bfloat16().cuda()
        assert dg.lib.group_linear(X.data_ptr(), pitch, W.data_ptr(), K, N * K, off.data_ptr(), order.data_ptr(), 1, 1,
                                   G, N, K, 0, None, 0, out.data_ptr(), pitch, stream) == dg.GEMM_OK
        close(out[:N], want[0], err[0], "Y")
        assert bool((out[N:] == MARK).all())
        dY = bf16(1, N, seed=3).cuda()
        dX = torch.full((K + 8,), MARK).bfloat16().cuda()
        dW = torch.full((G, N, K), MARK).bfloat16().cuda()
        assert dg.lib.group_linear_grad(dY.data_ptr(), pitch, X.data_ptr(), pitch, W.data_ptr(), K, N * K,
                                        off.data_ptr(), None, 1, 1, G, N, K, dX.data_ptr(), pitch, dW.data_ptr(), K,
                                        N * K, None, 0, stream) == dg.GEMM_OK
        v, e = product(dY.cpu(), W[1].cpu().t())
        close(dX[:K], v[0], e[0], "dX")
        assert bool((dX[K:] == MARK).all())
        v, e = product(dY.cpu().t(), X.cpu().t())
        close(dW[1], v, e, "dW")
        assert not bool(dW[0].any()) and not bool(dW[2].any())
    row = torch.empty(N, dtype=torch.bfloat16).cuda()
    dg.group_linear(X.as_strided((1, K), (1, 1)), W, off, order, out=row.as_strided((1, N), (1, 1)))
    close(row, want[0], err[0], "Y")


def test_no_tokens():
    G, N, K = 4, 16, 24
    new = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16).cuda()
    W = bf16(G, N, K, seed=2).cuda()
    off, order, place = dg.group_sort(torch.empty(0, 2, dtype=torch.int64).cuda(), G)
    assert dg.group_gather(new(0, K), place).shape == (0, K)
    assert dg.group_combine(new(0, K), place).shape == (0, K)
    dY, dw = dg.group_combine_grad(new(0, K), new(0, K), place)
    assert dY.shape == (0, K) and dw.shape == (0, 2)
    assert dg.group_linear(new(0, K), W, off, order, slots=2).shape == (0, N)
    dX, dW = dg.group_linear_grad(new(0, N), new(0, K), W, off, order, slots=2)
    assert dX.shape == (0, K) and not bool(dW.any())
    A, B = new(G, 8, K), new(G, N, 8)
    off, order, _ = dg.group_sort(torch.empty(0, 1, dtype=torch.int64).cuda(), G)
    assert dg.linear_adapters(new(0, K), bf16(N, K, seed=1).cuda(), A, B, off, order).shape == (0, N)


def test_narrow_matrices():
    """Rows far shorter than a tile is wide, in buffers that end with the last row."""
    for T, N, K in ((33, 8, 8), (64, 8, 16), (65, 16, 8), (97, 24, 8), (200, 8, 64)):
        _say("narrow", T, N, K)
        off = torch.tensor([0, T], dtype=torch.int32).cuda()
        X, W, dY = bf16(T, K, seed=1), bf16(1, N, K, seed=2), bf16(T, N, seed=3)
        dX, dW = dg.group_linear_grad(dY.cuda(), X.cuda(), W.cuda(), off)
        close(dX, *product(dY, W[0].t()), "dX")
        close(dW[0], *product(dY.t(), X.t()), "dW")


# ---- tables from elsewhere

def test_tables_that_are_none():
    """Offsets, orders and places that no sort wrote: rows come out unspecified, but
    nothing outside the buffers is written (the checks are the kernels' own)."""
    T, k, G, N, K = 70, 2, 5, 72, 40
    S = T * k
    X, W, dY = bf16(T, K, seed=1).cuda(), bf16(G, N, K, seed=2).cuda(), bf16(S, N, seed=3).cuda()
    A, B = bf16(G, 16, K, seed=4).cuda(), bf16(G, N, 16, seed=5).cuda()
    Wd = bf16(N, K, seed=6).cuda()
    w = torch.rand(T, k).cuda()
    big = 2 ** 31 - 1
    for numbers in ([0, S, 0, S, 0, S], [S, 0, 0, 0, 0, 0], [-5, 9, big, -big, 40, big], [big] * 6, [-big] * 6):
        off = torch.tensor(numbers, dtype=torch.int32).cuda()
        for order in (torch.arange(S, dtype=torch.int32), torch.full((S,), -1, dtype=torch.int32),
                      torch.full((S,), S, dtype=torch.int32), torch.full((S,), big, dtype=torch.int32),
                      torch.full((S,), 3, dtype=torch.int32)):
            order = order.cuda()
            _say("tables", numbers, int(order[0]))
            guard = lambda rows, cols: torch.full((rows + 64, cols), MARK).bfloat16().cuda()
            Y, dX, Z, Xs, O = guard(S, N), guard(S, K), guard(T, N), guard(S, K), guard(T, N)
            dW = guard(G * N, K)
            dg.group_linear(X, W, off, order, slots=k, out=Y[:S])
            dg.group_linear(X, W, off, order, slots=k, activation="silu", mul=dY, out=Y[:S])
            dg.group_linear_grad(dY, X, W, off, order, slots=k, dX=dX[:S], dW=dW[:G * N].view(G, N, K))
            dg.linear_adapters(X, Wd, A, B, off.clamp(max=T), order[:T].contiguous(), out=Z[:T])
            place = order.view(T, k)
            dg.group_gather(X, place, out=Xs[:S])
            dg.group_combine(dY, place, w, out=O[:T])
            dYo = guard(S, N)
            dg.group_combine_grad(O[:T], dY, place, w, dY=dYo[:S])
            torch.cuda.synchronize()
            for t, rows in ((Y, S), (dX, S), (Z, T), (Xs, S), (O, T), (dW, G * N), (dYo, S)):
                assert bool((t[rows:] == MARK).all())


# ---- past 2 and 4 GiB

def test_stacks_past_4_gib():
    """Groups' weights, their gradients and adapters more than 4 GiB apart: the same
    bits as close together."""
    T, k, G, N, K, R = 150, 2, 3, 136, 264, 24
    far = (1 << 31) + 64                                     # elements
    ids = make_ids(T, k, G, 1)
    off, order, _ = sorted_slots(ids, G)
    n = int(off[-1])
    off, order = off.cuda(), order.cuda()
    X, dY = bf16(T, K, seed=1).cuda(), bf16(T * k, N, seed=3).cuda()
    W = bf16(G, N, K, seed=2).cuda()
    room = torch.zeros(2 * far + (1 << 21), dtype=torch.bfloat16, device="cuda")
    Wf = room.as_strided((G, N, K), (far, K, 1))
    Wf.copy_(W)
    Y = dg.group_linear(X, W, off, order, slots=k)
    assert torch.equal(dg.group_linear(X, Wf, off, order, slots=k)[:n], Y[:n])
    dX, dW = dg.group_linear_grad(dY, X, W, off, order, slots=k)
    got, _ = dg.group_linear_grad(dY, X, Wf, off, order, slots=k, need_dW=False)
    assert torch.equal(got[:n], dX[:n])
    dg.group_linear_grad(dY, X, W, off, order, slots=k, need_dX=False, dW=Wf)
    assert torch.equal(Wf, dW)
    del Wf
    Wd = bf16(N, K, seed=7).cuda()
    for rank, rows in ((R, 150), (R, 20), (64, 150), (8, 40), (200, 150), (R, 1)):
        _say("adapters", rank, rows)
        off, order, _ = (t.cuda() for t in sorted_slots(make_ids(rows, 1, G, 2, none=0.1 * (rows > 1)), G))
        A, B = bf16(G, rank, K, seed=4, scale=K ** -0.5).cuda(), bf16(G, N, rank, seed=5, scale=0.3).cuda()
        want = dg.linear_adapters(X[:rows], Wd, A, B, off, order)
        Af, Bf = room.as_strided((G, rank, K), (far, K, 1)), room.as_strided((G, N, rank), (far, rank, 1), 1 << 20)
        Af.copy_(A)
        Bf.copy_(B)
        assert torch.equal(dg.linear_adapters(X[:rows], Wd, Af, Bf, off, order), want)


def test_rows_past_4_gib():
    """Sorted rows past 2 and 4 GiB: read, written, joined and summed right at the far
    end, whose rows are repeated in small buffers."""
    D, S = 2048, (1 << 20) + (1 << 18) + 40                  # 5.4 GB
    G, N = 3, 16
    tail = 1000
    big = torch.zeros(S, D, dtype=torch.bfloat16, device="cuda")
    rows = bf16(tail, D, seed=1).cuda()
    big[-tail:] = rows
    ends = [0, S - tail, S - 300, S]
    off = torch.tensor(ends, dtype=torch.int32).cuda()
    near = torch.tensor([0, 0, tail - 300, tail], dtype=torch.int32).cuda()
    W = bf16(G, N, D, seed=2, scale=D ** -0.5).cuda()
    Wn = bf16(G, D, N, seed=3).cuda()
    Y, want = dg.group_linear(big, W, off), dg.group_linear(rows, W, near)
    assert torch.equal(Y[-tail:], want) and not bool(Y[:-tail].any())
    dYs = bf16(tail, N, seed=4).cuda()
    dY = torch.zeros(S, N, dtype=torch.bfloat16, device="cuda")
    dY[-tail:] = dYs
    dX, dW = dg.group_linear_grad(dY, big, W, off)
    dXn, dWn = dg.group_linear_grad(dYs, rows, W, near)
    assert torch.equal(dX[-tail:], dXn) and torch.equal(dW[1:], dWn[1:]) and not bool(dW[0].any())
    assert not bool(dX[:-tail].any())
    # big as the gradient of outputs of D columns
    del dX
    xs = torch.zeros(S, N, dtype=torch.bfloat16, device="cuda")
    xs[-tail:] = dYs
    dX, dW = dg.group_linear_grad(big, xs, Wn, off)
    dXn, dWn = dg.group_linear_grad(rows, dYs, Wn, near)
    assert torch.equal(dX[-tail:], dXn) and torch.equal(dW[1:], dWn[1:])
    # rows by place, the last token at the far end
    T = S // 2
    place = torch.arange(S, dtype=torch.int32, device="cuda").view(T, 2)
    out = dg.group_combine(big, place)
    close(out[-100:], (rows[-200::2].double() + rows[-199::2].double()).cpu(),
          (UBF + 3 * U32) * (rows[-200::2].double().abs() + rows[-199::2].double().abs()).cpu(), "out")
    dYs, dw = dg.group_combine_grad(out, big, place)
    assert torch.equal(dYs[-200::2], out[-100:]) and torch.equal(dYs[-199::2], out[-100:])
    ref = (rows[-200:].double() * out[-100:].double().repeat_interleave(2, 0)).cpu()
    close(dw[-100:].reshape(-1), ref.sum(1), (D + 2) * U32 * ref.abs().sum(1), "dw")
    big.zero_()
    dg.group_gather(out, place, out=big)
    assert torch.equal(big[-200::2], out[-100:]) and torch.equal(big[-199::2], out[-100:])


# ---- the limits

@pytest.mark.parametrize("T,k,G", [(2 ** 24 - 1, 1, 512), (2 ** 18 - 1, 64, 3), (803000, 1, 130), (98 * 1024, 1, 7),
                                   (96 * 1024, 1, 512), (1025, 4, 512)])
def test_sort_of_many(T, k, G):
    """Up to the most slots there may be, against a stable sort of 64-bit integers."""
    _say("sort", T, k, G)
    ids = torch.randint(-1, G + 1, (T, k), generator=torch.Generator().manual_seed(T)).cuda()
    off, order, place = dg.group_sort(ids, G)
    key = torch.where((ids >= 0) & (ids < G), ids, G).reshape(-1)
    _, want = torch.sort(key, stable=True)
    assert torch.equal(order.long(), want)
    ends = torch.cumsum(torch.bincount(key.cpu(), minlength=G + 1), 0)[:G]
    assert int(off[0]) == 0 and torch.equal(off[1:].cpu().long(), ends)
    n = int(off[-1])
    at = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    at[want[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(place.reshape(-1), at)


def test_rows_of_most_tokens():
    """A workgroup a row and the most rows: 17 GB of them."""
    T, D = 2 ** 24 - 1, 520
    X = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    last = bf16(5, D, seed=1).cuda()
    X[-5:] = last
    place = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    Xs = dg.group_gather(X, place)
    assert torch.equal(Xs[:5], last.flip(0)) and not bool(Xs[5:].any())
    out = dg.group_combine(Xs, place)
    assert torch.equal(out[-5:], last) and not bool(out[:-5].any())
    dY, dw = dg.group_combine_grad(out, Xs, place)
    assert torch.equal(dY[:5], last.flip(0)) and not bool(dw[:-5].any())
    want = (last.double() ** 2).sum(1).cpu()
    close(dw[-5:, 0], want, (D + 2) * U32 * want, "dw")


def test_no_row_takes_part():
    T, k, G, N, K = 70, 2, 3, 72, 40
    ids = torch.full((T, k), -1).cuda()
    off, order, place = dg.group_sort(ids, G)
    X, W, dY = bf16(T, K, seed=1).cuda(), bf16(G, N, K, seed=2).cuda(), bf16(T * k, N, seed=3).cuda()
    Y = torch.full((T * k, N), MARK).bfloat16().cuda()
    dg.group_linear(X, W, off, order, slots=k, out=Y)
    dg.group_linear(X, W, off, order, slots=k, activation="relu", mul=dY, out=Y)
    dX = torch.full((T * k, K), MARK).bfloat16().cuda()
    _, dW = dg.group_linear_grad(dY, X, W, off, order, slots=k, dX=dX)
    assert bool((Y == MARK).all()) and bool((dX == MARK).all()) and not bool(dW.any())
    assert not bool(dg.group_combine(Y, place).any())
    dy, dw = dg.group_combine_grad(dY[:T].contiguous(), Y, place, dY=Y.clone())
    assert bool((dy == MARK).all()) and not bool(dw.any())
    Xs = torch.full((T * k, K), MARK).bfloat16().cuda()
    dg.group_gather(X, place, out=Xs)
    assert bool((Xs == MARK).all())
    for rows in (1, 20, 70):
        off, order, _ = dg.group_sort(ids[:rows, :1].contiguous(), G)
        A, B = bf16(G, 16, K, seed=4).cuda(), bf16(G, N, 16, seed=5).cuda()
        got = dg.linear_adapters(X[:rows], W[0], A, B, off, order)
        close(got, *product(X[:rows].cpu(), W[0].cpu()), "Y")


@pytest.mark.parametrize("T,k,G,N,K", [(3, 2, 2, 2 ** 20, 8), (2, 1, 2, 8, 2 ** 16), (130, 1, 2, 2 ** 16, 8),
                                       (150, 2, 2, 8, 2 ** 16)])
def test_widest(T, k, G, N, K):
    _say("widest", T, k, G, N, K)
    ids = make_ids(T, k, G, T)
    off, order, place = sorted_slots(ids, G)
    n = int(off[-1])
    X, W = bf16(T, K, seed=1), bf16(G, N, K, seed=2, scale=K ** -0.5)
    dev = X.cuda(), W.cuda(), off.cuda(), order.cuda()
    Y = dg.group_linear(*dev, slots=k)
    rows = order[:n].long() // k
    group = torch.bucketize(torch.arange(n), off[1:].long(), right=True)
    for g in range(G):
        at = torch.nonzero(group == g)[:, 0]
        close(Y[at.cuda()], *product(X[rows[at]], W[g]), f"Y of group {g}")
    if N > 2 ** 16:
        return
    dY = bf16(T * k, N, seed=3)
    dX, dW = dg.group_linear_grad(dY.cuda(), *dev, slots=k)
    for g in range(G):
        at = torch.nonzero(group == g)[:, 0]
        close(dX[at.cuda()], *product(dY[at], W[g].t()), f"dX of group {g}")
        close(dW[g], *product(dY[at].t(), X[rows[at]].t()), f"dW of group {g}")


def test_widest_rows():
    T, k, G, D = 3, 2, 2, 2 ** 20
    ids = make_ids(T, k, G, 1)
    off, order, place = sorted_slots(ids, G)
    n = int(off[-1])
    X = bf16(T, 2 * D, seed=1).cuda().view(torch.float32)
    Xs = dg.group_gather(X, place.cuda())
    assert torch.equal(Xs[:n].view(torch.int32), X.view(torch.int32)[(order[:n].long() // k).cuda()])
    Y, w = bf16(T * k, D, seed=2), torch.rand(T, k)
    out = dg.group_combine(Y.cuda(), place.cuda(), w.cuda())
    terms = torch.where((place >= 0)[:, :, None], Y[place.clamp(min=0).long()].double(), 0.0) * w.double()[:, :, None]
    close(out, terms.sum(1), UBF * terms.sum(1).abs() + k * U32 * terms.abs().sum(1), "out")


def test_adapters_of_most_rows():
    T, G, N, K, R = 2 ** 20, 512, 72, 64, 8
    ids = make_ids(T, 1, G, 5)
    X, W = bf16(T, K, seed=1), bf16(N, K, seed=2, scale=K ** -0.5)
    A, B = bf16(G, R, K, seed=3, scale=K ** -0.5), bf16(G, N, R, seed=4, scale=0.3)
    scale = torch.rand(G, generator=torch.Generator().manual_seed(5))
    off, order, _ = dg.group_sort(ids.cuda(), G)
    Y = dg.linear_adapters(X.cuda(), W.cuda(), A.cuda(), B.cuda(), off, order, scale=scale.cuda())
    some = torch.cat([torch.arange(300), torch.arange(T // 2, T // 2 + 300), torch.arange(T - 300, T)])
    o, p, _ = sorted_slots(ids[some], G)
    close(Y[some.cuda()], *_adapter_reference(X[some], W, A, B, scale, o, p), "Y")


# T, groups, N, K, R: few rows in slices of K and just too many for them, ranks around 16,
# 32, 64 and more, widths that are no multiple of 4
@pytest.mark.parametrize("T,groups,N,K,R", [(2, 2, 130, 8200, 8), (5, 3, 1001, 4104, 16), (33, 5, 600, 4104, 24),
                                            (65, 70, 129, 8200, 40), (130, 9, 1000, 2056, 64), (300, 4, 2050, 1000, 16),
                                            (512, 3, 264, 1032, 64), (513, 3, 264, 1032, 64), (100, 4, 3, 2056, 32),
                                            (1, 3, 333, 8200, 16), (1, 3, 1001, 1032, 256), (1, 2, 140003, 520, 256),
                                            (3, 2, 140003, 72, 16), (2048, 5, 100, 1032, 16), (2049, 5, 100, 1032, 16), (40, 5, 333, 1032, 256),
                                            (30, 5, 333, 4104, 136),
                                            (200, 512, 257, 1032, 72), (520, 3, 1000, 72, 16), (600, 20, 264, 136, 32),
                                            (900, 512, 72, 40, 24)])
def test_adapters_in_slices(T, groups, N, K, R):
    check_adapters(T, groups, N, K, R, "random", True)
    check_adapters(T, groups, N, K, R, "runs", False)
