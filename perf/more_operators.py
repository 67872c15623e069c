"""What is measured of linear layers whose weight depends on the row, and what
they are held against.

Every row of X belongs to a group: the experts that a router chose for a token,
the adapter of the request that a token is of.  Work runs over slots sorted by
group, a slot being one choice of one token (T tokens with k choices each).

  "route"     tokens sorted by expert and back: offsets, order and place of the
              slots, the rows of X in that order, and the experts' outputs
              joined again with the router's weights.  A "step" adds the
              gradients: of X from the sorted rows', of the experts' outputs
              and of the weights from the joined rows'.
  "experts"   every slot's row times its expert's weight, X taken as it lies
              (not sorted).  "forward" is one product, "gated" has the fused
              SiLU and multiplier of a gated feed-forward layer, "step" adds
              the gradients of the sorted rows and of all weights.
  "adapters"  X W^T for every row, plus scale * (X A^T) B^T with the row's own
              low-rank A and B: one batch with the requests of many adapters.

Slots with id -1 (padding, rows without an adapter) take no part.
"""
import math

import torch

own = False


def _route(name, kind, T, k, E, D, keep=1.0):
    return {"name": name, "op": "route", "pass": kind, "T": T, "k": k, "E": E, "D": D, "keep": keep}


def _experts(name, kind, T, k, E, N, K, keep=1.0):
    return {"name": name, "op": "experts", "pass": kind, "T": T, "k": k, "E": E, "N": N, "K": K,
            "keep": keep}


def _adapters(name, T, N, K, R, E, used, keep=1.0):
    return {"name": name, "op": "adapters", "pass": "forward", "T": T, "k": 1, "E": E, "N": N, "K": K,
            "R": R, "used": used, "keep": keep}


def listed():
    return [
        # one decoded token through a router of many small experts: latency
        _route("route_forward_1x8of64_2048", "forward", 1, 8, 64, 2048),
        # a prompt through few large experts
        _route("route_forward_4095x2of8_4096", "forward", 4095, 2, 8, 4096),
        # a fine-tuning step of odd width, a fifth of the tokens padding
        _route("route_step_597x4of60_1031", "step", 597, 4, 60, 1031, keep=0.8),
        # a pre-training step over many experts
        _route("route_step_8192x8of128_2048", "step", 8192, 8, 128, 2048),
        # one decoded token: two of eight large experts' weights are read
        _experts("experts_forward_1x2of8_11008x4096", "forward", 1, 2, 8, 11008, 4096),
        # a decode batch over many small experts, up projection fused in
        _experts("experts_gated_64x8of64_1024x2048", "gated", 64, 8, 64, 1024, 2048),
        # a prompt through few large experts, some padding
        _experts("experts_forward_4095x2of8_11008x4096", "forward", 4095, 2, 8, 11008, 4096, keep=0.9),
        # a training step over many small experts, 256 rows each
        _experts("experts_step_2048x4of32_1024x2048", "step", 2048, 4, 32, 1024, 2048),
        # one decoded token of a request with an adapter
        _adapters("adapters_1x11008x4096_r16", 1, 11008, 4096, 16, 4, 1),
        # a decode batch, requests of sixteen adapters and some of none
        _adapters("adapters_48x11008x4096_r16", 48, 11008, 4096, 16, 64, 16, keep=0.9),
        # a prefill of a few requests
        _adapters("adapters_597x11008x4096_r32", 597, 11008, 4096, 32, 16, 4),
        # a large prefill of many requests with wider adapters
        _adapters("adapters_4095x4096x4096_r64", 4095, 4096, 4096, 64, 32, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["route", "experts", "experts", "adapters"])
        T = _log(rng, 1, 8192)
        keep = rng.choice([1.0, round(rng.uniform(0.2, 1.0), 2)])
        if op == "route":
            E = _log(rng, 4, 256)
            k = min(E, rng.randint(1, 8))
            D = _log(rng, 128, 8192) if rng.random() < 0.3 else 8 * _log(rng, 16, 1024)
            if T * k * D <= 8192 * 8 * 2048:
                return {"op": op, "pass": rng.choice(["forward", "step"]), "T": T, "k": k, "E": E,
                        "D": D, "keep": keep}
        elif op == "experts":
            E = _log(rng, 4, 128)
            k = min(E, rng.randint(1, 8))
            N, K = 8 * _log(rng, 32, 1376), 8 * _log(rng, 32, 1024)
            kind = rng.choice(["forward", "gated", "step"])
            if T * k * N * K * (3 if kind == "step" else 1) <= 4095 * 2 * 11008 * 4096 and \
                    E * N * K <= 8 * 11008 * 4096:
                return {"op": op, "pass": kind, "T": T, "k": k, "E": E, "N": N, "K": K, "keep": keep}
        else:
            E = _log(rng, 1, 128)
            N, K = 8 * _log(rng, 64, 1376), 8 * _log(rng, 64, 1024)
            used = rng.randint(1, max(1, min(E, T, 32)))
            R = rng.choice([8, 16, 16, 32, 64, 128])
            if T * N * K <= 4095 * 2 * 11008 * 4096 and used * R <= 1024:
                return {"op": op, "pass": "forward", "T": T, "k": 1, "E": E, "N": N, "K": K, "R": R,
                        "used": used, "keep": keep}


def _tokens(case):
    """Tokens that take part."""
    return max(1, int(round(case["T"] * case["keep"])))


def _sorted_slots(ids, E):
    """Slots in the order of their group, those of none last; and per group."""
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < E)
    order = torch.sort(torch.where(valid, flat, E), stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=flat.device)
    place = torch.where(valid, position, -1).reshape(ids.shape)
    return offsets.int(), order.int(), place.int()


def prepare(case, seed):
    T, k, E = case["T"], case["k"], case["E"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    out_rows = torch.argsort(torch.rand(T, generator=g, device="cuda"))[_tokens(case):]
    state = {"case": case}
    if case["op"] == "adapters":
        # requests of some of the loaded adapters: runs of tokens for a prompt,
        # a token each in a decode batch
        N, K, R, used = case["N"], case["K"], case["R"], case["used"]
        loaded = torch.randperm(E, generator=g, device="cuda")[:used]
        cut = torch.sort(torch.rand(T, generator=g, device="cuda")).values
        ids = loaded[(cut * used).long().clamp_(max=used - 1)]
        if T <= 64:
            ids = ids[torch.randperm(T, generator=g, device="cuda")]
        ids = ids[:, None].clone()
        ids[out_rows] = -1
        state["X"] = randn(T, K).bfloat16()
        state["W"] = (randn(N, K) / math.sqrt(K)).bfloat16()
        state["A"] = (randn(E, R, K) / math.sqrt(K)).bfloat16()
        state["B"] = (randn(E, N, R) * 0.1).bfloat16()
        state["scale"] = 0.5 + torch.rand(E, generator=g, device="cuda")
        state["ids"] = ids
        # a serving program sorts a batch once for all its layers
        state["offsets"], state["order"], _ = _sorted_slots(ids, E)
        if own:
            import dense_gemm_linear_amd as dg
            state["workspace"] = torch.empty(dg.linear_adapters_workspace_bytes(T, R, E),
                                             dtype=torch.uint8, device="cuda")
        return state
    # a router's choices: distinct experts, some more popular than others
    top = torch.topk(randn(T, E) + 0.5 * randn(E), k, dim=1)
    ids = top.indices.clone()
    ids[out_rows] = -1
    S = T * k
    state["ids"] = ids
    if case["op"] == "route":
        D = case["D"]
        state["weights"] = torch.softmax(top.values, dim=1)
        state["X"] = randn(T, D).bfloat16()
        state["Y"] = randn(S, D).bfloat16()              # the experts' outputs, sorted
        # buffers that a program keeps; rows behind the last slot stay as they are
        state["Xs"] = torch.zeros(S, D, dtype=torch.bfloat16, device="cuda")
        if case["pass"] == "step":
            state["dout"] = randn(T, D).bfloat16()
            state["dXs"] = randn(S, D).bfloat16()
            state["dY"] = torch.zeros(S, D, dtype=torch.bfloat16, device="cuda")
        if own:
            import dense_gemm_linear_amd as dg
            state["workspace"] = torch.empty(dg.group_sort_workspace_bytes(T, k, E), dtype=torch.uint8,
                                             device="cuda")
        return state
    N, K = case["N"], case["K"]
    # the layer's rows were sorted by its router
    state["offsets"], state["order"], _ = _sorted_slots(ids, E)
    state["X"] = randn(T, K).bfloat16()
    state["W"] = (randn(E, N, K) / math.sqrt(K)).bfloat16()
    state["Y"] = torch.zeros(S, N, dtype=torch.bfloat16, device="cuda")
    if case["pass"] == "gated":
        state["mul"] = randn(S, N).bfloat16()
    if case["pass"] == "step":
        state["dY"] = randn(S, N).bfloat16()
        state["dX"] = torch.zeros(S, K, dtype=torch.bfloat16, device="cuda")
        if own:
            import dense_gemm_linear_amd as dg
            state["workspace"] = torch.empty(dg.group_linear_grad_workspace_bytes(T, k, K),
                                             dtype=torch.uint8, device="cuda")
    return state


def _run_own(s):
    import dense_gemm_linear_amd as dg
    c = s["case"]
    if c["op"] == "adapters":
        return dg.linear_adapters(s["X"], s["W"], s["A"], s["B"], s["offsets"], s["order"],
                                  scale=s["scale"], workspace=s["workspace"])
    if c["op"] == "route":
        offsets, order, place = dg.group_sort(s["ids"], c["E"], workspace=s["workspace"])
        Xs = dg.group_gather(s["X"], place, out=s["Xs"])
        out = dg.group_combine(s["Y"], place, s["weights"])
        if c["pass"] == "forward":
            return offsets, order, place, Xs, out
        dX = dg.group_combine(s["dXs"], place)
        dY, dweights = dg.group_combine_grad(s["dout"], s["Y"], place, s["weights"], dY=s["dY"])
        return offsets, order, place, Xs, out, dX, dY, dweights
    if c["pass"] == "gated":
        return dg.group_linear(s["X"], s["W"], s["offsets"], s["order"], slots=c["k"],
                               activation="silu", mul=s["mul"], out=s["Y"])
    Y = dg.group_linear(s["X"], s["W"], s["offsets"], s["order"], slots=c["k"], out=s["Y"])
    if c["pass"] == "forward":
        return Y
    dX, dW = dg.group_linear_grad(s["dY"], s["X"], s["W"], s["offsets"], s["order"], slots=c["k"],
                                  dX=s["dX"], workspace=s["workspace"])
    return Y, dX, dW


def _plain_route(s):
    c = s["case"]
    T, k, D = c["T"], c["k"], c["D"]
    offsets, order, place = _sorted_slots(s["ids"], c["E"])
    valid = (place >= 0).reshape(-1)
    token = order.long() // k
    live = valid[order.long()][:, None]
    at = place.reshape(-1).clamp(min=0).long()
    w = (s["weights"] * (place >= 0)).reshape(-1, 1)

    def joined(rows, weight):
        picked = torch.where(valid[:, None], rows[at].float(), 0.0)
        return (picked * weight).reshape(T, k, D).sum(1).bfloat16()

    out = (offsets, order, place, s["X"][token] * live, joined(s["Y"], w))
    if c["pass"] == "forward":
        return out
    dout = s["dout"].float()
    dY = torch.where(live, dout[token] * w[order.long()], 0.0).bfloat16()
    picked = torch.where(valid[:, None], s["Y"][at].float(), 0.0).reshape(T, k, D)
    return out + (joined(s["dXs"], 1.0), dY, (picked * dout[:, None, :]).sum(2))


def _plain_experts(s):
    # every expert in use gets as many rows as the busiest one, zeros behind its
    # own, and one batched product serves them all
    c = s["case"]
    K, N, E, S = c["K"], c["N"], c["E"], c["T"] * c["k"]
    counts = s["offsets"][1:] - s["offsets"][:-1]
    used = torch.nonzero(counts).squeeze(1)
    most = int(counts.max())
    position = s["offsets"][used][:, None] + torch.arange(most, device="cuda")
    live = position < s["offsets"][used + 1][:, None]
    position = torch.where(live, position, 0).long()
    X = s["X"].float()[s["order"].long() // c["k"]]
    Xp = X[position] * live[:, :, None]
    W = s["W"][used].float()
    y = torch.bmm(Xp, W.transpose(1, 2))[live]
    n = y.shape[0]

    def whole(rows, width):
        full = torch.zeros(S, width, dtype=torch.bfloat16, device="cuda")
        full[:n] = rows.bfloat16()
        return full

    if c["pass"] == "gated":
        y = y / (1.0 + torch.exp(-y)) * s["mul"][:n].float()
    out = whole(y, N)
    if c["pass"] != "step":
        return out
    dYp = s["dY"].float()[position] * live[:, :, None]
    dX = whole(torch.bmm(dYp, W)[live], K)
    dW = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    dW[used] = torch.bmm(dYp.transpose(1, 2), Xp).bfloat16()
    return out, dX, dW


def _plain_adapters(s):
    # the adapters in use side by side: every row's inner values for all of
    # them, with zeros where the adapter is not the row's own
    c = s["case"]
    used = torch.nonzero(s["offsets"][1:] - s["offsets"][:-1]).squeeze(1)
    X = s["X"].float()
    A = s["A"][used].float().reshape(-1, c["K"])
    B = s["B"][used].float().permute(0, 2, 1).reshape(-1, c["N"])
    factor = torch.where(s["ids"] == used, s["scale"][used], 0.0)
    inner = torch.matmul(X, A.t()) * factor.repeat_interleave(c["R"], dim=1)
    return (torch.matmul(X, s["W"].float().t()) + torch.matmul(inner, B)).bfloat16()


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "experts": _plain_experts,
            "adapters": _plain_adapters}[state["case"]["op"]](state)


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    S, n = T * k, _tokens(case) * k
    if case["op"] == "route":
        D = case["D"]
        row = 2 * D
        nbytes = 8 * S + 4 * (2 * S + E + 1) + row * (T + n) + 4 * S + row * (n + T)
        flops = 2 * n * D
        if case["pass"] == "step":
            nbytes += row * (n + T) + row * (T + n + n) + 4 * S
            flops += 4 * n * D
        return {"bytes": nbytes, "flops": flops}
    N, K = case["N"], case["K"]
    if case["op"] == "adapters":
        R, used = case["R"], case["used"]
        return {"bytes": 2 * (T * K + N * K + used * R * (K + N) + T * N) + 4 * (T + E + 1),
                "flops": 2 * T * N * K + 2 * n * R * (K + N)}
    # experts that some token chose, of uniform choices
    in_use = E * (1.0 - (1.0 - k / E) ** _tokens(case))
    nbytes = 2 * (_tokens(case) * K + in_use * N * K + n * N) + 4 * (S + E + 1)
    flops = 2 * n * N * K
    if case["pass"] == "gated":
        nbytes += 2 * n * N
    if case["pass"] == "step":
        nbytes += 2 * (n * N + n * K + E * N * K)
        flops *= 3
    return {"bytes": int(nbytes), "flops": flops}


def exact(case, seed):
    """The same values from the definitions in 64 bits, one group at a time."""
    s = prepare(case, seed)
    T, k, E = case["T"], case["k"], case["E"]
    S = T * k
    ids = s["ids"].reshape(-1)
    slots = [torch.nonzero(ids == e).squeeze(1) for e in range(E)]

    def f64(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if case["op"] == "adapters":
        Y = s["X"].double() @ s["W"].double().t()
        for e, rows in enumerate(slots):
            if rows.numel():
                inner = s["X"][rows].double() @ s["A"][e].double().t()
                Y[rows] += s["scale"][e].double() * (inner @ s["B"][e].double().t())
        return Y
    if case["op"] == "experts":
        N, K = case["N"], case["K"]
        Y = f64(S, N)
        step = case["pass"] == "step"
        dX, dW = (f64(S, K), f64(E, N, K)) if step else (None, None)
        at = 0
        for e, rows in enumerate(slots):
            m = rows.numel()
            if not m:
                continue
            X, W = s["X"][rows // k].double(), s["W"][e].double()
            y = X @ W.t()
            if case["pass"] == "gated":
                y = y * torch.sigmoid(y) * s["mul"][at:at + m].double()
            Y[at:at + m] = y
            if step:
                d = s["dY"][at:at + m].double()
                dX[at:at + m] = d @ W
                dW[e] = d.t() @ X
            at += m
        return (Y, dX, dW) if step else Y
    D = case["D"]
    order = torch.cat(slots + [torch.nonzero(ids < 0).squeeze(1)])
    offsets = torch.tensor([0] + [r.numel() for r in slots], device="cuda").cumsum(0)
    n = int(offsets[-1])
    token = order[:n] // k
    place = torch.full((S,), -1, dtype=torch.int64, device="cuda")
    place[order[:n]] = torch.arange(n, device="cuda")
    Xs = f64(S, D)
    Xs[:n] = s["X"][token].double()
    w = s["weights"].reshape(-1)[order[:n]].double()
    out = f64(T, D).index_add_(0, token, s["Y"][:n].double() * w[:, None])
    got = [offsets.int(), order.int(), place.reshape(T, k).int(), Xs, out]
    if case["pass"] == "step":
        dout = s["dout"].double()[token]
        dY = f64(S, D)
        dY[:n] = dout * w[:, None]
        dweights = f64(S)
        dweights[order[:n]] = (dout * s["Y"][:n].double()).sum(1)
        got += [f64(T, D).index_add_(0, token, s["dXs"][:n].double()), dY, dweights.reshape(T, k)]
    return tuple(got)
