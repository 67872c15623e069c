"""What is measured of the linear head's losses, and what they are held against.

A linear head has logits z = scale * X W^T over a vocabulary of V columns, X
[T, D] the hidden rows and W [V, D] the weight, both bf16.  Two losses are
taken from it without keeping z in memory:

  "ce"       softmax cross entropy with one label a row:
             loss = lse - z[y] + z_loss * lse^2, lse = log sum_v exp z[v]
  "distill"  the divergence of the softmax over z from a teacher's
             distribution over its k top columns: q = softmax(scale * teacher),
             loss = sum_j q_j (log q_j - logp_j), logp_j = z[index_j] - lse

A "forward" pass gives the losses, as evaluation and scoring do; a "step"
gives the losses and the gradients of X and W for given loss weights; a
"step_dx" leaves W's gradient out (a frozen head).  Rows whose label is
IGNORE (prompt and padding tokens) are out: loss, lse and gradient are 0.
"""
import math

import torch

own = False

IGNORE = -100


def _case(name, op, kind, T, V, D, k=0, keep=1.0, scale=1.0, z_loss=0.0):
    return {"name": name, "op": op, "pass": kind, "T": T, "V": V, "D": D, "k": k, "keep": keep,
            "scale": scale, "z_loss": z_loss}


def listed():
    return [
        # scoring one token of a small model's head: a weight read and latency
        _case("ce_score_1x50257x512", "ce", "forward", 1, 50257, 512),
        # scoring a decode batch with a wide head: the weight read bounds it
        _case("ce_score_48x50257x4096", "ce", "forward", 48, 50257, 4096),
        # perplexity of a 1024-token window through a GPT-2-sized head
        _case("ce_eval_1024x50257x512", "ce", "forward", 1024, 50257, 512),
        # perplexity of a long window, one token short of a power of two
        _case("ce_eval_4095x50257x4096", "ce", "forward", 4095, 50257, 4096),
        # a small fine-tuning step, half of the rows prompt tokens
        _case("ce_step_528x11007x1024", "ce", "step", 528, 11007, 1024, keep=0.5),
        # a training step of the GPT-2-sized head
        _case("ce_step_1024x50257x512", "ce", "step", 1024, 50257, 512),
        # a pre-training step of a wide head with the log-partition penalty,
        # some padding at the sequences' ends
        _case("ce_step_4096x50257x4096", "ce", "step", 4096, 50257, 4096, keep=0.9, z_loss=1e-4),
        # adapter tuning: the head is frozen, only the hidden rows' gradient
        _case("ce_step_dx_597x50257x4096", "ce", "step_dx", 597, 50257, 4096),
        # validation of a distilled model on a handful of tokens
        _case("distill_eval_8x50257x1024", "distill", "forward", 8, 50257, 1024, k=16),
        # validation over a window
        _case("distill_eval_2048x50257x2048", "distill", "forward", 2048, 50257, 2048, k=32),
        # a small distillation step at temperature 2
        _case("distill_step_500x11008x1024", "distill", "step", 500, 11008, 1024, k=9, keep=0.8,
              scale=0.5),
        # a distillation step over a large vocabulary
        _case("distill_step_2048x131072x4096", "distill", "step", 2048, 131072, 4096, k=64),
    ]


def _products(kind):
    # forward: the logits; gradient: the logits again (they are not kept) and
    # one product for each gradient
    return {"forward": 1, "step_dx": 3, "step": 4}[kind]


def draw(rng):
    limit = 2.0 * 4 * 2048 * 131072 * 4096
    while True:
        op = rng.choice(["ce", "distill"])
        kind = rng.choice(["forward", "step", "step", "step_dx"])
        T = int(round(math.exp(rng.uniform(0.0, math.log(8192)))))
        V = int(round(math.exp(rng.uniform(math.log(4000), math.log(131072)))))
        D = 8 * int(round(math.exp(rng.uniform(math.log(16), math.log(512)))))
        k = int(round(math.exp(rng.uniform(0.0, math.log(128))))) if op == "distill" else 0
        keep = rng.choice([1.0, round(rng.uniform(0.1, 1.0), 2)])
        scale = rng.choice([1.0, round(rng.uniform(0.25, 1.5), 3)])
        z_loss = rng.choice([0.0, 1e-4]) if op == "ce" else 0.0
        if 2.0 * _products(kind) * T * V * D <= limit:
            return {"op": op, "pass": kind, "T": T, "V": V, "D": D, "k": k, "keep": keep,
                    "scale": scale, "z_loss": z_loss}


def _kept(case):
    return max(1, int(round(case["T"] * case["keep"])))


def prepare(case, seed):
    T, V, D, k = case["T"], case["V"], case["D"], case["k"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # normalised hidden rows; weights that give logits a spread of 2; every row
    # leans towards its target, so the target's probability runs from nearly 0
    # to nearly 1
    W = (randn(V, D) * (2.0 / math.sqrt(D))).bfloat16()
    n = _kept(case)
    out_rows = torch.argsort(rand(T))[n:]                 # the rows that are out
    state = {"case": case}
    if case["op"] == "ce":
        # token ids in order of frequency: small ones are common
        labels = (rand(T) ** 3 * V).long().clamp_(max=V - 1)
        lead = labels.clone()
        labels[out_rows] = IGNORE
        state["labels"] = labels
    else:
        # the teacher's top k of its own logits, again with common small ids
        common = -1.5 * torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32))
        index, teacher = [], []
        for t0 in range(0, T, 512):
            rows = min(512, T - t0)
            top = torch.topk(2.5 * randn(rows, V) + common, k, dim=1)
            index.append(top.indices)
            teacher.append(top.values)
        index, teacher = torch.cat(index), torch.cat(teacher)
        lead = index[:, 0].clone()
        index[out_rows] = -1                              # rows with no slot filled
        state["index"], state["teacher"] = index, teacher.contiguous()
    pull = 4.0 * rand(T, 1)
    state["X"] = (randn(T, D) + pull * W[lead].float()).bfloat16()
    state["W"] = W
    # a mean over the kept rows, some of them weighted
    state["dloss"] = (0.5 + rand(T)) / n
    if own:
        import dense_gemm_linear_amd as dg
        nbytes = dg.linear_loss_workspace_bytes(T, V, D, k, backward=case["pass"] != "forward")
        state["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return state


def _run_own(s):
    import dense_gemm_linear_amd as dg
    c = s["case"]
    step, need_dW = c["pass"] != "forward", c["pass"] == "step"
    if c["op"] == "ce":
        kw = dict(scale=c["scale"], z_loss=c["z_loss"], ignore_index=IGNORE,
                  workspace=s["workspace"])
        loss, lse = dg.linear_cross_entropy(s["X"], s["W"], s["labels"], **kw)
        if not step:
            return loss, lse
        dX, dW = dg.linear_cross_entropy_grad(s["X"], s["W"], s["labels"], loss, lse,
                                              s["dloss"], need_dW=need_dW, **kw)
        return (loss, lse, dX, dW) if need_dW else (loss, lse, dX)
    kw = dict(scale=c["scale"], workspace=s["workspace"])
    loss, lse, logp = dg.linear_distillation(s["X"], s["W"], s["index"], s["teacher"], **kw)
    if not step:
        return loss, lse, logp
    dX, dW = dg.linear_distillation_grad(s["X"], s["W"], s["index"], s["teacher"], lse, logp,
                                         s["dloss"], need_dW=need_dW, **kw)
    return (loss, lse, logp, dX, dW) if need_dW else (loss, lse, logp, dX)


def _run_plain(s):
    c = s["case"]
    X, W = s["X"].float(), s["W"].float()
    z = torch.matmul(X, W.t()) * c["scale"]
    if c["op"] == "ce":
        keep = s["labels"] != IGNORE
        lead = s["labels"].clamp(min=0)[:, None]
    else:
        filled = s["index"] >= 0
        keep = filled.any(dim=1)
        at = s["index"].clamp(min=0)
        t = (s["teacher"].float() * c["scale"]).masked_fill(~filled, -math.inf)
        top_t, slot = t.max(dim=1, keepdim=True)
        t = t - torch.where(keep[:, None], top_t, 0.0)
        qe = torch.exp(t)
        qsum = torch.where(keep, qe.sum(dim=1), 1.0)[:, None]
        q = qe / qsum
        log_q = torch.where(filled, t - torch.log(qsum), 0.0)
        lead = at.gather(1, slot)
    # the log-sum-exp over the other columns than the row's leading target: the
    # target's log-probability is then exact for a probability near 1 too
    z_lead = z.gather(1, lead)
    others = z.scatter(1, lead, -math.inf)
    top = others.max(dim=1, keepdim=True).values
    e = torch.exp(others - top)
    lse_others = top + torch.log(e.sum(dim=1, keepdim=True))
    d = lse_others - z_lead
    nll = torch.clamp(d, min=0.0) + torch.log1p(torch.exp(-d.abs()))
    lse = z_lead + nll
    nll, lse = nll.squeeze(1), lse.squeeze(1)
    if c["op"] == "ce":
        loss = nll + c["z_loss"] * lse * lse
        out = (loss * keep, lse * keep)
    else:
        logp = (z.gather(1, at) - z_lead - nll[:, None]) * filled
        loss = (q * (log_q - logp)).sum(dim=1)
        out = (loss * keep, lse * keep, logp)
    if c["pass"] == "forward":
        return out
    p = torch.exp(z - lse[:, None])
    p_others = torch.exp(lse_others.squeeze(1) - lse)
    if c["op"] == "ce":
        extra = 2.0 * c["z_loss"] * lse
        dz = p * (1.0 + extra)[:, None]
        dz.scatter_(1, lead, (extra * torch.exp(-nll) - p_others)[:, None])
    else:
        dz = p.scatter_add(1, at, -q)
        q_others = q.scatter(1, slot, 0.0).sum(dim=1)
        dz.scatter_(1, lead, (q_others - p_others)[:, None])
    dz = dz * (s["dloss"] * keep * c["scale"])[:, None]
    out = out + (torch.matmul(dz, W).bfloat16(),)
    if c["pass"] == "step":
        out = out + (torch.matmul(dz.t(), X).bfloat16(),)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    T, V, D, k = case["T"], case["V"], case["D"], case["k"]
    n = _kept(case)
    targets = 8 * T if case["op"] == "ce" else 12 * T * k
    nbytes = 2 * n * D + 2 * V * D + targets + 8 * T + (4 * T * k)
    if case["pass"] != "forward":
        nbytes += 4 * T + 2 * T * D
    if case["pass"] == "step":
        nbytes += 2 * V * D
    return {"bytes": nbytes, "flops": 2 * _products(case["pass"]) * n * V * D}


def exact(case, seed):
    """The same values from the definitions in 64 bits, kept rows only, the
    vocabulary in one piece."""
    s = prepare(case, seed)
    T, V, k = case["T"], case["V"], case["k"]
    sc = float(case["scale"])
    ce = case["op"] == "ce"
    rows = torch.nonzero(s["labels"] != IGNORE if ce else (s["index"] >= 0).any(1)).squeeze(1)
    X, W = s["X"][rows].double(), s["W"].double()
    logits = sc * (X @ W.t())
    lse = torch.logsumexp(logits, dim=1)
    n = rows.numel()
    r = torch.arange(n, device="cuda")
    if ce:
        y = s["labels"][rows]
        loss = lse - logits[r, y] + case["z_loss"] * lse.square()
        logp = None
        gain = 1.0 + 2.0 * case["z_loss"] * lse
    else:
        idx = s["index"][rows]
        log_q = torch.log_softmax(sc * s["teacher"][rows].double(), dim=1)
        logp = logits.gather(1, idx) - lse[:, None]
        loss = torch.sum(log_q.exp() * (log_q - logp), dim=1)
        gain = torch.ones_like(lse)

    def spread(v):
        full = torch.zeros((T,) + v.shape[1:], dtype=torch.float64, device="cuda")
        full[rows] = v
        return full

    out = [spread(loss), spread(lse)] + ([] if ce else [spread(logp)])
    if case["pass"] != "forward":
        grad = torch.exp(logits - lse[:, None]).mul_(gain[:, None])
        del logits
        if ce:
            grad[r, y] -= 1.0
        else:
            for j in range(k):
                grad[r, idx[:, j]] -= log_q[:, j].exp()
        grad.mul_((sc * s["dloss"][rows].double())[:, None])
        out.append(spread(grad @ W))
        if case["pass"] == "step":
            out.append(grad.t() @ X)
    return tuple(out)
