"""The linear head's losses from their definitions in 64 bits (torch on any
device, elementary operations), and the error bounds the GPU tests hold the
kernels to.

Bounds, from the formats (u = 2^-24 one fp32 rounding, h = 2^-8 one bf16
rounding, both relative to the value):
  z      products of bf16 are exact in fp32; a sum of D of them in any order
         and the scale: ez = (D + 3) u |scale| sum_d |x w|
  lse    the largest ez of the row; the sum over V columns is made of at most
         4 + 4 (a row of a wave), 4 (waves), V / 2048 + 16 (tiles) additions
         and rescalings, each with an exponential of argument error
         2 u |z - max|: (64 + V / 2048 + 4 range) u, and 4 u |lse| to store it
  nll    the same through softplus, whose slope is at most 1, plus 4 u |nll|
  dz     p = exp(z - lse): relative ez + elze + (8 + 4 range) u, then
         one bf16 rounding: h |dz|; at a target column the difference p - q
         carries the errors of both sides
  dX     sum over V of dz W: the errors of dz, (V + 64) u sum |dz W|, and one
         rounding h |dX|; dW the same over T
These add worst cases, loose for long sums, so the Frobenius norm of the error
is held too: roundings of dz are independent, at most h each, so their
contribution to one element of dX has a root mean square of at most h
sqrt(sum (dz W)^2); twice that, plus the worst case of the rest.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
H = 2.0 ** -8


def problem(T, V, D, seed, pull=4.0, spread=2.0, device="cuda"):
    """X, W bf16 and one lead column a row that X leans to."""
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, D, generator=g) * (spread / math.sqrt(D))).bfloat16()
    lead = torch.randint(0, V, (T,), generator=g)
    X = torch.randn(T, D, generator=g) + pull * torch.rand(T, 1, generator=g) * W[lead].float()
    return X.bfloat16().to(device), W.to(device), lead.to(device)


def _targets(labels, index, teacher, scale, V, ignore_index, T, device):
    """(rows kept, list of (row, column) weights as a dense-by-slot pair idx, q, log q)."""
    if labels is not None:
        keep = labels != ignore_index
        idx = labels.clamp(min=0)[:, None]
        q = torch.ones(T, 1, dtype=torch.float64, device=device)
        return keep, idx, q, torch.zeros_like(q), torch.ones_like(idx, dtype=torch.bool)
    filled = (index >= 0) & (teacher != -math.inf)
    t = torch.where(filled, teacher.double() * scale, -math.inf)
    keep = filled.any(dim=1)
    t = t - torch.where(keep, t.max(dim=1).values, 0.0)[:, None]
    e = torch.where(filled, t.exp(), 0.0)
    s = torch.where(keep, e.sum(dim=1), 1.0)[:, None]
    return keep, index.clamp(min=0), e / s, torch.where(filled, t - s.log(), 0.0), filled


def reference(X, W, *, labels=None, index=None, teacher=None, dloss=None, scale=1.0, z_loss=0.0,
              ignore_index=-100):
    """A dict of the outputs in 64 bits and of bounds on a kernel's errors
    (key + "_tol" elementwise, key + "_fro" on the Frobenius norm)."""
    T, D = X.shape
    V = W.shape[0]
    dev = X.device
    keep, idx, q, log_q, filled = _targets(labels, index, teacher, scale, V, ignore_index, T, dev)
    rows = torch.nonzero(keep).squeeze(1)
    Xk, Wd = X[rows].double(), W.double()
    idx, q, log_q, filled = idx[rows], q[rows], log_q[rows], filled[rows]
    z = scale * (Xk @ Wd.t())
    ez = (D + 3) * U * abs(scale) * (Xk.abs() @ Wd.abs().t())
    lse = torch.logsumexp(z, dim=1)
    top = z.max(dim=1).values
    rng = (top - z.min(dim=1).values).clamp(max=100.0) if V > 0 else top
    e_lse = ez.max(dim=1).values + (64 + V / 2048 + 4 * rng) * U + 4 * U * lse.abs()
    logp = torch.where(filled, z.gather(1, idx) - lse[:, None], 0.0)
    # the lead's -log p from the other columns, as the definition allows
    e_logp = e_lse + ez.max(dim=1).values
    e_logp = e_logp[:, None] + 4 * U * logp.abs()
    out = {}

    def put(name, val, tol):
        full = torch.zeros((T,) + val.shape[1:], dtype=torch.float64, device=dev)
        bound = torch.zeros_like(full)
        full[rows], bound[rows] = val, tol
        out[name], out[name + "_tol"] = full, bound

    if labels is not None:
        nll = -logp[:, 0]
        loss = nll + z_loss * lse * lse
        tol = e_logp[:, 0] + abs(z_loss) * (2 * lse.abs() * e_lse + 8 * U * lse * lse) + 2 * U * loss.abs()
    else:
        loss = (q * (log_q - logp)).sum(dim=1)
        t = teacher[rows].double() * scale
        t = torch.where(filled, t, 0.0)
        trange = (t.max(dim=1).values - t.min(dim=1).values)[:, None]
        e_q = (32 + idx.shape[1] / 64 + 4 * trange + 2 * t.abs().max(dim=1).values[:, None]) * U
        tol = (q * e_logp).sum(dim=1) + (q * ((1 + (log_q - logp).abs()) * e_q
                                              + 2 * U * (log_q.abs() + logp.abs()))).sum(dim=1) \
            + (idx.shape[1] + 8) * U * (q * (log_q - logp).abs()).sum(dim=1)
        put("logp", logp, torch.where(filled, e_logp, 0.0))
    put("loss", loss, tol)
    put("lse", lse, e_lse)
    if dloss is None:
        return out
    w = (scale * dloss.double().expand(T))[rows]
    gain = 1.0 + 2.0 * z_loss * lse
    p = torch.exp(z - lse[:, None])
    e_p = p * (ez + (e_lse + (8 + 4 * rng) * U)[:, None])
    dz = p * gain[:, None]
    e_dz = e_p * gain.abs()[:, None] + 8 * U * dz.abs()
    dz = dz.scatter_add(1, idx, torch.where(filled, -q, 0.0))
    if labels is None:
        e_dz = e_dz.scatter_add(1, idx, torch.where(filled, q * e_q, 0.0))
    e_dz = e_dz.scatter_add(1, idx, torch.where(filled, p.gather(1, idx) * e_logp + 8 * U * (q + p.gather(1, idx)) * (idx.shape[1] > 1), 0.0))
    dz, e_dz = dz * w[:, None], e_dz * w.abs()[:, None]
    for name, a, e, b, n in (("dX", dz, e_dz, Wd, V), ("dW", dz.t(), e_dz.t(), Xk, len(rows))):
        g = a @ b
        mag = a.abs() @ b.abs()
        rest = e @ b.abs() + (n + 64) * U * mag
        tol = rest + H * mag * (1 + H) + H * (g.abs() + H * mag)
        fro = 2 * H * math.sqrt(float(((a * a) @ (b * b)).sum()) + float((g * g).sum())) \
            + float(rest.norm())
        if name == "dX":
            put("dX", g, tol)
        else:
            out["dW"], out["dW_tol"] = g, tol
        out[name + "_fro"] = fro
    return out


def check(got: dict, ref: dict, what: str):
    for name, val in got.items():
        if val is None:
            continue
        want, tol = ref[name], ref[name + "_tol"]
        v = val.double()
        assert v.shape == want.shape, f"{what}: {name} has shape {tuple(v.shape)}"
        assert bool(torch.isfinite(v).all()), f"{what}: {name} is not finite"
        err = (v - want).abs()
        # results below bf16's and fp32's normal range may flush
        over = err > tol + 1e-37
        assert not bool(over.any()), (
            f"{what}: {name} off at {int(over.sum())} of {over.numel()}: worst error "
            f"{float((err - tol).max()):.3e} over its bound, first at "
            f"{tuple(int(i) for i in torch.nonzero(over)[0])}")
        if name + "_fro" in ref:
            assert float(err.norm()) <= ref[name + "_fro"] + 1e-30, (
                f"{what}: {name} error norm {float(err.norm()):.3e}, bound {ref[name + '_fro']:.3e}")
