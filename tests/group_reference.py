"""The grouped rows' operators from their definitions, in 64 bits on the CPU, and
the error bounds their results are held to.

A product of K bf16 factors summed in fp32, in any order and with any grouping, is
off by at most K u S with S = sum |a b| and u = 2^-23 (a sum rounded to nearest is
off by half of that; the matrix cores' sums are taken to be as coarse as a
truncating one).  Rounding v to bf16 adds 2^-8 |v| at most."""
import torch

U32, UBF = 2.0 ** -23, 2.0 ** -8


def sorted_slots(ids, groups):
    """(offsets, order, place) as Python integers would sort them."""
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(groups + 1)]
    for s, g in enumerate(flat):
        lists[g if 0 <= g < groups else groups].append(s)
    order, offsets, place = [], [0], [-1] * len(flat)
    for g, slots in enumerate(lists):
        if g < groups:
            for i, s in enumerate(slots):
                place[s] = len(order) + i
        order += slots
        if g < groups:
            offsets.append(len(order))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(order, dtype=torch.int32),
            torch.tensor(place, dtype=torch.int32).reshape(ids.shape))


def make_ids(T, k, groups, seed, none=0.1, kind="random"):
    """kind "distinct": a router's (no group twice in a token), "random": any,
    "one": all in one group, "runs": few groups in long runs."""
    g = torch.Generator().manual_seed(seed)
    if kind == "distinct":
        ids = torch.topk(torch.rand(T, groups, generator=g) + torch.rand(groups, generator=g), k, dim=1).indices
    elif kind == "one":
        ids = torch.full((T, k), groups // 2)
    elif kind == "runs":
        ids = (torch.arange(T)[:, None] * 3 // max(T, 1) * 7 % groups).expand(T, k).clone()
    else:
        ids = torch.randint(0, groups, (T, k), generator=g)
    out = torch.rand(T, k, generator=g) < none
    # padding below 0 and ids past the last group
    return torch.where(out, torch.where(torch.rand(T, k, generator=g) < 0.5, -1, groups + 3), ids)


def bf16(*shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def close(got, want, err, what):
    """Elementwise |got - want| <= err; NaN only where the reference has it."""
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= err)
    bad &= ~(torch.isnan(got) & torch.isnan(want)) & ~((got == want) & torch.isinf(want))
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{float(got[i])} for {float(want[i])}, allowed {float(err[i])}")


def product(A, B):
    """A B^T in 64 bits and the bound of its fp32 form, rounded to bf16."""
    A, B = A.double(), B.double()
    v = A @ B.t()
    return v, UBF * v.abs() + (A.shape[1] + 2) * U32 * (A.abs() @ B.abs().t())


def activation(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * (1 + torch.erf(v / 2 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
    return v
