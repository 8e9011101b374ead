"""Plain forms of the order by expert, of the rows between tokens and experts and of the 8-bit operands, for the tests: loops and
64 bits, apart from the library's code."""
import torch


def order(ids, E):
    """offsets [E + 1] and inv [T, k] of ids (a nested list), pair by pair."""
    pairs = sorted((e, t, j) for t, row in enumerate(ids) for j, e in enumerate(row) if 0 <= e < E)
    offsets = [sum(p[0] < e for p in pairs) for e in range(E + 1)]
    inv = [[-1] * len(row) for row in ids]
    for r, (_, t, j) in enumerate(pairs):
        inv[t][j] = r
    return offsets, inv


def some_ids(T, k, E, seed, kind="distinct"):
    """int32 [T, k] on the CPU: k different experts a token; or any, the same one twice among them; or with pairs that have none."""
    g = torch.Generator().manual_seed(seed)
    if kind == "distinct":
        return torch.rand(T, E, generator=g).argsort(1)[:, :k].sort(1).values.int()
    ids = torch.randint(0, max(1, E // 2), (T, k), generator=g, dtype=torch.int32)
    if kind == "dropped":
        drop = torch.rand(T, k, generator=g) < 0.3
        ids[drop] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.randint(0, 4, (int(drop.sum()),), generator=g)]
    return ids


def numbers(x):
    """Whole numbers and scales of the rows of x, in 64 bits (a quotient of fp32 numbers rounded to 64 and then to fp32 bits is the one
    rounded to fp32 at once)."""
    v = x.double()
    s = (v.abs().amax(1) / 127.0).float().double()
    s = torch.where(s > 0, s, torch.ones_like(s))
    return torch.round((v / s[:, None]).float().double()).clamp(-127, 127), s


def product(q, s, wq, ws, dtype):
    """The definition: exact sums, two fp32 products, one rounding."""
    total = q.double() @ wq.double().T
    return (total.float() * s.float()[:, None] * ws.float()).to(dtype)


def gated_bound(h, dtype):
    """silu(gate) up in 64 bits of the fp32 products h [M, 2 I], and how far the library's may be off: the exponential by 2 + 1.2 |gate|
    steps of 2^-23, four more operations by 2^-24 each, and half a step of the result's type (or its smallest number).  Rounding to
    nearest gives an infinity from half a step above the type's largest number on, which is that number times 1 + eps / 4 (fp16: 65504 +
    16 = 65504 (1 + 2^-12)): what may reach it may be infinite."""
    gate, up = h[:, 0::2].double(), h[:, 1::2].double()
    y = gate / (1 + torch.exp(-gate)) * up
    bound = ((2 + 1.2 * gate.abs()) * 2.0 ** -23 + 4 * 2.0 ** -24 + torch.finfo(dtype).eps / 2) * y.abs()
    bound = bound * 1.001 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return y, torch.where(y.abs() + bound >= torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4), torch.inf, bound)
