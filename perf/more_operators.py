"""What is measured of the tokens' way to their experts and back and of the products in 8-bit integers.

``listed()`` and ``draw()`` give the cases, ``prepare()`` their inputs, ``run()`` one pass -- with ``own`` through the library,
else in elementary torch operations -- ``exact()`` the result from the definitions in 64 bits, and ``work()`` the bytes and
operations that a pass cannot do without.

Cases by ``op``:
  sort     token rows copied into expert order, weighted on the way where ``weights`` says "in"
  train    what surrounds the experts in a training step: rows into expert order and the experts' outputs back, weights applied
           on one of the ways, and the gradients of both
  linear   y = x W^T with 8-bit weights and a scale per channel; x comes in 16 or 32 bits and is quantised row by row in the call
  experts  a whole sparse layer behind its router: tokens quantised into expert order, gate and up products with SwiGLU, the
           result quantised row by row, down product, weighted sum; 8-bit weights with a scale per channel
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def _rows(name, op, T, k, d, E, dtype="bf16", weights="out"):
    return dict(name=name, op=op, T=T, k=k, d=d, E=E, dtype=dtype, weights=weights)


def listed():
    return [
        # a prefill chunk's tokens on their way to 128 experts
        _rows("sort_prefill", "sort", 4096, 8, 8192, 128),
        # four positions of a speculative step, weighted on the way in: nothing but latency
        _rows("sort_verify", "sort", 4, 8, 8192, 128, weights="in"),
        # a micro-batch of training; rows of odd width in fp32, weighted on the way in; a small batch in fp16
        _rows("train_batch", "train", 4096, 8, 4096, 128),
        _rows("train_odd", "train", 777, 5, 2055, 96, dtype="fp32", weights="in"),
        _rows("train_small", "train", 96, 6, 1000, 40, dtype="fp16"),
        # a projection of a decode step (8192 -> 4096), and back again for 16 tokens
        dict(name="linear_decode", op="linear", M=1, K=8192, N=4096, dtype="bf16"),
        dict(name="linear_verify", op="linear", M=16, K=4096, N=8192, dtype="bf16"),
        # the same projection for a prompt; a ragged batch through a narrow map
        dict(name="linear_prefill", op="linear", M=4096, K=8192, N=4096, dtype="bf16"),
        dict(name="linear_ragged", op="linear", M=777, K=1543, N=1001, dtype="fp32"),
        # a sparse layer: one decoded token, a prompt, and a small one of odd sizes
        dict(name="experts_decode", op="experts", T=1, k=8, d=8192, E=128, I=2048, dtype="bf16"),
        dict(name="experts_prefill", op="experts", T=4096, k=8, d=8192, E=128, I=2048, dtype="bf16"),
        dict(name="experts_odd", op="experts", T=100, k=3, d=1000, E=24, I=330, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["sort", "train", "train", "linear", "linear", "linear", "experts", "experts", "experts"])
    if op in ("sort", "train"):
        E = _log(rng, 4, 512)
        k = rng.randint(1, min(12, E))
        d = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            d = max(1, d // 64) * 64
        most = 4096 * 8 * (8192 if op == "sort" else 4096) // 2
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        T = max(1, min(_log(rng, 1, 16384), most // (k * d)))
        return dict(op=op, T=T, k=k, d=d, E=E, dtype=dtype, weights=rng.choice(["in", "out"]))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"] if op == "linear" else ["bf16", "bf16", "fp16"])
    if op == "linear":
        M, K, N = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:  # half of the maps have the even widths of a model
            K, N = max(1, K // 128) * 128, max(1, N // 128) * 128
        return dict(op=op, M=max(1, min(M, 4096 * 8192 * 4096 // (N * K))), K=K, N=N, dtype=dtype)
    E, d, I = _log(rng, 4, 128), _log(rng, 128, 8192), _log(rng, 32, 2048)
    if rng.random() < 0.5:
        d, I = max(1, d // 128) * 128, max(1, I // 64) * 64
    k = rng.randint(1, min(8, E))
    T = max(1, min(_log(rng, 1, 8192), 4096 * 8 * 8192 * 2048 // (k * d * I)))
    return dict(op=op, T=T, k=k, d=d, E=E, I=I, dtype=dtype)


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "sort":
        T, k, d, E = case["T"], case["k"], case["d"], case["E"]
        weighted = case["weights"] == "in"
        return {"bytes": size * T * d * (1 + k) + 4 * T * k * (2 + weighted) + 4 * E, "flops": T * k * d * weighted}
    if op == "train":
        T, k, d = case["T"], case["k"], case["d"]
        # x, dy in, y, dx out; the experts' outputs and their rows' gradients in, rows and the outputs' gradients out
        return {"bytes": size * T * d * (4 + 4 * k) + 4 * T * k * 3, "flops": 6 * T * k * d}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": size * M * (K + N) + N * K + 4 * N, "flops": 2 * M * N * K}
    T, k, d, E, I = case["T"], case["k"], case["d"], case["E"], case["I"]
    active = E * (1 - (1 - k / E) ** T)  # experts that a batch of this size meets
    return {"bytes": int(active * (3 * d * I + 4 * (2 * I + d)) + 2 * size * T * d + 8 * T * k), "flops": 6 * T * k * d * I}


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, K, dtype):
    """Normal rows of different sizes, some of them large, as the rows of a residual stream are."""
    x = _randn(g, rows, K) * torch.exp(0.3 * _randn(g, rows, 1))
    return x.to(DTYPES[dtype])


def _routing(g, T, k, E):
    """k different experts a token, some more popular than others, and weights that sum to 1."""
    logits = _randn(g, T, E) + 0.3 * _randn(g, E)
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(dim=1).values
    return ids.int(), torch.softmax(logits.gather(1, ids), 1)


def _weights(g, N, K):
    """8-bit weights and their channels' scales."""
    q = (_randn(g, N, K) * 36).round_().clamp_(-127, 127).to(torch.int8)
    return q, 0.02 / 36 * torch.exp(0.2 * _randn(g, N))


def _tiles(q):
    """q [N, K] in tiles of 128 rows x 64 values, the 16 values from 16 j on of all the rows of a tile next to each other."""
    N, K = q.shape
    p = torch.nn.functional.pad(q, (0, -K % 64, 0, -N % 128))
    return p.view(p.shape[0] // 128, 128, -1, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("sort", "train"):
        T, k, d, E = case["T"], case["k"], case["d"], case["E"]
        st["ids"], st["w"] = _routing(g, T, k, E)
        st["x"] = _activations(g, T, d, case["dtype"])
        if op == "train":
            st["dy"] = _activations(g, T, d, case["dtype"])
            st["outputs"] = _activations(g, T * k, d, case["dtype"])  # the experts' outputs, in expert order
            st["drows"] = _activations(g, T * k, d, case["dtype"])  # the gradient of their inputs
        return st
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = _activations(g, M, K, case["dtype"])
        st["wq"], st["ws"] = _weights(g, N, K)
        st["tiles"] = _tiles(st["wq"])  # the same as the library keeps it
        return st
    T, k, d, E, I = case["T"], case["k"], case["d"], case["E"], case["I"]
    st["ids"], st["w"] = _routing(g, T, k, E)
    st["most"] = int(torch.bincount(st["ids"].view(-1), minlength=E).max())  # rows of the busiest expert
    st["x"] = _activations(g, T, d, case["dtype"])
    for name, N, K in (("up", 2 * I, d), ("down", d, I)):  # rows 2 i and 2 i + 1 of the first: gate and up of channel i
        tile_bytes = -(-N // 128) * -(-K // 64) * 8192
        q, s = torch.empty(E, N, K, dtype=torch.int8, device="cuda"), torch.empty(E, N, device="cuda")
        tiles = torch.empty(E, tile_bytes, dtype=torch.int8, device="cuda")
        for e in range(E):
            q[e], s[e] = _weights(g, N, K)
            tiles[e] = _tiles(q[e])
        st[name + "_q"], st[name + "_s"], st[name + "_tiles"] = q, s, tiles.view(-1)
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _over(t, number):
    """t / number, rounded once (a division by a Python number may be a product with its reciprocal)."""
    return t / torch.full((1,), number, device=t.device)


def _codes(v):
    """Rows of v in 8 bits: whole numbers of -127 .. 127 in fp32, and a scale for each row."""
    s = _over(v.abs().amax(-1, keepdim=True), 127.0)
    s = torch.where(s > 0, s, 1.0)
    return torch.round(v / s).clamp(-127, 127), s


def _places(ids):
    """For each pair (token, slot) its row in expert order, and for each row its pair."""
    pairs = ids.view(-1).sort(stable=True).indices
    place = torch.empty_like(pairs)
    place[pairs] = torch.arange(pairs.numel(), device=pairs.device)
    return place, pairs


def _plain_experts(case, st):
    T, k, E, dtype = case["T"], case["k"], case["E"], DTYPES[case["dtype"]]
    flat = st["ids"].view(-1).long()
    x, sx = _codes(st["x"].float())
    token = torch.arange(T * k, device=flat.device) // k
    if T * k <= E:
        # each pair a batch of its own, with its expert's weights
        def put(v):
            return v[:, None]

        def product(v, s, name):
            return torch.bmm(v, st[name + "_q"][flat].float().transpose(1, 2)) * s * st[name + "_s"][flat][:, None]

        def take(v):
            return v[:, 0]
    else:
        # each expert's pairs a batch, as many rows as the busiest expert has
        place, pairs = _places(st["ids"])
        first = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
        first[1:] = torch.bincount(flat, minlength=E).cumsum(0)
        at = flat * st["most"] + place - first[flat]

        def put(v):
            room = torch.zeros(E * st["most"], v.shape[1], device=v.device)
            room[at] = v
            return room.view(E, st["most"], -1)

        def product(v, s, name):
            return torch.bmm(v, st[name + "_q"].float().transpose(1, 2)) * s * st[name + "_s"][:, None]

        def take(v):
            return v.reshape(-1, v.shape[2])[at]
    h = product(put(x[token]), put(sx[token]), "up")
    gate, up = h[:, :, 0::2], h[:, :, 1::2]
    h = (gate * torch.sigmoid(gate) * up).to(dtype)
    rows = take(product(*_codes(h.float()), "down").to(dtype)).float()
    return (st["w"][:, :, None] * rows.view(T, k, -1)).sum(1).to(dtype)


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, st)
    if op == "linear":
        x, s = _codes(st["x"].float())
        return ((x @ st["wq"].float().T) * s * st["ws"]).to(st["x"].dtype)
    if op == "experts":
        return _plain_experts(case, st)
    T, k, E, dtype, weighted_in = case["T"], case["k"], case["E"], st["x"].dtype, case["weights"] == "in"
    place, pairs = _places(st["ids"])
    token, w = pairs // k, st["w"].view(-1)[pairs][:, None]
    x = st["x"].float()[token]
    rows = (w * x if weighted_in else x).to(dtype)
    if op == "sort":
        ends = torch.bincount(st["ids"].view(-1), minlength=E).cumsum(0)
        return {"rows": rows, "ends": ends.int(), "place": place.int()}
    dy, drows, outputs = st["dy"].float(), st["drows"].float(), st["outputs"].float()
    y = outputs[place].view(T, k, -1)
    dx = drows[place].view(T, k, -1)
    if weighted_in:
        dw = (x * drows).sum(1)[place].view(T, k)
        dx = st["w"][:, :, None] * dx
        doutputs = dy[token]
    else:
        dw = (y * dy[:, None]).sum(2)
        y = st["w"][:, :, None] * y
        doutputs = w * dy[token]
    return {"rows": rows, "y": y.sum(1).to(dtype), "dx": dx.sum(1).to(dtype), "dw": dw, "doutputs": doutputs.to(dtype)}


def _run_own(case, op, st):
    from bit_expert_ffn_moe_gb300 import ops

    if op == "linear":
        if "W" not in st:
            st["W"] = ops.Int8Weights(case["N"], case["K"], st["tiles"], st["ws"])
            st["workspace"] = ops.int8_workspace(case["M"], case["N"], case["K"])
        return ops.int8_linear(st["x"], st["W"], st["workspace"])
    if op == "experts":
        if "layer" not in st:
            from bit_expert_ffn_moe_gb300.block import Int8Experts
            E, d, I = case["E"], case["d"], case["I"]
            st["layer"] = Int8Experts(ops.Int8Weights(2 * I, d, st["up_tiles"], st["up_s"]),
                                      ops.Int8Weights(d, I, st["down_tiles"], st["down_s"]), case["T"], case["k"])
        return st["layer"](st["x"], st["ids"], st["w"])
    weights_in, weights_out = (st["w"], None) if case["weights"] == "in" else (None, st["w"])
    order = ops.expert_order(st["ids"], case["E"])
    rows = ops.tokens_to_experts(st["x"], order, weights_in)
    if op == "sort":
        return {"rows": rows, "ends": order.offsets[1:], "place": order.inv.view(-1)}
    y = ops.experts_to_tokens(st["outputs"], order, weights_out)
    doutputs, dw_out = ops.experts_to_tokens_backward(st["dy"], order, st["outputs"], weights_out)
    dx, dw_in = ops.tokens_to_experts_backward(st["drows"], order, st["x"], weights_in)
    return {"rows": rows, "y": y, "dx": dx, "dw": dw_out if dw_in is None else dw_in, "doutputs": doutputs}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _fp32(t):
    """A 64-bit result rounded once to fp32, where the format's rule rounds."""
    return t.float().double()


def _numbers(x):
    """The whole numbers that the 8-bit rows of x hold and the rows' scales, in 64 bits."""
    v = x.double()
    scale = _fp32(v.abs().max(dim=-1).values / 127.0)
    scale[scale == 0] = 1.0
    quotient = _fp32(v / scale[:, None])
    lower = quotient.floor()
    rest = quotient - lower
    up = (rest > 0.5) | ((rest == 0.5) & (lower.remainder(2) == 1))
    return lower + up, scale[:, None]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    dtype = DTYPES[case["dtype"]]
    if op == "linear":
        q, scale = _numbers(st["x"])
        return (q @ st["wq"].double().T) * scale * st["ws"].double()
    T, k, E = case["T"], case["k"], case["E"]
    ids, w = st["ids"].long(), st["w"].double()
    if op == "experts":
        q, scale = _numbers(st["x"])
        y = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
        for e in range(E):
            token, slot = (ids == e).nonzero(as_tuple=True)
            if token.numel() == 0:
                continue
            h = (q[token] @ st["up_q"][e].double().T) * scale[token] * st["up_s"][e].double()
            gate, up = h.view(h.shape[0], -1, 2).unbind(2)
            hq, hs = _numbers((gate / (1 + torch.exp(-gate)) * up).to(dtype))  # in the inputs' type, as the definition has it
            out = ((hq @ st["down_q"][e].double().T) * hs * st["down_s"][e].double()).to(dtype).double()
            y.index_add_(0, token, w[token, slot][:, None] * out)
        return y
    x, d = st["x"].double(), case["d"]
    # pairs by (expert, token, slot): sorted by one number each
    rank = (ids.view(-1) * (T * k) + torch.arange(T * k, device="cuda")).sort().values
    pair = rank % (T * k)
    token, weight = pair // k, w.view(-1)[pair]
    weighted_in = case["weights"] == "in"
    rows = x[token] * (weight[:, None] if weighted_in else 1.0)
    if op == "sort":
        place = torch.zeros(T * k, dtype=torch.int32, device="cuda").scatter_(0, pair, torch.arange(T * k, device="cuda").int())
        ends = (rank[None, :] // (T * k) <= torch.arange(E, device="cuda")[:, None]).sum(1) if E * T * k <= 1 << 24 else None
        return {"rows": rows, "ends": None if ends is None else ends.int(), "place": place}
    dy, drows, outputs = st["dy"].double(), st["drows"].double(), st["outputs"].double()
    way_out = weight[:, None] if not weighted_in else 1.0
    way_in = weight[:, None] if weighted_in else 1.0
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add_(0, token, outputs * way_out)
    dx = torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add_(0, token, drows * way_in)
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    dw[pair] = torch.einsum("pd,pd->p", x[token], drows) if weighted_in else torch.einsum("pd,pd->p", dy[token], outputs)
    return {"rows": rows, "y": y, "dx": dx, "dw": dw.view(T, k), "doutputs": dy[token] * way_out}
