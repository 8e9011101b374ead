"""What is measured of the routing rules, of their gradients and of the dense NVFP4 products.

``listed()`` and ``draw()`` give the cases, ``prepare()`` their inputs, ``run()`` one pass -- with ``own`` through
the library, else in elementary torch operations -- ``exact()`` the result from the definitions in 64 bits, and
``work()`` the bytes and operations that a pass cannot do without.

Cases by ``op``:
  route    scores, balance bias, groups, top-k and weights of a batch of router logits (serving)
  tune     the same and the gradient of the logits (tuning the router over frozen experts)
  combine  gradients of the weighted sum of the expert outputs
  linear   y = x W^T with NVFP4 weights; x comes in 16 or 32 bits and is quantised in the call (serving)
  train    an NVFP4 linear map's forward and both gradients; x, W and dy come in bf16
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------ cases

def _route(name, op, T, E, k, dtype="fp32", score="sigmoid", bias=True, groups=1, top_groups=1, group_score="top2",
           renormalize=True, scale=1.0, out_of_service=0):
    return dict(name=name, op=op, T=T, E=E, k=k, dtype=dtype, score=score, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renormalize=renormalize, scale=scale,
                out_of_service=out_of_service)


def listed():
    return [
        # one token of a decode step: nothing but latency
        _route("route_decode", "route", 1, 256, 8, groups=8, top_groups=4, scale=2.5),
        # two prefill chunks of 8192 tokens, balance bias and group-limited choice
        _route("route_prefill", "route", 16384, 256, 8, groups=8, top_groups=4, scale=2.5),
        # the plain rule on 16-bit logits, a prompt of 4096 tokens
        _route("route_softmax", "route", 4096, 128, 8, dtype="bf16", score="softmax", bias=False),
        # one micro-batch of router tuning
        _route("tune_sigmoid", "tune", 8192, 256, 8, groups=8, top_groups=4, scale=2.5),
        # odd sizes, softmax over groups chosen by their maximum, three experts out of service
        _route("tune_softmax_odd", "tune", 1003, 160, 6, dtype="fp16", score="softmax", groups=8, top_groups=3,
               group_score="max", renormalize=False, scale=16.0, out_of_service=3),
        # the weighted sum of the prefill workload, and of an odd small batch
        dict(name="combine_prefill", op="combine", T=4096, k=8, d=8192),
        dict(name="combine_odd", op="combine", T=333, k=5, d=2056),
        # the latent projection of a decode step (8192 -> 4096), and back again for 16 tokens
        dict(name="linear_decode", op="linear", M=1, K=8192, N=4096, dtype="bf16"),
        dict(name="linear_verify", op="linear", M=16, K=4096, N=8192, dtype="bf16"),
        # the same projection for a prompt; a ragged batch through a narrow map
        dict(name="linear_prefill", op="linear", M=4096, K=8192, N=4096, dtype="bf16"),
        dict(name="linear_ragged", op="linear", M=777, K=1544, N=1000, dtype="fp16"),
        # one micro-batch of training that projection
        dict(name="train_latent", op="train", M=4096, K=8192, N=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "route", "tune", "tune", "combine", "linear", "linear", "linear", "train"])
    if op in ("route", "tune"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, _log(rng, 16, 512) // groups)
        T = min(_log(rng, 1, 16384), (16384 * 256) // E)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        case = _route("", op, T, E, k, rng.choice(["fp32", "bf16", "fp16"]), rng.choice(["sigmoid", "softmax"]),
                      rng.random() < 0.7, groups, top_groups, rng.choice(["max", "top2"]), rng.random() < 0.7,
                      rng.choice([1.0, 2.5]), rng.choice([0, 0, 1, 5]) if E >= 16 else 0)
        del case["name"]
        return case
    if op == "combine":
        T, k, d = _log(rng, 1, 8192), rng.randint(1, 12), 8 * _log(rng, 16, 1024)
        return dict(op=op, T=max(1, min(T, 4096 * 8 * 8192 // (k * d))), k=k, d=d)
    dtype = rng.choice(["bf16", "fp16", "fp32"] if op == "linear" else ["bf16"])
    M = _log(rng, 1, 8192) if op == "linear" else _log(rng, 64, 8192)
    K, N = _log(rng, 256, 8192), _log(rng, 256, 8192)
    if rng.random() < 0.5:  # half of the maps have the even widths of a model
        K, N = max(1, K // 256) * 256, max(1, N // 256) * 256
    M = max(1, min(M, 4096 * 8192 * 4096 // (N * K)))
    return dict(op=op, M=M, K=K, N=N, dtype=dtype)


def work(case):
    op = case["op"]
    if op in ("route", "tune"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return {"bytes": T * E * size + 4 * E * case["bias"] + 8 * T * k, "flops": 8 * T * E}
        return {"bytes": 2 * T * E * size + 4 * E * case["bias"] + 12 * T * k, "flops": 16 * T * E}
    if op == "combine":
        T, k, d = case["T"], case["k"], case["d"]
        return {"bytes": 2 * T * d + 4 * T * k * d + 12 * T * k, "flops": 3 * T * k * d}
    M, N, K = case["M"], case["N"], case["K"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "linear":
        return {"bytes": size * M * (K + N) + N * K * 9 // 16, "flops": 2 * M * N * K}
    return {"bytes": 2 * 2 * (M * K + N * K + M * N), "flops": 6 * M * N * K}


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, K, dtype):
    """Normal rows of different sizes, some of them large, as the rows of a residual stream are."""
    x = _randn(g, rows, K) * torch.exp(0.3 * _randn(g, rows, 1))
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("route", "tune"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(g, T, E)
        if case["out_of_service"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[:case["out_of_service"]]] = -float("inf")
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        # the size a balance bias reaches: a few times the spread of the scores near the choice's border
        st["bias"] = _randn(g, E) * (0.05 if case["score"] == "sigmoid" else 0.5 / E) if case["bias"] else None
        if op == "tune":
            st["dw"] = _randn(g, T, k)
        return st
    if op == "combine":
        T, k, d = case["T"], case["k"], case["d"]
        E = max(16, k)
        ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].sort(1).values
        inv = torch.empty(T * k, dtype=torch.int64, device="cuda")
        inv[ids.reshape(-1).argsort(stable=True)] = torch.arange(T * k, device="cuda")
        st["inv_pos"] = inv.int()
        st["dy"] = _randn(g, T, d).bfloat16()
        st["y_perm"] = _randn(g, T * k, d).bfloat16()
        st["w"] = torch.softmax(_randn(g, T, k), 1)
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"] = _activations(g, M, K, case["dtype"])
    w = _randn(g, N, K) * 0.02
    if op == "linear":
        # the stored weights: packed codes, scale bytes and one scale of the matrix; and, for the tensor cores, the
        # same codes and scales in their operand layout
        gs = _over(w.abs().max(), 2688.0)
        codes, scales = _codes(w, gs.expand(N, 1))
        st["wg"] = gs.reshape(1)
        st["wq"], st["ws"] = _pack(codes), scales.to(torch.float8_e4m3fn).view(torch.uint8)
        st["wq_tiles"], st["ws_atoms"] = _tiles(st["wq"]), _atoms(st["ws"])
    else:
        st["w"] = w.bfloat16()
        st["dy"] = _activations(g, M, N, case["dtype"])
    return st


def _over(t, number):
    """t / number, rounded once (a division by a Python number may be a product with its reciprocal)."""
    return t / torch.full((1,), number, device=t.device)


def _pad(t, rows, cols):
    return torch.nn.functional.pad(t, (0, -t.shape[1] % cols, 0, -t.shape[0] % rows))


def _pack(codes):
    """Codes [rows][K] -> bytes [rows][K/2], element 2i in the low nibble; K counts whole blocks of 32 here."""
    c = _pad(codes, 1, 32).view(codes.shape[0], -1, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4)


def _tiles(q):
    """Packed codes as tiles of 128 rows x 128 bytes, the 16-byte piece j of row r at place j ^ (r % 8)."""
    p = _pad(q, 128, 128)
    t = p.view(p.shape[0] // 128, 128, -1, 8, 16).permute(0, 2, 1, 3, 4)
    r, j = torch.arange(128, device=q.device), torch.arange(8, device=q.device)
    at = (j[None, :] ^ (r[:, None] % 8)).view(1, 1, 128, 8, 1).expand_as(t)
    return t.gather(3, at).reshape(-1).contiguous()


def _atoms(s):
    """Scale bytes [rows][K/16] as 512-byte atoms of 128 rows x 4 scales."""
    p = _pad(_pad(s, 1, 16), 128, 4)
    return p.view(p.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_route(case, logits, bias):
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    l = logits.double()  # the choice is made on values next to a border
    served = l > -float("inf")
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    v = l if bias is None else s + bias.double()
    if groups > 1:
        gv = v if case["group_score"] == "max" else (s if bias is None else v)
        gv = torch.where(served, gv, -float("inf")).view(T, groups, -1).sort(dim=2, descending=True).values
        gs = gv[:, :, 0]
        if case["group_score"] == "top2" and gv.shape[2] > 1:
            gs = gs + torch.where(gv[:, :, 1] > -float("inf"), gv[:, :, 1], 0.0)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        stays = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        stays = stays.repeat_interleave(E // groups, 1)
    else:
        stays = torch.ones_like(served)
    rank = torch.where(stays, torch.where(served, v, -1e300), -float("inf"))
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
    s = (torch.sigmoid(logits.float()) if case["score"] == "sigmoid" else torch.softmax(logits.float(), 1))
    u = s.gather(1, ids)
    w = case["scale"] * (u / u.sum(1, keepdim=True) if case["renormalize"] else u)
    return ids, s, u, w


def _plain_route_backward(case, s, ids, u, dw):
    if case["renormalize"]:
        S = u.sum(1, keepdim=True)
        du = case["scale"] * (dw - (dw * u).sum(1, keepdim=True) / S) / S
    else:
        du = case["scale"] * dw
    ds = torch.zeros_like(s).scatter_(1, ids, du)
    if case["score"] == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _codes(v, gs):
    """Codes [rows][K] and scale values [rows][ceil(K/16)] of fp32 v under the row scales gs [rows][1]."""
    rows, K = v.shape
    b = _pad(v, 1, 16).view(rows, -1, 16)
    scales = _over(b.abs().amax(2) / gs, 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    D = (scales * gs)[:, :, None]
    m = torch.where(D > 0, b.abs() / D, 0.0)
    c = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte() +
         (m >= 3.5).byte() + (m > 5.0).byte())
    c = torch.where((b < 0) & (c > 0), c + 8, c)
    return c.view(rows, -1)[:, :K], scales


def _values(codes, scales):
    """The numbers that codes and scale values stand for, without the row scale."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    v = table[_pad(codes, 1, 16).int()].view(codes.shape[0], -1, 16) * scales[:, :, None]
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _quantized(x):
    """x [rows][K] as NVFP4 rows: their values without the row scale, and the row scales."""
    v = x.float()
    gs = _over(v.abs().amax(1, keepdim=True), 2688.0)
    gs = torch.where(gs > 0, gs, 1.0)
    return _values(*_codes(v, gs)), gs


def _product(a, b, dtype):
    return ((a[0] @ b[0].T) * (a[1] * b[1].T)).to(dtype)


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, st)
    if op in ("route", "tune"):
        ids, s, u, w = _plain_route(case, st["logits"], st["bias"])
        if op == "route":
            return {"ids": ids.int(), "w": w}
        dl = _plain_route_backward(case, s, ids, u, st["dw"])
        return {"ids": ids.int(), "w": w, "dlogits": dl.to(st["logits"].dtype)}
    if op == "combine":
        T, k = case["T"], case["k"]
        dy, at = st["dy"].float(), st["inv_pos"].long()
        dw = (dy[:, None, :] * st["y_perm"].float()[at].view(T, k, -1)).sum(2)
        dy_perm = torch.empty_like(st["y_perm"])
        dy_perm[at] = (st["w"][:, :, None] * dy[:, None, :]).view(T * k, -1).bfloat16()
        return {"dw": dw, "dy_perm": dy_perm}
    if op == "linear":
        N, K = case["N"], case["K"]
        codes = torch.stack((st["wq"] & 15, st["wq"] >> 4), 2).view(N, -1)[:, :K]
        scales = st["ws"].view(torch.float8_e4m3fn).float()
        return _product(_quantized(st["x"]), (_values(codes, scales), st["wg"].expand(N, 1)), st["x"].dtype)
    x, w, dy = st["x"], st["w"], st["dy"]
    return {"y": _product(_quantized(x), _quantized(w), x.dtype),
            "dx": _product(_quantized(dy), _quantized(w.T), x.dtype),
            "dw": _product(_quantized(dy.T), _quantized(x.T), x.dtype)}


def _run_own(case, op, st):
    from bit_expert_ffn_moe_gb300 import binding as B
    from bit_expert_ffn_moe_gb300 import ops

    if op in ("route", "tune"):
        if "rule" not in st:
            st["rule"] = ops.route_rule(case["score"], case["groups"], case["top_groups"], case["group_score"],
                                        case["renormalize"], case["scale"])
        ids, w = ops.route_scores(st["logits"], case["k"], st["rule"], st["bias"])
        if op == "route":
            return {"ids": ids, "w": w}
        return {"ids": ids, "w": w, "dlogits": ops.route_scores_backward(st["logits"], ids, st["dw"], st["rule"])}
    if op == "combine":
        dw, dy_perm = ops.combine_backward(st["dy"], st["y_perm"], st["inv_pos"], st["w"])
        return {"dw": dw, "dy_perm": dy_perm}
    if op == "linear":
        if "W" not in st:
            st["W"] = ops.Nvfp4Operand(case["N"], case["K"], st["wq_tiles"], st["ws_atoms"], st["wg"])
            st["workspace"] = ops.nvfp4_workspace(case["M"], case["N"], case["K"])
        return ops.nvfp4_linear(st["x"], st["W"], st["workspace"])
    M, N, K = case["M"], case["N"], case["K"]
    if "workspace" not in st:
        st["workspace"] = ops.nvfp4_workspace(M, N, K)
        st["xr"], st["xc"] = ops.nvfp4_operand(M, K), ops.nvfp4_operand(K, M)
        st["wr"], st["wc"] = ops.nvfp4_operand(N, K), ops.nvfp4_operand(K, N)
        st["dr"], st["dc"] = ops.nvfp4_operand(M, N), ops.nvfp4_operand(N, M)
    ws = st["workspace"]
    ops.nvfp4_quantize(st["x"], st["xr"], st["xc"], ws)
    ops.nvfp4_quantize(st["w"], st["wr"], st["wc"], ws)
    ops.nvfp4_quantize(st["dy"], st["dr"], st["dc"], ws)
    return {"y": ops.nvfp4_matmul(st["xr"], st["wr"], st["x"].dtype, ws),
            "dx": ops.nvfp4_matmul(st["dr"], st["wc"], st["x"].dtype, ws),
            "dw": ops.nvfp4_matmul(st["dc"], st["xc"], st["x"].dtype, ws)}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_route(case, logits, bias, dw):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    out = np.isneginf(logits)
    with np.errstate(over="ignore"):
        if case["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-logits))
        else:
            e = np.exp(logits - logits.max(1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
    v = logits.copy() if bias is None else s + bias
    key = np.where(out, -1e200, v)
    if G > 1:
        per = E // G
        g = np.where(out, -np.inf, s if bias is None and case["group_score"] == "top2" else v).reshape(T, G, per)
        top = -np.sort(-g, axis=2)[:, :, :2]
        gs = top[:, :, 0].copy()
        if case["group_score"] == "top2" and per > 1:
            gs += np.where(np.isneginf(top[:, :, 1]), 0.0, top[:, :, 1])
        order = np.argsort(-gs, axis=1, kind="stable")
        place = np.empty_like(order)
        np.put_along_axis(place, order, np.broadcast_to(np.arange(G), (T, G)), 1)
        key = np.where(np.repeat(place < case["top_groups"], per, axis=1), key, -np.inf)
    ids = np.sort(np.argsort(-key, axis=1, kind="stable")[:, :k], axis=1)
    u = np.take_along_axis(s, ids, 1)
    S = u.sum(1, keepdims=True)
    c = case["scale"]
    w = c * u / S if case["renormalize"] else c * u
    if dw is None:
        return {"ids": torch.from_numpy(ids.astype(np.int32)), "w": torch.from_numpy(w)}
    du = c * (dw / S - (dw * u).sum(1, keepdims=True) / S ** 2) if case["renormalize"] else c * dw
    if case["score"] == "sigmoid":
        dl = np.zeros((T, E))
        lu = np.take_along_axis(logits, ids, 1)
        np.put_along_axis(dl, ids, du * u / (1.0 + np.exp(lu)), 1)
    else:
        dl = -s * (du * u).sum(1, keepdims=True)
        np.put_along_axis(dl, ids, np.take_along_axis(dl, ids, 1) + du * u, 1)
    return {"ids": torch.from_numpy(ids.astype(np.int32)), "w": torch.from_numpy(w), "dlogits": torch.from_numpy(dl)}


def _fp32(t):
    """A 64-bit result rounded once to fp32, where the format's rule rounds."""
    return t.float().double()


def _exact_rows(x):
    """The numbers that the NVFP4 rows of x stand for, in 64 bits: nearest scale and code among the format's values."""
    v = x.double()
    rows, K = v.shape
    gs = _fp32(v.abs().amax(1) / 2688.0)
    gs = torch.where(gs == 0, torch.ones_like(gs), gs)
    blocks = -(-K // 16)
    b = torch.zeros(rows, blocks * 16, dtype=torch.float64, device=v.device)
    b[:, :K] = v
    b = b.view(rows, blocks, 16)
    t = _fp32(_fp32(b.abs().amax(2) / gs[:, None]) / 6.0)
    ebits = torch.arange(127, device=v.device)  # the non-negative finite E4M3 values, by code
    e4m3 = torch.where(ebits >= 8, (8 + ebits % 8) * 2.0 ** ((ebits // 8).double() - 10), ebits * 2.0 ** -9)
    scale = e4m3[_nearest(t, e4m3)]
    D = _fp32(scale * gs[:, None])[:, :, None]
    mag = _fp32(b.abs() / torch.where(D > 0, D, torch.ones_like(D)))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    q = grid[_nearest(mag, grid)] * torch.sign(b) * scale[:, :, None] * (D > 0)
    return q.view(rows, -1)[:, :K] * gs[:, None]


def _nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, beyond the last: the last."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
    mid = (grid[hi - 1] + grid[hi]) / 2
    up = (v > mid) | ((v == mid) & (hi % 2 == 0))
    return torch.where(up, hi, hi - 1)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("route", "tune"):
        host = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return _exact_route(case, host(st["logits"]), host(st["bias"]), host(st.get("dw")))
    if op == "combine":
        T, k = case["T"], case["k"]
        at = st["inv_pos"].long().view(T, k)
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        dy_perm = torch.empty(T * k, case["d"], dtype=torch.float64, device="cuda")
        dy = st["dy"].double()
        for j in range(k):
            dw[:, j] = torch.einsum("td,td->t", dy, st["y_perm"][at[:, j]].double())
            dy_perm[at[:, j]] = dy * st["w"][:, j:j + 1].double()
        return {"dw": dw, "dy_perm": dy_perm}
    if op == "linear":
        N, K = case["N"], case["K"]
        low, high = st["wq"].long() % 16, st["wq"].long() // 16
        c = torch.stack((low, high), 2).reshape(N, -1)[:, :K]
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        sb = st["ws"].long().repeat_interleave(16, 1)[:, :K]
        scale = torch.where(sb >= 8, (8 + sb % 8) * 2.0 ** ((sb // 8).double() - 10), sb * 2.0 ** -9)
        w = grid[c % 8] * (1 - 2 * (c // 8)) * scale * st["wg"].double()
        return _exact_rows(st["x"]) @ w.T
    x, w, dy = st["x"], st["w"], st["dy"]
    return {"y": _exact_rows(x) @ _exact_rows(w).T, "dx": _exact_rows(dy) @ _exact_rows(w.T).T,
            "dw": _exact_rows(dy.T) @ _exact_rows(x.T).T}
