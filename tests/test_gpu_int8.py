"""Products in 8-bit integers against the definition in 64 bits.  Sums below 2^24 are exact on both sides, so results are equal bit for
bit; gated ones are held to the bound of expert_reference.gated_bound."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def acts(g, rows, K, dtype):
    return (torch.randn(rows, K, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


def whole(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-4


SHAPES = [(1, 1, 1), (1, 130, 64), (1, 4096, 2048), (2, 7, 63), (3, 128, 65), (4, 256, 128), (5, 100, 1000), (8, 1000, 320), (16, 129, 777),
          (17, 64, 64), (33, 300, 130), (64, 512, 1024), (100, 333, 500), (129, 257, 192), (256, 128, 4096), (257, 384, 320), (300, 1001, 1543),
          (520, 640, 512), (1000, 2000, 96), (2100, 1300, 700)]
# whole tiles and shared ones behind them, in one CTA and in several, and products whose last tiles alone are shared
MANY = [(1100, 4100, 2100), (2500, 5000, 1500), (450, 9000, 4096), (3500, 2000, 3300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    g = gen(M + N + K)
    x, wq, ws = acts(g, M, K, dtype), whole(g, N, K), scales(g, N)
    y = ops.int8_linear(x, ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K))
    assert y.dtype == dtype and torch.equal(y, R.product(*R.numbers(x), wq, ws, dtype))


@pytest.mark.parametrize("M,N,K", MANY)
def test_more_tiles_than_ctas(M, N, K):
    g = gen(M + N + K)
    x, wq, ws = acts(g, M, K, torch.bfloat16), whole(g, N, K), scales(g, N)
    W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
    want = R.product(*R.numbers(x), wq, ws, torch.bfloat16)
    for _ in range(3):
        assert torch.equal(ops.int8_linear(x, W, space), want)
    y, bound = R.gated_bound(R.product(*R.numbers(x), wq, ws, torch.float32), torch.bfloat16)
    assert ((ops.int8_linear(x, W, space, gated=True).double() - y).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,I,K", [(1, 1, 64), (2, 65, 100), (9, 64, 640), (40, 200, 333), (300, 130, 512), (700, 500, 128)])
def test_gated(M, I, K, dtype):
    g = gen(M + I + K)
    x, gate, up, s, u = acts(g, M, K, dtype), whole(g, I, K), whole(g, I, K), scales(g, I), scales(g, I)
    W = ops.int8_weights(gate, s, up, u)
    q, sx = R.numbers(x)
    h = torch.stack((R.product(q, sx, gate, s, torch.float32), R.product(q, sx, up, u, torch.float32)), 2).view(M, -1)
    ws = ops.int8_workspace(M, 2 * I, K)
    assert torch.equal(ops.int8_matmul(ops.int8_quantize(x), W, torch.float32, ws), h)
    y, bound = R.gated_bound(h, dtype)
    assert ((ops.int8_linear(x, W, ws, gated=True).double() - y).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_every_kind(dtype):
    """Zeros, one number, halves between whole numbers, the type's largest and smallest numbers."""
    info, g = torch.finfo(dtype), gen(2)
    x = acts(g, 12, 200, dtype)
    x[0] = 0
    x[1] = 0
    x[1, 77] = -3.0
    x[2] = (torch.arange(200, device="cuda") - 100).to(dtype) / 2
    x[2, 0] = 127
    x[3] = info.max
    x[4] = info.smallest_normal
    x[5] = info.smallest_normal * info.eps  # the smallest number
    x[6] = 0
    x[6, 199] = info.smallest_normal * info.eps
    x[7, ::2] = info.max
    q, s = R.numbers(x)
    rows = ops.int8_quantize(x)
    assert torch.equal(rows.s[:12], s.float())
    assert torch.equal(rows.values()[:12], (q * s[:, None]).float())
    wq, ws = whole(g, 50, 200), scales(g, 50)
    y = ops.int8_linear(x, ops.int8_weights(wq, ws), ops.int8_workspace(12, 50, 200))
    assert torch.equal(y, R.product(q, s, wq, ws, dtype))


def test_nan_and_infinity_make_their_row_nan():
    g = gen(3)
    for M in (3, 40):
        x = acts(g, M, 300, torch.bfloat16)
        clean = x.clone()
        x[0, 5], x[2, 299] = float("nan"), -float("inf")
        W, ws = ops.int8_weights(whole(g, 70, 300), scales(g, 70)), ops.int8_workspace(M, 70, 300)
        y, want = ops.int8_linear(x, W, ws), ops.int8_linear(clean, W, ws)
        assert torch.isnan(y[[0, 2]]).all()
        keep = torch.ones(M, dtype=torch.bool)
        keep[[0, 2]] = False
        assert torch.equal(y[keep], want[keep])


def test_quantised_weights():
    g = gen(4)
    for dtype in TYPES:
        w = acts(g, 3 * 130, 200, dtype).view(3, 130, 200)
        W = ops.int8_weights(w)
        q, s = R.numbers(w.view(-1, 200))
        assert W.E == 3 and torch.equal(W.s, s.float()) and torch.equal(W.values().view(-1, 200), (q * s[:, None]).float())


@pytest.mark.parametrize("M", [1, 3, 20, 300])
def test_largest_sums(M):
    """Sums of one sign up to 127 x 127 x 131072: exact up to 2^24, behind that each of at most K / 16 additions of an fp32 sum rounds by
    2^-24, and so do two products (the library adds in whole numbers or in fp32)."""
    K, N = 131072, 40
    x = torch.ones(M, K, device="cuda").bfloat16()
    wq = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    wq[::2] = -127
    y = ops.int8_linear(x, ops.int8_weights(wq, torch.ones(N, device="cuda")), ops.int8_workspace(M, N, K))
    want = torch.full((M, N), 127.0 * K, dtype=torch.float64, device="cuda")
    want[:, ::2] *= -1
    assert ((y.double() - want).abs() <= (K / 16 * 2.0 ** -24 + 2.0 ** -8 + 2.0 ** -20) * want.abs()).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [2, 30, 270])
@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 0), (8, 1), (0, 3)])
def test_strides_and_addresses(M, dtype, pad, shift):
    g = gen(5)
    K, N = 328, 214
    x, W, ws = acts(g, M, K, dtype), ops.int8_weights(whole(g, N, K), scales(g, N)), ops.int8_workspace(M, N, K)

    def odd(n):
        return torch.full((M * (n + pad) + shift,), 7.0, device="cuda", dtype=dtype)[shift:].view(M, n + pad)
    xo, yo = odd(K), odd(N)
    xo[:, :K] = x
    for gated in (False, True):
        n = N // 2 if gated else N
        want = ops.int8_linear(x, W, ws, gated)
        yo.fill_(7.0)
        y = ops.int8_linear(xo[:, :K], W, ws, gated, yo[:, :n])
        assert y.data_ptr() == yo.data_ptr() and torch.equal(y, want) and (yo[:, n:] == 7.0).all()


def test_results_in_another_type():
    g = gen(6)
    x, wq, s = acts(g, 20, 100, torch.float16), whole(g, 30, 100), scales(g, 30)
    W, ws = ops.int8_weights(wq, s), ops.int8_workspace(20, 30, 100)
    for dtype in TYPES:
        want = R.product(*R.numbers(x), wq, s, dtype)
        assert torch.equal(ops.int8_matmul(ops.int8_quantize(x), W, dtype, ws), want)
        assert torch.equal(ops.int8_linear(x, W, ws, out=torch.empty(20, 30, dtype=dtype, device="cuda")), want)


def test_experts_of_many_tiles():
    """Whole and shared tiles of experts of every size, with single CTAs and with pairs."""
    g = gen(12)
    for counts in ([700, 0, 30, 1, 900, 200], [5] * 60 + [0, 300, 77]):
        E, N, K = len(counts), 1300, 2100
        ids, order = sorted_order(counts)
        M = len(ids)
        x, wq, ws = acts(g, M, K, torch.bfloat16), whole(g, E, N, K), scales(g, E, N)
        W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
        q, s = R.numbers(x)
        want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            t = (ids.view(-1) == e).nonzero().view(-1)
            want[order.inv.view(-1)[t].long()] = R.product(q[t], s[t], wq[e], ws[e], torch.bfloat16)
        rows = ops.int8_quantize(x, order)
        for _ in range(2):
            assert torch.equal(ops.int8_matmul(rows, W, torch.bfloat16, space), want)


COUNTS = [[1], [0, 0, 1], [1] * 8, [3, 0, 5, 1, 0, 2], [0, 40, 0, 7], [300, 0, 1, 17, 256, 257, 0], [16, 15, 17, 128, 129], [0, 0]]


def sorted_order(counts):
    """An order of one slot whose experts have these many tokens, in turns."""
    ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(len(ids)))].view(-1, 1)
    return ids.cuda(), ops.expert_order(ids.cuda(), len(counts))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(1, 64), (130, 200), (384, 1000), (600, 64)])
def test_experts_products(counts, N, K, dtype):
    g = gen(sum(counts) + N + K)
    E = len(counts)
    ids, order = sorted_order(counts)
    M = len(ids)
    x, wq, ws = acts(g, M, K, dtype), whole(g, E, N, K), scales(g, E, N)
    W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
    q, s = R.numbers(x)
    want = torch.empty(M, N, dtype=dtype, device="cuda")
    for e in range(E):
        t = (ids.view(-1) == e).nonzero().view(-1)
        want[order.inv.view(-1)[t].long()] = R.product(q[t], s[t], wq[e], ws[e], dtype)
    rows = ops.int8_quantize(x, order)
    assert torch.equal(ops.int8_matmul(rows, W, dtype, space), want)
    spread = ops.tokens_to_experts(x, order)
    again = ops.int8_quantize(spread, order, ordered=True)
    assert torch.equal(ops.int8_matmul(again, W, dtype, space), want)
    if N % 2 == 0:
        h = ops.int8_matmul(rows, W, torch.float32, space)
        y, bound = R.gated_bound(h, dtype)
        assert ((ops.int8_matmul(rows, W, dtype, space, gated=True).double() - y).abs() <= bound).all()


def test_rows_behind_the_last_stay():
    g = gen(7)
    ids = R.some_ids(50, 4, 10, 7, "dropped").cuda()
    order = ops.expert_order(ids, 10)
    n = int(order.offsets[-1])
    assert 0 < n < 200
    x, W, ws = acts(g, 50, 96, torch.bfloat16), ops.int8_weights(whole(g, 10, 66, 96), scales(g, 10, 66)), ops.int8_workspace(200, 66, 96)
    out = torch.full((200, 66), 7.0, device="cuda").bfloat16()
    ops.int8_matmul(ops.int8_quantize(x, order), W, torch.bfloat16, ws, out=out)
    assert (out[n:] == 7.0).all() and not (out[:n] == 7.0).all(1).any()


LAYERS = [(1, 1, 64, 1, 1), (1, 8, 512, 16, 64), (4, 2, 200, 5, 33), (30, 3, 1000, 24, 330), (64, 8, 256, 8, 128), (500, 4, 384, 12, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["distinct", "dropped"])
@pytest.mark.parametrize("T,k,d,E,I", LAYERS)
def test_sparse_layer(T, k, d, E, I, kind, dtype):
    """Every stage is the definition's of what the stage before gave, bit for bit but for the gate's exponential and the sum."""
    from bit_expert_ffn_moe_gb300.block import Int8Experts
    g = gen(T + k + d + E + I)
    ids = R.some_ids(T, k, E, T + d, kind).cuda()
    x, w = acts(g, T, d, dtype), torch.rand(T, k, generator=g, device="cuda")
    gate, upper, down = whole(g, E, I, d), whole(g, E, I, d), whole(g, E, d, I)
    s1, s2, s3 = scales(g, E, I) / 100, scales(g, E, I) / 100, scales(g, E, d)
    layer = Int8Experts(ops.int8_weights(gate, s1, upper, s2), ops.int8_weights(down, s3), T, k, dtype)
    y = layer(x, ids, w)
    rows, order = layer.outputs(x, ids)
    assert torch.equal(y, ops.experts_to_tokens(rows, order, w))
    q, s = R.numbers(x)
    h = ops.int8_matmul(ops.int8_quantize(x, order), layer.up, dtype, layer.workspace, gated=True)
    flat = ids.view(-1)
    for e in range(E):
        p = (flat == e).nonzero().view(-1)
        if not len(p):
            continue
        r, t = order.inv.view(-1)[p].long(), p // k
        products = torch.stack((R.product(q[t], s[t], gate[e], s1[e], torch.float32), R.product(q[t], s[t], upper[e], s2[e], torch.float32)), 2)
        want, bound = R.gated_bound(products.view(len(p), -1), dtype)
        assert ((h[r].double() - want).abs() <= bound).all()
        assert torch.equal(rows[r], R.product(*R.numbers(h[r]), down[e], s3[e], dtype))


def test_in_graphs_that_share_a_workspace():
    g = gen(8)
    W, ws = ops.int8_weights(whole(g, 700, 640), scales(g, 700)), ops.int8_workspace(400, 700, 640)
    inputs = [acts(g, M, 640, torch.bfloat16) for M in (1, 13, 400)]
    plain = [ops.int8_linear(x, W, ws) for x in inputs]
    graphs, outs = [], []
    for x in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ops.int8_linear(x, W, ws))
        graphs.append(graph)
    for i in (0, 1, 2, 2, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], plain[i])


def test_many_calls_in_a_row():
    """No call waits for the host, and none takes anything over from the one before."""
    g = gen(9)
    W, ws = ops.int8_weights(whole(g, 512, 1024), scales(g, 512)), ops.int8_workspace(300, 512, 1024)
    xs = [acts(g, M, 1024, torch.bfloat16) for M in (1, 300, 2, 40, 7, 128, 300, 1) * 4]
    ys = [ops.int8_linear(x, W, ws) for x in xs]
    for x, y in zip(xs, ys):
        assert torch.equal(y, ops.int8_linear(x, W, ops.int8_workspace(x.shape[0], 512, 1024)))


def test_a_row_does_not_depend_on_the_others():
    g = gen(10)
    x, W = acts(g, 300, 900, torch.bfloat16), ops.int8_weights(whole(g, 200, 900), scales(g, 200))
    ws = ops.int8_workspace(300, 200, 900)
    y = ops.int8_linear(x, W, ws)
    for a, b in ((0, 1), (7, 10), (100, 140), (44, 300)):
        assert torch.equal(ops.int8_linear(x[a:b], W, ws), y[a:b])


def test_no_rows():
    g = gen(11)
    W = ops.int8_weights(whole(g, 20, 64), scales(g, 20))
    assert ops.int8_linear(torch.empty(0, 64, device="cuda"), W, ops.int8_workspace(4, 20, 64)).shape == (0, 20)
    ids = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    up, down = ops.int8_weights(whole(g, 4, 32, 64), scales(g, 4, 32)), ops.int8_weights(whole(g, 4, 64, 16), scales(g, 4, 64))
    ws = ops.int8_experts_workspace(3, 2, 64, 16, 4)
    x = torch.randn(3, 64, device="cuda").bfloat16()
    assert (ops.int8_experts(x, ids, torch.rand(3, 2, device="cuda"), up, down, ws) == 0).all()
    assert ops.int8_experts(x[:0], ids[:0], torch.rand(0, 2, device="cuda"), up, down, ws).shape == (0, 64)


# long rows, whose last tiles several CTAs share: two of them, four and more, with whole tiles in front of them and without
@pytest.mark.parametrize("M,N,K", [(512, 8192, 8192), (700, 4100, 8300), (300, 19300, 16400), (40, 19100, 8257), (1300, 2100, 40000), (257, 9800, 131072),
                                   (150, 19000, 131072)])
def test_tiles_of_several_ctas(M, N, K):
    """Whole numbers of at most 63 or 20 beside activations of a scale of 1: sums stay below 2^24 (127 * 20 sqrt(131072 * 1.3) is far from it)."""
    g = gen(M + N + K)
    most = 63 if K < 20000 else 20
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wq, ws = torch.randint(-most, most + 1, (N, K), generator=g, device="cuda", dtype=torch.int8), scales(g, N)
    W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
    rows = torch.cat((torch.arange(0, M, max(1, M // 40), device="cuda"), torch.arange(M - 3, M, device="cuda")))
    q, s = R.numbers(x[rows])
    want = torch.cat([R.product(q, s, wq[n:n + 2000], ws[n:n + 2000], torch.float32) for n in range(0, N, 2000)], 1)
    y = ops.int8_linear(x, W, space)
    for _ in range(2):
        assert torch.equal(ops.int8_linear(x, W, space), y)
    assert torch.equal(y[rows], want.to(y.dtype))
    if N % 2 == 0:
        out, bound = R.gated_bound(want, torch.bfloat16)
        assert ((ops.int8_linear(x, W, space, gated=True)[rows].double() - out).abs() <= bound).all()


def test_experts_tiles_of_several_ctas():
    g = gen(12)
    E, N, K = 5, 1500, 17000
    wq, s = torch.randint(-63, 64, (E, N, K), generator=g, device="cuda", dtype=torch.int8), scales(g, E, N)
    W = ops.int8_weights(wq, s)
    for counts in ((90, 0, 300, 17, 150), (10, 9, 12, 5, 8), (0, 0, 0, 0, 400)):
        ids = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)]).int().cuda()[:, None]
        order = ops.expert_order(ids, E)
        x = torch.randn(len(ids), K, generator=g, device="cuda").half()
        y = ops.int8_matmul(ops.int8_quantize(x, order), W, torch.float32, ops.int8_workspace(len(ids), N, K))
        for e in range(E):
            t = torch.nonzero(ids[:, 0] == e)[:, 0]
            if len(t):
                assert torch.equal(y[order.inv[t, 0].long()], R.product(*R.numbers(x[t]), wq[e], s[e], torch.float32)), (counts, e)
