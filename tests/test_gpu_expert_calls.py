"""Calls of the rows between tokens and experts and of the 8-bit products as programs make them: beside autograd, captured, on several
streams, with one workspace for several operators, beyond 32-bit offsets, and in the example."""
import os
import sys

import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops
from bit_expert_ffn_moe_gb300.block import Int8Experts, Int8Linear

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-4


def experts(g, E, d, I):  # noqa: E741
    up = ops.int8_weights(whole(g, E, I, d), scales(g, E, I), whole(g, E, I, d), scales(g, E, I))
    return up, ops.int8_weights(whole(g, E, d, I), scales(g, E, d))


def routing(T, k, E, seed, kind="any"):
    return R.some_ids(T, k, E, seed, kind).cuda(), torch.rand(T, k, generator=gen(seed), device="cuda")


def forms():
    """Name, input, and the differentiable result of it."""
    g = gen(0)
    ids, w = routing(6, 3, 8, 1)
    order = ops.expert_order(ids, 8)
    x, rows = torch.randn(6, 64, generator=g, device="cuda"), torch.randn(18, 64, generator=g, device="cuda")
    W, (up, down) = ops.int8_weights(whole(g, 40, 64), scales(g, 40)), experts(g, 8, 64, 32)
    ws, space = ops.int8_workspace(6, 40, 64), ops.int8_experts_workspace(6, 3, 64, 32, 8, torch.float32)
    linear, layer = Int8Linear(torch.randn(40, 64, generator=g, device="cuda"), 6), Int8Experts(up, down, 6, 3, torch.float32)
    yield "rows of x", x, lambda t: ops.tokens_to_experts(t, order, w)
    yield "rows of w", w, lambda t: ops.tokens_to_experts(x, order, t)
    yield "tokens of rows", rows, lambda t: ops.experts_to_tokens(t, order, w)
    yield "tokens of w", w, lambda t: ops.experts_to_tokens(rows, order, t)
    yield "linear", x, lambda t: ops.int8_linear(t, W, ws)
    yield "experts of x", x, lambda t: ops.int8_experts(t, ids, w, up, down, space)
    yield "experts of w", w, lambda t: ops.int8_experts(x, ids, t, up, down, space)
    yield "Int8Linear", x, linear
    yield "Int8Experts", w, lambda t: layer(x, ids, t)


def test_backward_is_an_error_where_a_gradient_would_be_lost():
    for name, x, f in forms():
        plain = f(x)
        assert not plain.requires_grad, name
        leaf = x.clone().requires_grad_(True)
        with torch.no_grad():
            assert not f(leaf).requires_grad, name
        y = f(leaf)
        assert torch.equal(y, plain), name
        with pytest.raises(RuntimeError, match="no autograd formula"):
            (leaf.sum() + y.sum()).backward()
        assert leaf.grad is None, name


def test_results_in_given_tensors_stay_what_they_are():
    ids, w = routing(6, 3, 8, 1, "distinct")
    order = ops.expert_order(ids, 8)
    x = torch.randn(6, 64, device="cuda", requires_grad=True)
    g = gen(2)
    up, down = experts(g, 8, 64, 32)
    for out, call in ((torch.empty(18, 64, device="cuda"), lambda o: ops.tokens_to_experts(x, order, w, o)),
                      (torch.empty(6, 64, device="cuda"), lambda o: ops.experts_to_tokens(x.repeat(3, 1), order, w, o)),
                      (torch.empty(6, 40, device="cuda"),
                       lambda o: ops.int8_linear(x, ops.int8_weights(whole(g, 40, 64), scales(g, 40)), ops.int8_workspace(6, 40, 64), out=o)),
                      (torch.empty(6, 64, device="cuda"), lambda o: ops.int8_experts(
                          x, ids, w, up, down, ops.int8_experts_workspace(6, 3, 64, 32, 8, torch.float32), o))):
        y = call(out)
        assert y.data_ptr() == out.data_ptr() and not y.requires_grad and not out.requires_grad


def test_gradients_are_captured_beside_a_living_autograd_graph():
    """The gradient calls know nothing of autograd: captured while a graph of the same leaves lives, they replay what they compute."""
    ids, w0 = routing(50, 3, 8, 4, "dropped")
    order = ops.expert_order(ids, 8)
    w = w0.clone().requires_grad_(True)
    x = torch.randn(50, 72, device="cuda", requires_grad=True)
    alive = ops.tokens_to_experts(x, order, w).sum() + (x * x).sum()
    dy, rows = torch.randn(50, 72, device="cuda"), torch.randn(150, 72, device="cuda")
    used = order.inv.view(-1)[order.inv.view(-1) >= 0].long()

    def both():
        a, da = ops.experts_to_tokens_backward(dy, order, rows, w)
        b, db = ops.tokens_to_experts_backward(rows, order, x, w)
        return a, da, b, db
    want = both()
    assert not any(t.requires_grad for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    graph.replay()
    assert torch.equal(got[0][used], want[0][used]) and all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    with pytest.raises(RuntimeError, match="no autograd formula"):
        alive.backward()


@pytest.mark.parametrize("T,k,d,E,I", [(1, 2, 256, 16, 128), (40, 4, 320, 8, 200), (700, 2, 512, 6, 384)])
def test_the_layer_in_a_graph_with_new_inputs(T, k, d, E, I):  # noqa: E741
    g = gen(5)
    up, down = experts(g, E, d, I)
    layer = Int8Experts(up, down, T, k)
    x = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.ones(T, k, device="cuda")
    x.normal_(generator=g)
    layer(x, ids, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, ids, w)
    for seed, kind in ((6, "distinct"), (7, "dropped"), (8, "any"), (9, "distinct")):
        x.normal_(generator=g)
        new_ids, new_w = routing(T, k, E, seed, kind)
        ids.copy_(new_ids), w.copy_(new_w)
        graph.replay()
        rows, order = layer.outputs(x, ids)
        assert torch.equal(y, ops.experts_to_tokens(rows, order, w)), (seed, kind)
    assert B.moe_get_device_status(layer.workspace) == B.MOE_OK


def test_two_streams_at_once():
    """Each with its own workspace; the same weights."""
    g = gen(10)
    up, down = experts(g, 16, 512, 256)
    W = ops.int8_weights(whole(g, 4100, 512), scales(g, 4100))
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i, T in enumerate((300, 17)):
        ids, w = routing(T, 4, 16, 11 + i, "distinct")
        x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
        layer, ws = Int8Experts(up, down, T, 4), ops.int8_workspace(T, 4100, 512)
        want = (layer(x, ids, w), ops.int8_linear(x, W, ws))
        work.append((x, ids, w, layer, ws, want, []))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, (x, ids, w, layer, ws, _, got) in zip(streams, work):
            with torch.cuda.stream(stream):
                got.append((layer(x, ids, w), ops.int8_linear(x, W, ws)))
    torch.cuda.synchronize()
    for *_, want, got in work:
        assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))


def test_one_workspace_for_several_operators():
    g = gen(12)
    up, down = experts(g, 8, 256, 128)
    W = ops.int8_weights(whole(g, 3000, 256), scales(g, 3000))
    ids, w = routing(90, 3, 8, 13, "dropped")
    x = torch.randn(90, 256, generator=g, device="cuda").bfloat16()
    space = Int8Experts(up, down, 90, 3).workspace
    calls = [lambda ws: ops.int8_experts(x, ids, w, up, down, ws), lambda ws: ops.int8_linear(x, W, ws), lambda ws: ops.int8_linear(x[:1], W, ws),
             lambda ws: ops.int8_matmul(ops.int8_quantize(x), W, torch.float32, ws), lambda ws: ops.int8_experts(x[:2], ids[:2], w[:2], up, down, ws)]
    want = [f(Int8Experts(up, down, 90, 3).workspace) for f in calls]
    for i in (0, 1, 2, 3, 4, 4, 3, 1, 0, 2, 0):
        assert torch.equal(calls[i](space), want[i]), i


def test_weights_of_minus_128():
    g = gen(14)
    x = torch.randn(200, 1032, generator=g, device="cuda")
    x[0] = 1.0  # (codes of 127: with weights of -128 the largest sums that are exact)
    wq = torch.randint(-128, 128, (150, 1032), generator=g, device="cuda", dtype=torch.int8)
    wq[0] = -128
    s = scales(g, 150)
    W, ws = ops.int8_weights(wq, s), ops.int8_workspace(200, 150, 1032)
    want = R.product(*R.numbers(x), wq, s, torch.float32)
    for M in (1, 3, 40, 200):  # dot products, a cluster's tiles, the persistent kernel
        assert torch.equal(ops.int8_linear(x[:M], W, ws), want[:M])


def test_many_experts_and_slots():
    """1024 experts and 32 slots, most experts without rows, or all of them with some."""
    g = gen(15)
    gate, upper, down = whole(g, 1024, 32, 64), whole(g, 1024, 32, 64), whole(g, 1024, 64, 32)
    s1, s2, s3 = scales(g, 1024, 32), scales(g, 1024, 32), scales(g, 1024, 64)
    up, lower = ops.int8_weights(gate, s1, upper, s2), ops.int8_weights(down, s3)
    for T in (1, 30, 400):
        ids, w = routing(T, 32, 1024, 16, "distinct")
        x = torch.randn(T, 64, generator=g, device="cuda").bfloat16()
        layer = Int8Experts(up, lower, T, 32)
        y = layer(x, ids, w)
        rows, order = layer.outputs(x, ids)
        assert torch.equal(y, ops.experts_to_tokens(rows, order, w))
        h = ops.int8_matmul(ops.int8_quantize(x, order), up, torch.bfloat16, layer.workspace, gated=True)
        q, s = R.numbers(x)
        for t, j in {(0, 0), (T // 2, 13), (T - 1, 31)}:  # some pairs by the definition
            e, r = int(ids[t, j]), int(order.inv[t, j])
            one = q[t:t + 1], s[t:t + 1]
            both = torch.stack((R.product(*one, gate[e], s1[e], torch.float32), R.product(*one, upper[e], s2[e], torch.float32)), 2)
            want, bound = R.gated_bound(both.view(1, -1), torch.bfloat16)
            assert ((h[r].double() - want).abs() <= bound).all()
            assert torch.equal(rows[r:r + 1], R.product(*R.numbers(h[r:r + 1]), down[e], s3[e], torch.bfloat16))


def test_offsets_beyond_the_rows_count_as_all_of_them():
    g = gen(17)
    W, ws = ops.int8_weights(whole(g, 3, 40, 64), scales(g, 3, 40)), ops.int8_workspace(300, 40, 64)
    for M in (12, 300):  # dot products, the tensor cores
        order = ops.ExpertOrder(3, torch.tensor([0, 5, 9, M], dtype=torch.int32, device="cuda"), torch.zeros(M, 1, dtype=torch.int32, device="cuda"))
        x = torch.randn(M, 64, generator=g, device="cuda")
        rows = ops.int8_quantize(x, order, ordered=True)
        want = ops.int8_matmul(rows, W, torch.float32, ws)
        buffer = torch.full((M + 50, 40), 7.0, device="cuda")
        order.offsets[3] = M + 40
        got = ops.int8_matmul(rows, W, torch.float32, ws, out=buffer[:M])
        assert torch.equal(got, want) and (buffer[M:] == 7).all()


def test_rows_beyond_32_bits():
    """More than 2^31 elements on the longer side; the last rows and some others by the definition."""
    T, k, d = 140000, 2, 8192
    ids, w = routing(T, k, 5, 18)
    order = ops.expert_order(ids, 5)
    x = torch.randn(T, d, generator=gen(19), device="cuda").bfloat16()
    rows = ops.tokens_to_experts(x, order, w)
    some = torch.cat((order.inv.view(-1).argsort()[-400:], torch.arange(0, T * k, 997, device="cuda")))
    r, t = order.inv.view(-1)[some].long(), some // k
    assert int(r.max()) == T * k - 1
    assert torch.equal(rows[r], (x[t].float() * w.view(-1)[some][:, None]).bfloat16())
    dx, dw = ops.tokens_to_experts_backward(rows, order, x, w)
    sums = (x[t].double() * rows[r].double())
    assert ((dw.view(-1)[some].double() - sums.sum(1)).abs() <= d * 2.0 ** -24 * sums.abs().sum(1)).all()
    del sums
    last = torch.arange(T - 300, T, device="cuda")
    both = [rows[order.inv[last, j].long()].double() * w[last, j][:, None].double() for j in range(k)]
    want, size = both[0] + both[1], both[0].abs() + both[1].abs()
    for got in (dx[last], ops.experts_to_tokens(rows, order, w)[last]):  # (2 products and their sum in fp32, rounded to bf16)
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * size).all()


def by_the_definition(x, wq, s, rows, y):
    assert torch.equal(y[rows], R.product(*R.numbers(x[rows]), wq, s, y.dtype))


def test_products_beyond_32_bits():
    g = gen(20)
    M, N, K = 300000, 16, 8192  # the operand: more than 2^32 bytes
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wq, s = torch.randint(-7, 8, (N, K), generator=g, device="cuda", dtype=torch.int8), scales(g, N)  # (sums below 2^24)
    rows = torch.cat((torch.arange(0, M, 1009, device="cuda"), torch.arange(M - 200, M, device="cuda")))
    by_the_definition(x, wq, s, rows, ops.int8_linear(x, ops.int8_weights(wq, s), ops.int8_workspace(M, N, K)))
    M, N, K = 70000, 32768, 64  # the result: more than 2^31 elements
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    wq, s = whole(g, N, K), scales(g, N)
    rows = torch.cat((torch.arange(0, M, 5003, device="cuda"), torch.arange(M - 20, M, device="cuda")))
    by_the_definition(x, wq, s, rows, ops.int8_linear(x, ops.int8_weights(wq, s), ops.int8_workspace(M, N, K)))


def test_weights_beyond_32_bits():
    """Experts of more than 2^31 bytes in all."""
    g = gen(21)
    E, N, K = 36, 8192, 8192
    wq, s = torch.randint(-7, 8, (E, N, K), generator=g, device="cuda", dtype=torch.int8), scales(g, E, N)
    W = ops.int8_weights(wq, s)
    for T in (6, 200):
        ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
        ids[:3, 0] = torch.tensor([0, 17, 35], dtype=torch.int32, device="cuda")
        order = ops.expert_order(ids, E)
        x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
        y = ops.int8_matmul(ops.int8_quantize(x, order), W, torch.float32, ops.int8_workspace(T, N, K))
        for e in (0, 17, 35):
            t = torch.nonzero(ids[:, 0] == e)[:, 0]
            assert torch.equal(y[order.inv[t, 0].long()], R.product(*R.numbers(x[t]), wq[e], s[e], torch.float32))


def test_example_router_gradient_against_autograd():
    """dW_r against 64-bit autograd of the same frozen pass: choice and expert outputs held.  fp32 sums of d = 512 terms (logits, dw, the
    last product) are off by at most 2^-15 of their terms' magnitudes, which are some sqrt(512) times the sums."""
    import int8_experts as example
    layer = example.Layer(200)
    g = gen(22)
    x = torch.randn(200, layer.d, generator=g, device="cuda").bfloat16()
    dy = torch.randn(200, layer.d, generator=g, device="cuda").bfloat16()
    y, got = layer.forward_and_gradient(x, lambda y: dy)
    assert torch.equal(y, layer(x))
    _, ids, w = layer.route(x)
    rows, order = layer.experts.outputs(x, ids)
    W_r = layer.W_r.double().requires_grad_(True)
    u = torch.sigmoid(x.double() @ W_r.t()).gather(1, ids.long())
    weights = layer.rule.scale * u / u.sum(1, keepdim=True)
    out = (weights[:, :, None] * rows.double()[order.inv.long()]).sum(1)
    (out * dy.double()).sum().backward()
    assert torch.linalg.norm(got.double() - W_r.grad) <= 2.0 ** -10 * torch.linalg.norm(W_r.grad)
    # along the gradient the frozen pass changes by its square
    with torch.no_grad():
        step = 1e-6 / float(W_r.grad.norm())

        def value(m):
            u = torch.sigmoid(x.double() @ m.t()).gather(1, ids.long())
            wt = layer.rule.scale * u / u.sum(1, keepdim=True)
            return float(((wt[:, :, None] * rows.double()[order.inv.long()]).sum(1) * dy.double()).sum())
        slope = (value(W_r + step * got.double()) - value(W_r - step * got.double())) / (2 * step)
    assert abs(slope - float(W_r.grad.norm() ** 2)) <= 2.0 ** -9 * float(W_r.grad.norm() ** 2)


def test_example_runs():
    import int8_experts as example
    layer = example.Layer(64)
    x = torch.randn(64, layer.d, generator=gen(23), device="cuda").bfloat16()
    losses = example.tune(layer, x, torch.zeros_like(x), 3, 0.1)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
    assert B.moe_get_device_status(layer.experts.workspace) == B.MOE_OK


@pytest.mark.parametrize("T,k,d,E,I,kind", [(1, 8, 640, 128, 96, "distinct"), (4, 8, 300, 16, 130, "any"), (31, 1, 129, 4, 64, "dropped"),
                                            (30, 1, 256, 2, 64, "any"), (16, 2, 16500, 8, 40, "any"), (2, 4, 200, 5, 16500, "distinct"),
                                            (32, 1, 64, 1024, 7, "any"), (5, 3, 1000, 1, 33, "any")])
def test_a_few_pairs_are_the_products_of_their_parts(T, k, d, E, I, kind):  # noqa: E741
    """The layer quantises the rows of a few pairs within its products (up to 16384 values a row): the results are those of the parts."""
    g = gen(24)
    up, down = experts(g, E, d, I)
    ids, w = routing(T, k, E, 25, kind)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = torch.randn(T, d + 3, generator=g, device="cuda").to(dtype)[:, 1:d + 1]
        layer = Int8Experts(up, down, T, k, dtype)
        rows, order = layer.outputs(x, ids)
        assert torch.equal(layer(x, ids, w), ops.experts_to_tokens(rows, order, w)), dtype
