"""Order by expert, rows between tokens and experts, and their gradients, against plain forms.  Copies and single products are equal bit
for bit.  A sum of k products: k roundings of 2^-24 of the sum of the magnitudes, and half a step of the type.  dw: the longest serial
chain of an fp32 dot product has d / 32 + 8 terms, then a tree: (d / 32 + 24) 2^-24 of the sum of the magnitudes."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("kind", ["distinct", "any", "dropped"])
@pytest.mark.parametrize("T,k,E", [(0, 3, 5), (1, 1, 1), (1, 8, 128), (7, 3, 5), (33, 2, 1024), (100, 8, 129), (700, 3, 40), (683, 3, 33),
                                   (3000, 4, 1000), (20000, 2, 6)])
def test_order(T, k, E, kind):
    if kind == "distinct" and k > E:
        kind = "any"
    ids = R.some_ids(T, k, E, 11, kind)
    o = ops.expert_order(ids.cuda(), E)
    flat = ids.reshape(-1).long()
    has = (flat >= 0) & (flat < E)
    place = torch.where(has, flat, E).sort(stable=True).indices
    inv = torch.full((T * k,), -1)
    inv[place[:int(has.sum())]] = torch.arange(int(has.sum()))
    ends = torch.bincount(flat[has], minlength=E).cumsum(0)
    assert o.offsets.tolist() == [0] + ends.tolist()
    assert torch.equal(o.inv.cpu().long(), inv.view(T, k))
    if T * k < 1000:
        offsets, want = R.order(ids.tolist(), E)
        assert o.offsets.tolist() == offsets and o.inv.tolist() == want


def given(T, k, d, dtype, kind="distinct", seed=0, pad=0, E=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = E or max(k, 6)

    def rows(n):
        return torch.randn(n, d + pad, generator=g, device="cuda").to(dtype)[:, :d]
    order = ops.expert_order(R.some_ids(T, k, E, seed, kind).cuda(), E)
    return order, rows(T), rows(T * k), torch.randn(T, k, generator=g, device="cuda")


def at(order):
    """Flat rows of the pairs (those without one: 0) and which have one."""
    inv = order.inv.reshape(-1).long()
    return inv.clamp(min=0), inv >= 0


SHAPES = [(1, 1, 1), (1, 8, 8192), (3, 5, 128), (9, 2, 264), (17, 9, 521), (5, 32, 1032), (333, 5, 2055), (70, 8, 2048), (1000, 1, 64), (64, 17, 771),
          (2, 3, 20000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["distinct", "dropped"])
@pytest.mark.parametrize("T,k,d", SHAPES)
def test_rows_and_back(T, k, d, kind, dtype):
    order, x, rows, w = given(T, k, d, dtype, kind, T + d)
    i, has = at(order)
    token = torch.arange(T * k, device="cuda") // k
    for weights in (None, w):
        out = torch.full((T * k, d), 7.0, device="cuda", dtype=dtype)
        assert ops.tokens_to_experts(x, order, weights, out).data_ptr() == out.data_ptr()
        want = torch.full_like(out, 7.0)
        want[i[has]] = (x[token] if weights is None else (w.reshape(-1, 1) * x[token].float()).to(dtype))[has]
        assert torch.equal(out, want)
        y = ops.experts_to_tokens(rows, order, weights)
        part = torch.where(has[:, None], rows[i].double(), 0.0) * (1.0 if weights is None else w.double().reshape(-1, 1))
        part = part.view(T, k, d)
        err = (y.double() - part.sum(1)).abs()
        bound = (k + 1) * 2.0 ** -24 * part.abs().sum(1) + torch.finfo(dtype).eps / 2 * part.sum(1).abs() * 1.01
        assert (err <= bound + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["distinct", "dropped"])
@pytest.mark.parametrize("T,k,d", SHAPES)
def test_gradients(T, k, d, kind, dtype):
    order, x, rows, w = given(T, k, d, dtype, kind, T + d + 1)
    i, has = at(order)
    prod = x.double()[:, None, :] * torch.where(has[:, None], rows[i].double(), 0.0).view(T, k, d)
    bound = (d / 32 + 24) * 2.0 ** -24 * prod.abs().sum(2)
    # both ways have the same dw, of x and the rows' gradient or of dy and the rows; the rest is the other way's map
    for weights in (None, w):
        drows, dw = ops.experts_to_tokens_backward(x, order, rows, weights)
        want = ops.tokens_to_experts(x, order, weights)
        assert torch.equal(drows[i[has]], want[i[has]])
        dx, dw2 = ops.tokens_to_experts_backward(rows, order, x, weights)
        assert torch.equal(dx, ops.experts_to_tokens(rows, order, weights))
        assert (dw is None) == (dw2 is None) == (weights is None)
        if weights is None:
            continue
        for got in (dw, dw2):
            assert ((got.double() - prod.sum(2)).abs() <= bound).all()
        none, dw3 = ops.experts_to_tokens_backward(x, order, rows, w, need_drows=False)
        none2, dw4 = ops.tokens_to_experts_backward(rows, order, x, w, need_dx=False)
        assert none is None and none2 is None and torch.equal(dw3, dw) and torch.equal(dw4, dw2)
        drows5, none3 = ops.experts_to_tokens_backward(x, order, None, w)
        dx5, none4 = ops.tokens_to_experts_backward(rows, order, None, w)
        assert none3 is None and none4 is None and torch.equal(drows5[i[has]], drows[i[has]]) and torch.equal(dx5, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 0), (8, 1), (0, 3)])
def test_strides_and_addresses(dtype, pad, shift):
    """Rows further apart than they are wide, and matrices that start on any element: the same bits as contiguous ones."""
    T, k, d = 37, 4, 328
    order, x, rows, w = given(T, k, d, dtype, "dropped", 3)
    i, has = at(order)

    def odd(m, n):
        room = torch.zeros(n * (d + pad) + shift, device="cuda", dtype=dtype)[shift:].view(n, d + pad)[:, :d]
        if m is not None:
            room.copy_(m)
        return room
    xo, ro = odd(x, T), odd(rows, T * k)
    out = ops.tokens_to_experts(xo, order, w, odd(None, T * k))
    assert torch.equal(out[i[has]], ops.tokens_to_experts(x, order, w)[i[has]])
    assert torch.equal(ops.experts_to_tokens(ro, order, w, odd(None, T)), ops.experts_to_tokens(rows, order, w))
    drows, dw = ops.experts_to_tokens_backward(xo, order, ro, w)
    dx, dw2 = ops.tokens_to_experts_backward(ro, order, xo, w)
    assert torch.equal(dx, ops.experts_to_tokens(rows, order, w)) and torch.equal(drows[i[has]], out[i[has]])
    prod = x.double()[:, None, :] * torch.where(has[:, None], rows[i].double(), 0.0).view(T, k, d)
    for got in (dw, dw2):
        assert ((got.double() - prod.sum(2)).abs() <= (d / 32 + 24) * 2.0 ** -24 * prod.abs().sum(2)).all()


def test_gradients_against_differences():
    """y = sum_j w rows is linear in each of rows, w; rows = w x in each of w, x: central differences of the 64-bit forms."""
    T, k, d = 5, 3, 40
    order, x, rows, w = given(T, k, d, torch.float32, "any", 4, E=6)
    i, _ = at(order)
    token = torch.arange(T * k, device="cuda") // k
    dy, drows = torch.randn_like(x), torch.randn_like(rows)

    def back(rows, w):
        return (dy.double() * (w.reshape(-1, 1) * rows[i]).view(T, k, d).sum(1)).sum()

    def there(x, w):
        return (drows.double()[i] * (w.reshape(-1, 1) * x[token])).sum()
    g_rows, g_w = ops.experts_to_tokens_backward(dy, order, rows, w)
    g_x, g_w2 = ops.tokens_to_experts_backward(drows, order, x, w)
    for f, at_, other, grad, first in ((back, rows, w, g_rows, True), (back, w, rows, g_w, False), (there, x, w, g_x, True),
                                       (there, w, x, g_w2, False)):
        step = torch.randn(at_.shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64).cuda()
        a, b = at_.double() + step, at_.double() - step
        o = other.double()
        diff = (f(a, o) - f(b, o) if first else f(o, a) - f(o, b)) / 2
        want = (grad.double() * step).sum()
        # fp32 results of at most 64 terms each, summed over all entries
        assert abs(diff - want) <= 64 * 2.0 ** -24 * (grad.double() * step).abs().sum() + 1e-4


def test_infinities_and_nan_stay_where_they_are():
    T, k, d = 6, 2, 64
    order, x, rows, w = given(T, k, d, torch.bfloat16, "distinct", 5)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    out = ops.tokens_to_experts(x, order)
    assert torch.equal(torch.isnan(out).nonzero()[:, 1], torch.tensor([3, 3], device="cuda"))
    assert int(torch.isinf(out).sum()) == 2
    rows[order.inv[4, 1].long(), 7] = float("nan")
    y = ops.experts_to_tokens(rows, order, w)
    assert torch.isnan(y).nonzero().tolist() == [[4, 7]]


def test_in_a_graph_and_on_another_stream():
    T, k, d = 50, 3, 512
    order, x, rows, w = given(T, k, d, torch.bfloat16, "distinct", 6)
    ids = R.some_ids(T, k, 6, 6).cuda()

    def all_of_it():
        o = ops.expert_order(ids, 6)
        r = ops.tokens_to_experts(x, o, w)
        return (r, ops.experts_to_tokens(r, o, w), *ops.experts_to_tokens_backward(x, o, r, w), *ops.tokens_to_experts_backward(r, o, x, w))
    plain = all_of_it()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        aside = all_of_it()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_of_it()
    keep = x.clone()
    x.mul_(2.0)
    graph.replay()
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(plain, aside, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_no_tokens_and_no_experts():
    order = ops.expert_order(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4)
    assert order.offsets.tolist() == [0] * 5
    x = torch.empty(0, 64, device="cuda")
    assert ops.tokens_to_experts(x, order).shape == (0, 64) and ops.experts_to_tokens(x, order).shape == (0, 64)
    none = ops.expert_order(torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), 4)
    rows = torch.randn(10, 64, device="cuda")
    assert (ops.experts_to_tokens(rows, none) == 0).all()
    dx, dw = ops.tokens_to_experts_backward(rows, none, torch.randn(5, 64, device="cuda"), torch.randn(5, 2, device="cuda"))
    assert (dx == 0).all() and (dw == 0).all()
