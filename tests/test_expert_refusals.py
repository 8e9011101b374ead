"""Refusals of the rows between tokens and experts and of the 8-bit products.  Everything is refused before a launch, so the C calls need no
GPU: the addresses they get are never read."""
import ctypes

import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

INVALID, SHAPE, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_WORKSPACE
P = 4096  # an address on 16 bytes
BF16, F32 = B.MOE_BF16, B.MOE_F32


@pytest.fixture(scope="module")
def lib():
    return B.load()


def sweep(call, cases):
    """Each case is one argument's change and the status it gives."""
    for change, status in cases:
        assert call(**change) == status, change


def test_order(lib):
    def call(ids=P, T=4, k=2, E=8, offsets=P, inv=P):
        return lib.moe_expert_order(ids, T, k, E, offsets, inv, None)
    sweep(call, [({"k": 0}, SHAPE), ({"k": 33}, SHAPE), ({"E": 0}, SHAPE), ({"E": 1025}, SHAPE), ({"T": -1}, SHAPE),
                 ({"T": 2 ** 30, "k": 2}, SHAPE), ({"ids": None}, INVALID), ({"offsets": None}, INVALID), ({"inv": None}, INVALID),
                 ({"T": 0, "offsets": None}, INVALID)])
    for name in ("ids", "offsets", "inv"):
        for off in (1, 2, 3):
            assert call(**{name: P + off}) == INVALID, (name, off)


@pytest.mark.parametrize("dtype,odd", [(BF16, 1), (B.MOE_F16, 1), (F32, 2)])
def test_rows(lib, dtype, odd):
    def there(a=P, ld=64, inv=P, w=P, T=4, k=2, d=64, out=P, ldo=64, dtype=dtype):
        return lib.moe_tokens_to_experts(a, dtype, ld, inv, w, T, k, d, out, ldo, None)

    def back(a=P, ld=64, inv=P, w=P, T=4, k=2, d=64, out=P, ldo=64, dtype=dtype):
        return lib.moe_experts_to_tokens(a, dtype, ld, inv, w, T, k, d, out, ldo, None)
    shapes = [({"k": 0}, SHAPE), ({"k": 33}, SHAPE), ({"T": -1}, SHAPE), ({"d": 0}, SHAPE), ({"T": 2 ** 30, "k": 2}, SHAPE),
              ({"T": 2 ** 24, "k": 32, "d": 2 ** 14}, SHAPE), ({"ld": 63}, SHAPE), ({"dtype": 99}, INVALID), ({"inv": None}, INVALID),
              ({"inv": P + 2}, INVALID), ({"a": None}, INVALID), ({"a": P + odd}, INVALID)]
    for call in (there, back):
        sweep(call, shapes + [({"w": P + 2}, INVALID), ({"out": None}, INVALID), ({"out": P + odd}, INVALID), ({"ldo": 63}, SHAPE)])
        assert call(T=0, a=None, inv=None, out=None) == B.MOE_OK
        assert call(T=0, dtype=99) == INVALID

    def there_back(a=P, ld=64, b=P, ldb=64, inv=P, w=P, T=4, k=2, d=64, out=P, ldo=64, dw=P, dtype=dtype):
        return lib.moe_tokens_to_experts_backward(a, dtype, ld, b, ldb, inv, w, T, k, d, out, ldo, dw, None)

    def back_back(a=P, ld=64, b=P, ldb=64, inv=P, w=P, T=4, k=2, d=64, out=P, ldo=64, dw=P, dtype=dtype):
        return lib.moe_experts_to_tokens_backward(a, dtype, ld, b, ldb, inv, w, T, k, d, out, ldo, dw, None)
    for call in (there_back, back_back):
        sweep(call, shapes + [({"out": None, "dw": None}, INVALID), ({"b": None}, INVALID), ({"b": P + odd}, INVALID), ({"ldb": 63}, SHAPE),
                              ({"dw": P + 1}, INVALID), ({"w": P + 1}, INVALID), ({"out": P + odd}, INVALID), ({"ldo": 63}, SHAPE)])


def weights(q=P, s=P):
    return ctypes.byref(B.moe_int8_weights(q, s))


def rows(q=P, s=P, room=1024):
    return ctypes.byref(B.moe_int8_rows(q, s, room))


def test_sizes():
    assert B.moe_int8_weights_bytes(128, 64) == 8192 and B.moe_int8_weights_bytes(129, 65) == 4 * 8192
    for N, K in ((-1, 64), (64, 0), (64, 131073), (2 ** 40, 64)):
        assert B.moe_int8_weights_bytes(N, K) == 0, (N, K)
    assert B.moe_int8_rows_room(0, 0) >= 0 and B.moe_int8_rows_room(9, 0) == 32 and B.moe_int8_rows_room(9, 4) == 64
    for M, E in ((-1, 0), (4, -1), (4, 1025), (2 ** 40, 0)):
        assert B.moe_int8_rows_room(M, E) == 0, (M, E)
    assert B.moe_int8_rows_bytes(32, 65) == 32 * 128 * 2 and B.moe_int8_rows_bytes(32, 131073) == 0
    assert B.moe_int8_workspace_size(4, 64, 131073) == 0 and B.moe_int8_workspace_size(-1, 64, 64) == 0
    assert B.moe_int8_workspace_size(4, 64, 64) < B.moe_int8_workspace_size(400, 64, 640)
    good = dict(T=4, d=64, E=8, k=2, I=32, dtype=BF16)
    assert B.moe_int8_experts_workspace_size(*good.values()) > 0
    for bad in ({"T": -1}, {"d": 0}, {"d": 131073}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 33}, {"I": 0}, {"I": 131073}, {"dtype": 99},
                {"T": 2 ** 30}):
        assert B.moe_int8_experts_workspace_size(*{**good, **bad}.values()) == 0, bad


def test_weights(lib):
    def layout(w=P, s=P, E=2, n=32, K=64, ld=64, first=0, step=1, N=32, W=weights()):
        return lib.moe_int8_weights_layout(w, s, E, n, K, ld, first, step, N, W, None)

    def quantize(w=P, dtype=BF16, E=2, n=32, K=64, ld=64, first=0, step=1, N=32, W=weights()):
        return lib.moe_int8_weights_quantize(w, dtype, E, n, K, ld, first, step, N, W, None)
    for call in (layout, quantize):
        sweep(call, [({"E": -1}, SHAPE), ({"E": 1025}, SHAPE), ({"n": -1}, SHAPE), ({"n": 33}, SHAPE), ({"K": 0}, SHAPE), ({"K": 131073}, SHAPE),
                     ({"ld": 63}, SHAPE), ({"first": 1}, SHAPE), ({"first": -1}, SHAPE), ({"step": 0}, SHAPE), ({"step": 2}, SHAPE),
                     ({"step": 2 ** 40}, SHAPE), ({"w": None}, INVALID), ({"W": None}, INVALID), ({"W": weights(q=P + 8)}, INVALID),
                     ({"W": weights(s=P + 2)}, INVALID), ({"W": weights(q=None)}, INVALID), ({"W": weights(s=None)}, INVALID),
                     ({"E": 0, "w": None}, B.MOE_OK)])
    sweep(layout, [({"s": None}, INVALID), ({"s": P + 2}, INVALID)])
    sweep(quantize, [({"dtype": 99}, INVALID), ({"w": P + 1}, INVALID)])


def test_quantize(lib):
    def call(x=P, dtype=BF16, T=4, K=64, ldx=64, inv=P, k=2, offsets=P, E=8, r=rows()):
        return lib.moe_int8_quantize(x, dtype, T, K, ldx, inv, k, offsets, E, r, None)
    sweep(call, [({"dtype": 99}, INVALID), ({"offsets": None}, INVALID), ({"inv": None, "offsets": None}, INVALID), ({"E": 0}, INVALID),
                 ({"E": 1025}, INVALID), ({"k": 0}, SHAPE), ({"k": 33}, SHAPE), ({"T": -1}, SHAPE), ({"T": 2 ** 62}, SHAPE), ({"K": 0}, SHAPE),
                 ({"K": 131073}, SHAPE), ({"ldx": 63}, SHAPE), ({"x": None}, INVALID), ({"x": P + 1}, INVALID), ({"inv": P + 2}, INVALID),
                 ({"offsets": P + 2}, INVALID), ({"r": None}, INVALID), ({"r": rows(q=P + 8)}, INVALID), ({"r": rows(s=P + 2)}, INVALID),
                 ({"r": rows(room=80)}, SHAPE), ({"r": rows(room=100)}, SHAPE), ({"T": 0, "x": None}, B.MOE_OK)])


def test_products(lib):
    plenty = 1 << 40

    def matmul(r=rows(), offsets=P, E=8, M=4, W=weights(), N=32, K=64, gated=0, y=P, dtype=BF16, ldy=32, ws=P, ws_bytes=plenty):
        return lib.moe_int8_matmul(r, offsets, E, M, W, N, K, gated, y, dtype, ldy, ws, ws_bytes, None)

    def linear(x=P, x_dtype=F32, M=4, K=64, ldx=64, W=weights(), N=32, gated=0, y=P, dtype=BF16, ldy=32, ws=P, ws_bytes=plenty):
        return lib.moe_int8_linear(x, x_dtype, M, K, ldx, W, N, gated, y, dtype, ldy, ws, ws_bytes, None)
    for call in (matmul, linear):
        sweep(call, [({"M": -1}, SHAPE), ({"N": -1}, SHAPE), ({"K": 0}, SHAPE), ({"K": 131073}, SHAPE), ({"gated": 1, "N": 31}, SHAPE),
                     ({"y": None}, INVALID), ({"y": P + 1}, INVALID), ({"dtype": 99}, INVALID), ({"W": None}, INVALID),
                     ({"W": weights(q=P + 8)}, INVALID), ({"W": weights(s=P + 1)}, INVALID), ({"ws": None}, WS)])
        sweep(call, [({"ldy": 31}, SHAPE), ({"ws_bytes": 64}, WS), ({"ws": P + 1}, WS)])
        assert call(M=0, y=None, ws=None) == B.MOE_OK and call(N=0, y=None, ws=None, ldy=0) == B.MOE_OK
    sweep(matmul, [({"offsets": None}, INVALID), ({"E": 0}, INVALID), ({"E": 1025}, INVALID), ({"offsets": P + 2}, INVALID), ({"r": None}, INVALID),
                   ({"r": rows(room=80)}, SHAPE), ({"r": rows(q=P + 8)}, INVALID)])
    sweep(linear, [({"x": None}, INVALID), ({"x": P + 2}, INVALID), ({"ldx": 63}, SHAPE), ({"x_dtype": 99}, INVALID)])
    size = B.moe_int8_workspace_size(4, 32, 64)
    assert linear(ws_bytes=size - 1) == WS


def test_sparse_layer(lib):
    def call(x=P, dtype=BF16, ldx=64, ids=P, w=P, T=4, d=64, E=8, k=2, I=32, up=weights(), down=weights(), y=P, ldy=64, ws=P,  # noqa: E741
             ws_bytes=1 << 40):
        return lib.moe_int8_experts(x, dtype, ldx, ids, w, T, d, E, k, I, up, down, y, ldy, ws, ws_bytes, None)
    sweep(call, [({"T": -1}, SHAPE), ({"d": 0}, SHAPE), ({"E": 0}, SHAPE), ({"E": 1025}, SHAPE), ({"k": 0}, SHAPE), ({"k": 33}, SHAPE),
                 ({"I": 0}, SHAPE), ({"ldx": 63}, SHAPE), ({"ldy": 63}, SHAPE), ({"dtype": 99}, INVALID), ({"x": None}, INVALID),
                 ({"x": P + 1}, INVALID), ({"ids": None}, INVALID), ({"ids": P + 2}, INVALID), ({"w": None}, INVALID), ({"w": P + 2}, INVALID),
                 ({"up": None}, INVALID), ({"up": weights(q=P + 4)}, INVALID), ({"down": None}, INVALID), ({"down": weights(s=None)}, INVALID),
                 ({"y": None}, INVALID), ({"y": P + 1}, INVALID), ({"ws": None}, WS), ({"ws": P + 1}, WS),
                 ({"T": 0, "x": None, "ids": None}, B.MOE_OK)])
    size = B.moe_int8_experts_workspace_size(4, 64, 8, 2, 32, BF16)
    assert call(ws_bytes=size - 1) == WS


class Elsewhere(torch.Tensor):
    """A tensor without memory that says which device it is on."""
    __torch_dispatch__ = None


def refused_elsewhere():
    device = torch.device("cuda", torch.cuda.current_device() + 1 if torch.cuda.is_available() else 1)

    def new(*shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(Elsewhere, shape, dtype=dtype, device=device)
    i32, u8 = torch.int32, torch.uint8
    order = ops.ExpertOrder(8, new(9, dtype=i32), new(4, 2, dtype=i32))
    W = object.__new__(ops.Int8Weights)
    W.N, W.K, W.E, W.q, W.s, W.struct = 64, 64, 8, new(8 * 8192, dtype=u8), new(8 * 64), B.moe_int8_weights(P, P)
    W.args = (W.struct, 8, 64, 64, device.index)
    r = object.__new__(ops.Int8Rows)
    r.M, r.K, r.order, r.q, r.s, r.room, r.struct = 8, 64, order, new(96 * 64, dtype=torch.float16), new(96), 96, B.moe_int8_rows(P, P, 96)
    one = object.__new__(ops.Int8Weights)
    one.struct, one.args = W.struct, (W.struct, 1, 64, 64, device.index)
    ws, x, ids, w = new(1 << 20, dtype=u8), new(4, 64), new(4, 2, dtype=i32), new(4, 2)
    calls = [lambda: ops.expert_order(ids, 8), lambda: ops.tokens_to_experts(x, order, w),
             lambda: ops.tokens_to_experts_backward(new(8, 64), order, x, w), lambda: ops.experts_to_tokens(new(8, 64), order, w),
             lambda: ops.experts_to_tokens_backward(x, order, new(8, 64), w), lambda: ops.int8_quantize(x),
             lambda: ops.int8_quantize(x, order), lambda: ops.int8_matmul(r, W, torch.float32, ws), lambda: ops.int8_linear(x, one, ws),
             lambda: ops.int8_experts(x, ids, w, W, W, ws)]
    if torch.cuda.is_available():  # (the Python-level checks ask torch for the current device)
        calls += [lambda: ops.int8_weights(new(64, 64)), lambda: ops.int8_workspace(4, 64, 64, device),
                  lambda: ops.int8_experts_workspace(4, 2, 64, 32, 8, device=device)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="another device than the current one"):
            call()
            pytest.fail("call %d" % i)


def test_tensors_of_another_device_are_refused():
    refused_elsewhere()


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused_beside_a_gpu():
    refused_elsewhere()


def test_tensors_of_the_host_are_refused():
    x, ids = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    order = ops.ExpertOrder(8, torch.zeros(9, dtype=torch.int32), ids)
    for call in (lambda: ops.expert_order(ids, 8), lambda: ops.tokens_to_experts(x, order), lambda: ops.int8_quantize(x),
                 lambda: ops.experts_to_tokens(x, order), lambda: ops.int8_weights(x), lambda: ops.Int8Weights(64, 64, x, x),
                 lambda: ops.tokens_to_experts_backward(x, order), lambda: ops.experts_to_tokens_backward(x, order)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_torch_level_refusals():
    x, w = torch.randn(4, 64, device="cuda"), torch.rand(4, 2, device="cuda")
    ids = torch.randint(0, 8, (4, 2), device="cuda", dtype=torch.int32)
    order, rows_ = ops.expert_order(ids, 8), torch.randn(8, 64, device="cuda")
    W, one = ops.int8_weights(torch.randn(8, 64, 64, device="cuda")), ops.int8_weights(torch.randn(40, 64, device="cuda"))
    up, down = ops.int8_weights(torch.randn(8, 32, 64, device="cuda"), up=torch.randn(8, 32, 64, device="cuda")), \
        ops.int8_weights(torch.randn(8, 64, 32, device="cuda"))
    ws, space = ops.int8_workspace(8, 64, 64), ops.int8_experts_workspace(4, 2, 64, 32, 8, torch.float32)
    q8 = torch.zeros(8, 64, dtype=torch.int8, device="cuda")
    bad = [lambda: ops.expert_order(ids.long(), 8), lambda: ops.expert_order(ids[:, :1], 8), lambda: ops.expert_order(ids, 0),
           lambda: ops.expert_order(ids.view(-1), 8), lambda: ops.tokens_to_experts(x[:3], order), lambda: ops.tokens_to_experts(x.t(), order),
           lambda: ops.tokens_to_experts(x, order, w[:, :1]), lambda: ops.tokens_to_experts(x, order, w.double()),
           lambda: ops.tokens_to_experts(x, order, out=rows_.half()), lambda: ops.tokens_to_experts(x, order, out=rows_[:7]),
           lambda: ops.tokens_to_experts(x[:1].expand(4, 64), order), lambda: ops.experts_to_tokens(rows_[:7], order, w),
           lambda: ops.experts_to_tokens(rows_, order, w.t()), lambda: ops.experts_to_tokens(rows_, order, out=x.bfloat16()),
           lambda: ops.tokens_to_experts_backward(rows_, order, x.half(), w), lambda: ops.tokens_to_experts_backward(rows_[:5], order),
           lambda: ops.experts_to_tokens_backward(x, order, rows_[:, :60], w), lambda: ops.experts_to_tokens_backward(rows_, order),
           lambda: ops.int8_quantize(x[:3], order), lambda: ops.int8_quantize(x, order, ordered=True), lambda: ops.int8_quantize(x.t()),
           lambda: ops.int8_weights(q8), lambda: ops.int8_weights(q8, torch.ones(7, device="cuda")),
           lambda: ops.int8_weights(x, torch.ones(4, device="cuda")), lambda: ops.int8_weights(x, up=x[:3]),
           lambda: ops.int8_weights(x, up_scales=torch.ones(4, device="cuda")), lambda: ops.int8_weights(x.t()),
           lambda: ops.int8_weights(x.double()), lambda: ops.int8_weights(x[:0]),
           lambda: ops.Int8Weights(64, 64, W.q[:-1], W.s), lambda: ops.Int8Weights(64, 64, W.q, W.s[:-1]),
           lambda: ops.int8_matmul(ops.int8_quantize(x), W, torch.float32, ws), lambda: ops.int8_matmul(ops.int8_quantize(x, order), one, torch.float32, ws),
           lambda: ops.int8_matmul(ops.int8_quantize(x[:, :63]), one, torch.float32, ws),
           lambda: ops.int8_matmul(ops.int8_quantize(x), one, torch.float32, ws, out=torch.empty(4, 40, device="cuda").half()),
           lambda: ops.int8_linear(x, W, ws), lambda: ops.int8_linear(x[:, :63], one, ws), lambda: ops.int8_linear(x, one, ws[1::2]),
           lambda: ops.int8_linear(x, one, ws, out=torch.empty(4, 39, device="cuda")),
           lambda: ops.int8_linear(x, ops.int8_weights(torch.randn(5, 64, device="cuda")), ws, gated=True),
           lambda: ops.int8_workspace(4, 64, 0), lambda: ops.int8_experts_workspace(4, 33, 64, 32, 8),
           lambda: ops.int8_experts(x, ids, w, down, up, space), lambda: ops.int8_experts(x, ids[:3], w, up, down, space),
           lambda: ops.int8_experts(x, ids.long(), w, up, down, space), lambda: ops.int8_experts(x, ids, w.half(), up, down, space),
           lambda: ops.int8_experts(x, ids, w, up, down, space, out=x.half())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d" % i)
    for call in (lambda: ops.tokens_to_experts(x.long(), order), lambda: ops.int8_linear(x.double(), one, ws),
                 lambda: ops.int8_matmul(ops.int8_quantize(x), one, torch.int32, ws), lambda: ops.int8_quantize(x.int())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ops.expert_order(ids, 8) and ops.expert_order(ids.expand(4, 2).repeat(1, 17), 8), lambda: ops.int8_linear(x, one, ws[:4096]),
                 lambda: ops.int8_experts(x, ids, w, up, down, space[:-256])):
        with pytest.raises(B.MoeError):
            call()


@pytest.mark.gpu
def test_modules_refuse_what_they_were_not_built_for():
    from bit_expert_ffn_moe_gb300.block import Int8Experts, Int8Linear
    up, down = ops.int8_weights(torch.randn(8, 32, 64, device="cuda"), up=torch.randn(8, 32, 64, device="cuda")), \
        ops.int8_weights(torch.randn(8, 64, 32, device="cuda"))
    layer = Int8Experts(up, down, 4, 2)
    x, w = torch.randn(5, 64, device="cuda").bfloat16(), torch.rand(5, 2, device="cuda")
    ids = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: layer(x, ids, w), lambda: layer(x[:4], ids[:4, :1].contiguous(), w[:4]), lambda: layer.outputs(x, ids),
                 lambda: Int8Experts(down, up, 4, 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.MoeError):  # (a workspace for two-byte types)
        layer(x[:4].float(), ids[:4], w[:4])
    linear = Int8Linear(torch.randn(32, 640, device="cuda"), 4)
    with pytest.raises(B.MoeError):
        linear(torch.randn(400, 640, device="cuda"))
