"""NVFP4 operands and their dense product.

Operands: codes, scales, padding and layout equal the oracle packer's byte for byte, each row packed as a matrix of its own.
Products: against 64-bit products of the operands' own values.  The tensor core adds 64 exact products to an fp32 accumulator per
instruction; each addition is taken to err by at most 2^-22 of the magnitudes it meets (a truncating fp32 sum errs by 2^-23), over
4 K/256 instructions; the two scalings and the store's rounding come on top.  Sums that are exact in fp32 have to come out exact."""
import numpy as np
import pytest
import torch

import ops_reference as R
from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops
from oracle import oracle as O

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def matrix(R_, C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R_, C, generator=g) * torch.exp(torch.randn(R_, 1, generator=g))
    if R_ > 2:
        x[1] = 0.0                       # a row of zeros
        x[2, 16:48] = 0.0                # blocks of zeros
    if R_ > 4 and C > 20:
        x[3] = torch.arange(C) % 7 - 3   # values on the grid: exact ties
        x[4, :20] *= 1e-3                # small blocks: subnormal scales
    return x.to(TYPES[dtype])


def oracle_rows(x):
    """Codes [rows][pad256(K)], scale bytes, row scales of the rows of x (numpy fp32)."""
    rows, K = x.shape
    Kp = -(-K // 256) * 256
    codes, scales, gs = np.zeros((rows, Kp), np.int64), np.zeros((rows, Kp // 16), np.int64), np.zeros(rows, np.float32)
    for r in range(rows):
        v = np.zeros((1, Kp), np.float32)
        v[0, :K] = x[r]
        q, s, g = O.nvfp4_pack(v)
        q = np.asarray(q).reshape(-1).astype(np.int64)
        codes[r, 0::2], codes[r, 1::2] = q & 15, q >> 4
        scales[r] = np.asarray(s).reshape(-1)
        gs[r] = np.asarray(g).reshape(-1)[0]
    return codes, scales, gs


def check_operand(op, x):
    codes, scales, gs = oracle_rows(x)
    np.testing.assert_array_equal(op.gs.cpu().numpy(), gs)
    q, s = R.operand_bytes(codes, scales)
    gq, gsb = op.q.cpu().numpy().astype(np.int64), op.s.cpu().numpy().astype(np.int64)
    np.testing.assert_array_equal(gq[q >= 0], q[q >= 0])
    np.testing.assert_array_equal(gsb[s >= 0], s[s >= 0])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R_,C", [(1, 1), (1, 16), (3, 33), (5, 256), (7, 300), (130, 544), (66, 1000), (257, 129), (2, 9000)])
def test_operands_of_a_matrix_and_its_transpose(dtype, R_, C):
    x = matrix(R_, C, dtype, R_ * C)
    host = x.float().numpy()
    dev = x.cuda()
    ws = ops.nvfp4_workspace(R_, C, C)
    rows, cols, rows2, cols2 = (ops.nvfp4_operand(*s) for s in ((R_, C), (C, R_), (R_, C), (C, R_)))
    ops.nvfp4_quantize(dev, rows)
    ops.nvfp4_quantize(dev, None, cols, ws)
    ops.nvfp4_quantize(dev, rows2, cols2, ws)
    check_operand(rows, host)
    check_operand(cols, np.ascontiguousarray(host.T))
    check_operand(rows2, host)
    check_operand(cols2, np.ascontiguousarray(host.T))
    # the values are those of the packed bytes
    codes, scales, gs = oracle_rows(host)
    v = rows.values().cpu().numpy()
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float32)
    e4m3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    want = (grid[codes % 8] * (1 - 2 * (codes // 8))).astype(np.float32) * np.repeat(e4m3[scales], 16, axis=1) * gs[:, None]
    np.testing.assert_array_equal(v, want[:, :C].astype(np.float32))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_operands_of_strided_and_unaligned_rows(dtype):
    whole = matrix(40, 700, dtype, 3).cuda()
    for view in (whole[:, 1:600], whole[3:, 8:520], whole[::2, :512], whole[:1, 5:]):
        r, c = ops.nvfp4_operand(*view.shape), ops.nvfp4_operand(view.shape[1], view.shape[0])
        ops.nvfp4_quantize(view, r, c, ops.nvfp4_workspace(view.shape[0], view.shape[1], 1))
        host = view.float().cpu().numpy()
        check_operand(r, host)
        check_operand(c, np.ascontiguousarray(host.T))


def test_given_scales_saturate():
    x = matrix(6, 300, "fp32", 4)
    x[0, 7], x[0, 8], x[5, 0] = 1e30, -1e30, float("inf")
    for n in (1, 6):
        op, opt = ops.nvfp4_operand(6, 300), ops.nvfp4_operand(300, 6)
        op.gs = torch.full((n,), 2.0 ** -9, device="cuda")
        op.struct.gs, op.struct.gs_rows = op.gs.data_ptr(), int(n == 6)
        opt.gs.fill_(2.0 ** -9)
        ops.nvfp4_quantize(x.cuda(), op, opt, scales_given=True)
        for v in (op.values().cpu(), opt.values().cpu().T):
            top = 6 * 448 * 2.0 ** -9
            assert v[0, 7] == top and v[0, 8] == -top and v[5, 0] == top
            keep = x.abs() <= top
            keep[0, :16] = False
            keep[5, :16] = False
            blocks = torch.nn.functional.pad(x, (0, 4)).view(6, -1, 16).abs().amax(2).repeat_interleave(16, 1)[:, :300]
            ok = keep & (blocks <= top)
        # within half a step of the coarsest grid spacing (2 of 6) and the scale's rounding (2^-4)
        assert ((op.values().cpu() - x).abs()[ok] <= (1 / 6 + 2.0 ** -4) * blocks[ok] + 2.0 ** -9 * 2.0 ** -9 * 6).all()


@pytest.mark.parametrize("scale", [1e-36, 1e-20, 1e20, 1e35])
def test_far_scales_take_the_division(scale):
    x = matrix(9, 64, "fp32", 6) * scale
    op = ops.nvfp4_operand(9, 64)
    ops.nvfp4_quantize(x.cuda(), op)
    check_operand(op, x.numpy())


def test_every_mantissa_of_the_scale_decides_as_the_division():
    """Block scale D = g (an E4M3 scale of one) for all 2^23 mantissas of g, elements within two ulps of each value where the code
    changes: the codes are those of the quotients rounded to fp32."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    rows, K = 1 << 19, 16 * 5
    for part in range(1 << 4):
        g = (torch.arange(rows, device="cuda", dtype=torch.int32) + part * rows + 0x3F800000).view(torch.float32)
        near = (mids[None, :] * g[:, None].double()).float()
        x = torch.zeros(rows, K, device="cuda")
        for j in range(5):
            x[:, 16 * j] = 6.0 * g  # the block's largest: scale 1
            x[:, 16 * j + 1:16 * j + 8] = (near.view(torch.int32) + (j - 2)).view(torch.float32)
            x[:, 16 * j + 8:16 * j + 15] = -(near.view(torch.int32) + (j - 2)).view(torch.float32)
        op = ops.nvfp4_operand(rows, K)
        op.gs.copy_(g)
        ops.nvfp4_quantize(x, op, scales_given=True)
        q = (x.abs().double() / g[:, None].double()).float()  # rounded once more than the quotient in 64 bits: innocuous
        code = sum(((q > m) if i % 2 == 0 else (q >= m)).int() for i, m in enumerate(mids.float().tolist()))
        want = (grid[code.long()] * torch.sign(x) * g[:, None])
        assert torch.equal(op.values(), want)


def check_product(a, b, dtype, out=None):
    ws = ops.nvfp4_workspace(a.rows, b.rows, a.K)
    y = ops.nvfp4_matmul(a, b, TYPES[dtype], ws, out)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    va, vb = a.values().double(), b.values().double()
    ref, mag = va @ vb.T, va.abs() @ vb.abs().T
    steps = 4 * -(-a.K // 256)
    tol = (steps + 2) * 2.0 ** -22 * mag + 2.0 ** -22 * ref.abs()
    tol = tol + {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype] * ref.abs() + (6e-8 if dtype == "fp16" else 0)
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())
    # far inside that bound on the whole
    off = torch.linalg.norm(y.double() - ref) / torch.linalg.norm(ref)
    assert off < {"fp32": 1e-5, "bf16": 4e-3, "fp16": 5e-4}[dtype]
    return y


def operand(rows, K, seed, dtype="fp32"):
    op = ops.nvfp4_operand(rows, K)
    g = torch.Generator(device="cuda").manual_seed(seed)
    ops.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda").to(TYPES[dtype]), op)
    return op


SHAPES = [(1, 128, 256), (1, 4096, 8192), (3, 200, 300), (8, 1000, 2048), (9, 128, 16), (16, 8192, 4096), (17, 640, 1),
          (33, 264, 4096), (64, 512, 2000), (65, 1000, 1544), (128, 128, 8192), (100, 4100, 512), (129, 257, 256),
          (300, 1000, 1544), (256, 256, 512), (777, 1000, 1544), (1000, 130, 4096), (2048, 2048, 2048),
          # CTA pairs: ragged last tiles, rows that start on 2 and 4 bytes, a short K, an odd last 128-row block on either side
          (1500, 1501, 300), (2100, 1100, 520), (1153, 2305, 16), (1300, 1298, 4096), (2944, 1152, 256)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, dtype):
    check_product(operand(M, K, M + K), operand(N, K, N), dtype)


@pytest.mark.parametrize("M,N", [(1, 384), (7, 384), (16, 384), (31, 384), (64, 384), (128, 384), (130, 384), (512, 384), (1400, 1600),
                                 (2050, 1111)])
def test_exact_sums_come_out_exact(M, N):
    """Codes of whole numbers under scales of one: every partial sum is a small whole number."""
    K = 1024
    g = torch.Generator(device="cuda").manual_seed(M)
    vals = torch.tensor([0., 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device="cuda")
    x = vals[torch.randint(0, 11, (M, K), generator=g, device="cuda")]
    w = vals[torch.randint(0, 11, (N, K), generator=g, device="cuda")]
    x[:, ::16], w[:, ::16] = 6.0, 6.0            # each block's largest is 6: scale 448 under gs = 6/2688, values unchanged
    a, b = ops.nvfp4_operand(M, K), ops.nvfp4_operand(N, K)
    for op, v in ((a, x), (b, w)):
        op.gs.fill_(1.0)
        ops.nvfp4_quantize(v, op, scales_given=True)
        assert torch.equal(op.values(), v)
    y = ops.nvfp4_matmul(a, b, torch.float32, ops.nvfp4_workspace(M, N, K))
    assert torch.equal(y.double(), x.double() @ w.double().T)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [1, 5, 40, 200, 2500])
def test_linear_is_quantise_then_product(M, dtype):
    N, K = 520, 1100
    W = operand(N, K, 9)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K + 3, generator=g, device="cuda").to(TYPES[dtype])[:, 3:]
    ws = ops.nvfp4_workspace(M, N, K)
    y = ops.nvfp4_linear(x, W, ws)
    a = ops.nvfp4_operand(M, K)
    ops.nvfp4_quantize(x, a)
    assert torch.equal(y, ops.nvfp4_matmul(a, W, TYPES[dtype], ws))
    assert torch.equal(y, ops.nvfp4_linear(x, W, ws))
    check_product(a, W, dtype)
    assert B.moe_get_device_status(ws) == B.MOE_OK


def test_a_tokens_result_does_not_depend_on_its_batch():
    N, K = 512, 1024
    W = operand(N, K, 2)
    x = matrix(24, K, "bf16", 8).cuda()
    ws = ops.nvfp4_workspace(24, N, K)
    whole = ops.nvfp4_linear(x, W, ws, torch.empty(24, N, device="cuda"))
    again = ops.nvfp4_linear(x[8:24], W, ws, torch.empty(16, N, device="cuda"))
    tol = (4 * K / 256 + 4) * 2.0 ** -22
    assert ((whole[8:] - again).abs() <= tol * whole.abs().amax(1, keepdim=True)[8:] * 32).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_outputs_with_row_strides(dtype):
    for M, N, K, ld in ((4, 200, 256, 333), (200, 300, 256, 304), (200, 300, 512, 301), (1300, 1400, 256, 1404), (1300, 1399, 256, 1401)):
        room = torch.full((M, ld), 7.0, dtype=TYPES[dtype], device="cuda")
        y = check_product(operand(M, K, 1), operand(N, K, 2), dtype, room[:, :N])
        assert y.data_ptr() == room.data_ptr() and (room[:, N:] == 7.0).all()


def test_packed_weights_are_operands():
    """moe_nvfp4_pack's weights and their tensor-core copies, one global scale per matrix."""
    N, K, M = 256, 512, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    q, s, gs = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (N * K // 2, N * K // 16, 4))
    gs = gs.view(torch.float32)
    B.moe_nvfp4_pack(w, 1, N, K, q, s, gs)
    qt, st = torch.empty_like(q), torch.empty_like(s)
    B.moe_mxfp4_codes_to_mma(q, N, K, qt)
    B.moe_mxfp4_scales_to_mma(s, N, 2 * K, st)
    W = ops.Nvfp4Operand(N, K, qt, st, gs)
    want = torch.empty(N, K, device="cuda")
    B.moe_nvfp4_unpack(q, s, gs, 1, N, K, want)
    assert torch.equal(W.values(), want)
    check_product(operand(M, K, 4), W, "bf16")


def test_gradient_products():
    """dx = dy W and dw = dy^T x from the transposed operands."""
    M, N, K = 300, 264, 520
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((M, K), (N, K), (M, N)))
    ws = ops.nvfp4_workspace(M, N, K)
    xc, wc, dr, dc = (ops.nvfp4_operand(*s) for s in ((K, M), (K, N), (M, N), (N, M)))
    ops.nvfp4_quantize(x, None, xc, ws)
    ops.nvfp4_quantize(w, None, wc, ws)
    ops.nvfp4_quantize(dy, dr, dc, ws)
    dx, dw = check_product(dr, wc, "bf16"), check_product(dc, xc, "fp32")
    # and they are the gradients of y = x w^T up to the quantisation: its error per element is at most (1/6 + 2^-4) of the
    # block's largest, near 10% rms, so both factors together stay below 20%
    for got, ref in ((dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double())):
        assert torch.linalg.norm(got.double() - ref) / torch.linalg.norm(ref) < 0.2


def test_no_rows_other_streams_and_capture():
    W = operand(256, 512, 7)
    ws = ops.nvfp4_workspace(40, 256, 512)
    assert ops.nvfp4_linear(torch.empty(0, 512, device="cuda"), W, ws).shape == (0, 256)
    x = torch.randn(40, 512, device="cuda").bfloat16()
    y = ops.nvfp4_linear(x, W, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = ops.nvfp4_linear(x, W, ws)
    side.synchronize()
    assert torch.equal(y, y1)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(y)
    with torch.cuda.graph(graph):
        ops.nvfp4_linear(x, W, ws, out)
    x.copy_(torch.randn(40, 512, device="cuda").bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.nvfp4_linear(x, W, ws))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R_,C", [(5000, 40), (2500, 1544), (650, 7112), (700, 8192)])
def test_operands_of_many_rows(dtype, R_, C):
    """More rows than the SMs hold at once; rows of zeros, and of scales that take the division (fp32), among them."""
    x = matrix(R_, C, dtype, R_ + C)
    x[R_ // 3] = 0
    x[R_ - 1] *= 2.0 ** -10
    if dtype == "fp32":
        x[5] *= 1e-30
    op, strided = ops.nvfp4_operand(R_, C), ops.nvfp4_operand(R_, C)
    ops.nvfp4_quantize(x.cuda(), op)
    check_operand(op, x.float().numpy())
    wide = torch.zeros(R_, C + 24, dtype=x.dtype, device="cuda")
    wide[:, 8:C + 8] = x.cuda()
    ops.nvfp4_quantize(wide[:, 8:C + 8], strided)
    check_operand(strided, x.float().numpy())
    given = ops.nvfp4_operand(R_, C)
    given.gs.copy_(op.gs)
    ops.nvfp4_quantize(x.cuda(), given, scales_given=True)
    assert torch.equal(given.values(), op.values())


def test_calls_in_a_row_see_what_the_calls_before_them_wrote():
    """No synchronisation between the steps: operands of a weight and of x are made right before the products that read them."""
    def steps(pause):
        out = []
        x = matrix(300, 520, "bf16", 1).cuda()
        w = matrix(264, 520, "bf16", 2).cuda()
        W, Wt, X = ops.nvfp4_operand(264, 520), ops.nvfp4_operand(520, 264), ops.nvfp4_operand(300, 520)
        ws = ops.nvfp4_workspace(300, 520, 520)
        for i in range(24):
            x.mul_(1.03125)
            w.add_(0.0625 * (i % 3))
            pause()
            ops.nvfp4_quantize(w, W, Wt, ws)
            pause()
            y = ops.nvfp4_linear(x[:1 + 13 * i], W, ws)
            pause()
            ops.nvfp4_quantize(x, X)
            pause()
            z = ops.nvfp4_matmul(X, W, torch.bfloat16, ws)
            pause()
            back = ops.nvfp4_linear(z, Wt, ws)
            pause()
            out += [y, z, back]
        torch.cuda.synchronize()
        return out
    together, apart = steps(lambda: None), steps(torch.cuda.synchronize)
    for a, b in zip(together, apart):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R_,C,first", [(1, 1, 1), (2, 31, 1), (9, 1023, 3), (9, 1024, 1), (9, 1025, 2), (37, 2047, 0), (1300, 300, 1),
                                        (700, 7111, 5), (3, 8192, 1)])
def test_operands_of_rows_that_start_anywhere(dtype, R_, C, first):
    whole = matrix(R_ + 1, C + 7, dtype, R_ + C)
    x = whole.flatten()[first:first + R_ * (C + 5)].view(R_, C + 5)[:, :C]
    dev = whole.cuda().flatten()[first:first + R_ * (C + 5)].view(R_, C + 5)[:, :C]
    op = ops.nvfp4_operand(R_, C)
    ops.nvfp4_quantize(dev, op)
    check_operand(op, x.float().numpy())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R_,C", [(10000, 40), (5003, 1544), (1301, 7112), (1300, 8192)])
def test_operands_of_rows_by_the_thousand(dtype, R_, C):
    x = matrix(R_, C, dtype, R_ + C)
    x[7] = 0
    op = ops.nvfp4_operand(R_, C)
    ops.nvfp4_quantize(x.cuda(), op)
    check_operand(op, x.float().numpy())
