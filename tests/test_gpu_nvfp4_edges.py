"""NVFP4 operands at the ends of their range, against the format's rule written out here in fp32 steps: equal, not close."""
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def rule_values(x, gs):
    """The numbers that the rows of x (CPU) stand for under given row scales gs [rows]: t = (max|block| / g) / 6 to the nearest E4M3
    (at most 448), D = scale g, nearest E2M1 to v / D."""
    v = x.float()
    rows, K = v.shape
    b = torch.nn.functional.pad(v, (0, -K % 16)).view(rows, -1, 16)
    g = gs.view(-1, 1).expand(rows, 1)
    t = (b.abs().amax(2) / g) / torch.tensor(6.0)
    scale = t.clamp(max=448.0).to(torch.float8_e4m3fn).float()
    D = (scale * g)[:, :, None]
    m = torch.where(D > 0, b.abs() / D, torch.zeros_like(b))
    code = sum(((m > c) if i % 2 == 0 else (m >= c)).int() for i, c in enumerate(MIDS))
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6])
    out = grid[code.long()] * torch.where(b < 0, -1.0, 1.0) * scale[:, :, None] * g[:, :, None]
    return out.view(rows, -1)[:, :K]


def all_forms(x, gs_rows, gs_cols, ld_extra=0):
    """Values of the operand of x (given scales) from the row form alone, and of both forms from one call and the column form alone."""
    R, C = x.shape
    dev = torch.zeros(R, C + ld_extra, dtype=x.dtype, device="cuda")[:, :C]
    dev.copy_(x)
    made = []
    for want_rows, want_cols in ((True, False), (True, True), (False, True)):
        r, c = (ops.nvfp4_operand(R, C) if want_rows else None), (ops.nvfp4_operand(C, R) if want_cols else None)
        if r:
            r.gs.copy_(gs_rows)
        if c:
            c.gs.copy_(gs_cols)
        ops.nvfp4_quantize(dev, r, c, scales_given=True)
        made += [("rows", o) for o in (r,) if o] + [("cols", o) for o in (c,) if o]
    return made


# (rows x columns: a few, many short ones, and as many as are streamed through shared memory; the last with unaligned rows)
SHAPES = [(6, 300, 0), (40, 64, 0), (2600, 4096, 0), (300, 1111, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,C,extra", SHAPES)
def test_given_scales_saturate_whatever_the_type(dtype, R, C, extra):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=g).to(TYPES[dtype])
    top = torch.finfo(TYPES[dtype]).max
    x[0, 3], x[0, 20], x[0, 40] = float("inf"), -float("inf"), top
    x[1, 5], x[2, 6] = -top, top / 2
    x[3, C - 1] = float("inf")
    x[R - 1, 0] = -float("inf")
    gs_rows = 2.0 ** torch.randint(-12, -6, (R,), generator=g).float() * 1.25
    gs_cols = 2.0 ** torch.randint(-12, -6, (C,), generator=g).float() * 1.375
    want = {"rows": rule_values(x, gs_rows), "cols": rule_values(x.T.contiguous(), gs_cols)}
    assert torch.isfinite(want["rows"]).all() and torch.isfinite(want["cols"]).all()
    for form, op in all_forms(x, gs_rows, gs_cols, extra):
        assert torch.equal(op.values().cpu(), want[form]), form


def both_ways(x, extra=0):
    """Values of x's operand rows from the row form alone and from the call for both, and of its columns from both calls that make them."""
    R, C = x.shape
    dev = torch.zeros(R, C + extra, dtype=x.dtype, device="cuda")[:, :C]
    dev.copy_(x)
    ws = ops.nvfp4_workspace(R, C, C)
    r, r2, c, c2 = (ops.nvfp4_operand(*s) for s in ((R, C), (R, C), (C, R), (C, R)))
    ops.nvfp4_quantize(dev, r)
    ops.nvfp4_quantize(dev, r2, c, ws)
    ops.nvfp4_quantize(dev, None, c2, ws)
    return (r, r2), (c, c2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,C,extra", SHAPES)
def test_a_nan_reaches_its_row_and_no_other(dtype, R, C, extra):
    g = torch.Generator().manual_seed(R * C)
    x = torch.randn(R, C, generator=g).to(TYPES[dtype])
    clean = both_ways(x, extra)
    at = [(0, 0), (2, C - 1), (2, 17), (R - 1, 33)]
    for r, c in at:
        x[r, c] = float("nan")
    x[1] = float("nan")           # a whole row
    x[3, 5] = -float("inf")       # an infinite scale
    bad_rows = torch.zeros(R, dtype=torch.bool)
    bad_rows[[0, 1, 2, 3, R - 1]] = True
    got = both_ways(x, extra)
    for now, was in zip(got[0], clean[0]):
        v = now.values().cpu()
        assert torch.isnan(v[bad_rows]).all() and torch.isnan(now.gs.cpu()[[0, 1, 2, R - 1]]).all()
        assert torch.equal(v[~bad_rows], was.values().cpu()[~bad_rows])
    for op in got[1]:
        assert torch.isnan(op.values()).all()  # (row 1 reaches every column)
    x[1] = 0.5
    bad_cols = torch.zeros(C, dtype=torch.bool)
    bad_cols[[0, C - 1, 17, 33, 5]] = True
    y = x.clone()
    y[:, bad_cols] = 0.0
    for now, was in zip(both_ways(x, extra)[1], both_ways(y, extra)[1]):
        v = now.values().cpu()
        assert torch.isnan(v[bad_cols]).all()
        assert torch.equal(v[~bad_cols], was.values().cpu()[~bad_cols])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_nan_under_given_scales_reaches_its_block(dtype):
    R, C = 40, 300
    x = torch.randn(R, C, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    gs_rows, gs_cols = torch.full((R,), 2.0 ** -10), torch.full((C,), 2.0 ** -9)
    want = {"rows": rule_values(x, gs_rows), "cols": rule_values(x.T.contiguous(), gs_cols)}
    x[7, 40] = float("nan")
    for form, op in all_forms(x, gs_rows, gs_cols):
        v, r, b = op.values().cpu(), *((7, 32) if form == "rows" else (40, 0))
        assert torch.isnan(v[r, b:b + 16]).all()
        v[r, b:b + 16] = want[form][r, b:b + 16]
        assert torch.equal(v, want[form]), form


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [1, 5, 40, 200, 1500])
def test_a_nan_activation_shows_in_its_row_of_the_product(dtype, M):
    N, K = 1600, 300
    g = torch.Generator(device="cuda").manual_seed(M)
    W = ops.nvfp4_operand(N, K)
    ops.nvfp4_quantize(torch.randn(N, K, generator=g, device="cuda"), W)
    x = torch.randn(M, K, generator=g, device="cuda").to(TYPES[dtype])
    ws = ops.nvfp4_workspace(M, N, K)
    clean = ops.nvfp4_linear(x, W, ws)
    x[M // 2, 250] = float("nan")
    y = ops.nvfp4_linear(x, W, ws)
    assert torch.isnan(y[M // 2]).all()
    others = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[others], clean[others])
    assert B.moe_get_device_status(ws) == B.MOE_OK


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,C,extra", SHAPES)
def test_a_given_scale_of_zero_makes_zeros(dtype, R, C, extra):
    g = torch.Generator().manual_seed(R)
    x = torch.randn(R, C, generator=g).to(TYPES[dtype])
    x[0] = 0.0                      # what a scale of zero is usually worked out from
    x[1, :16] = 0.0
    x[:, 1] = 0.0
    x[2, 20] = float("inf")
    gs_rows, gs_cols = torch.full((R,), 2.0 ** -9), torch.full((C,), 2.0 ** -9)
    gs_rows[:3], gs_cols[:3] = 0.0, 0.0
    want = {"rows": rule_values(x, torch.where(gs_rows > 0, gs_rows, 1.0)), "cols": rule_values(x.T.contiguous(), torch.where(gs_cols > 0, gs_cols, 1.0))}
    want["rows"][:3], want["cols"][:3] = 0.0, 0.0
    for form, op in all_forms(x, gs_rows, gs_cols, extra):
        assert torch.equal(op.values().cpu(), want[form]), form
        other = ops.nvfp4_operand(9, op.K)
        ops.nvfp4_quantize(torch.ones(9, op.K, device="cuda"), other)
        y = ops.nvfp4_matmul(op, other, torch.float32, ops.nvfp4_workspace(op.rows, 9, op.K))
        assert (y[:3] == 0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 130, 300), (9, 264, 1024), (40, 130, 300), (100, 1000, 520), (200, 600, 300), (1500, 1501, 300)])
@pytest.mark.parametrize("x_size,w_size", [(3e38, 1e-9), (3e38, 1e-37), (1e36, 1e-30), (1e-37, 1e30), (2e-44, 1e36), (1e-18, 1e-18), (1e18, 1e18)])
def test_rows_of_any_size_give_what_fp32_can_hold(out, M, N, K, x_size, w_size):
    """Rows of x of magnitude 1 and of x_size (the type's largest, say, as a mask value) times weights around w_size.  Against 64-bit products of
    the operands' values: (4 K/256 + 4) 2^-22 of the sum of the magnitudes, as in the other tests of the products, half a step of the result's type
    and of the smallest number that it has; results beyond the type are infinite."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").clamp(-1, 1)
    w = torch.randn(N, K, generator=g, device="cuda").clamp(-1, 1).double() * w_size
    big = torch.rand(M, 1, generator=g, device="cuda") < 0.5
    big[0] = True
    x = torch.where(big, x.double() * x_size, x.double()).float()
    a, b = ops.nvfp4_operand(M, K), ops.nvfp4_operand(N, K)
    ops.nvfp4_quantize(x, a)
    ops.nvfp4_quantize(w.float(), b)
    ws = ops.nvfp4_workspace(M, N, K)
    y = ops.nvfp4_matmul(a, b, TYPES[out], ws).double()
    va, vb = (exact_values(o) for o in (a, b))
    ref, mag = va @ vb.T, va.abs() @ vb.abs().T
    info = torch.finfo(TYPES[out])
    tol = (4 * -(-K // 256) + 4) * 2.0 ** -22 * mag + info.eps / 2 * ref.abs() + info.smallest_normal * info.eps
    sure = ref.abs() + tol <= info.max
    assert ((y - ref).abs() <= tol)[sure].all()
    assert torch.isinf(y[ref.abs() - tol > 1.01 * info.max]).all()
    assert torch.equal(y.to(TYPES[out]), ops.nvfp4_linear(x, b, ws, torch.empty(M, N, dtype=TYPES[out], device="cuda")))
    assert B.moe_get_device_status(ws) == B.MOE_OK


def exact_values(op):
    """An operand's numbers without the rounding of its values(): that of the same codes under scales of one, times the row scales."""
    one = ops.Nvfp4Operand(op.rows, op.K, op.q, op.s, torch.ones_like(op.gs))
    return one.values().double() * op.gs.double()[:, None]
