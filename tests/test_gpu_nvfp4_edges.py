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
