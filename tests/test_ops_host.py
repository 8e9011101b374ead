"""Argument checks of the routing rules and the dense NVFP4 products (no GPU: everything is refused before a launch), their size
helpers and struct layouts."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SHAPE, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED_SHAPE, B.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return B.load()


def rule(**kw):
    r = ops.route_rule()
    for name, v in kw.items():
        setattr(r, name, v)
    return r


def test_route_scores_refusals(lib):
    def call(logits=256, dtype=0, ld=64, bias=None, T=4, E=64, k=8, r=None, ids=256, w=256):
        return lib.moe_route_scores(logits, dtype, ld, bias, T, E, k, rule() if r is None else r, ids, w, None, None, None)
    assert call(T=0) == B.MOE_OK
    assert call(T=-1) == SHAPE and call(E=0) == SHAPE and call(E=1025, ld=2000) == SHAPE
    assert call(k=0) == SHAPE and call(k=33) == SHAPE and call(E=4, ld=4, k=5) == SHAPE
    assert call(ld=63) == SHAPE
    assert call(dtype=3) == INVALID and call(logits=None) == INVALID and call(ids=None) == INVALID and call(w=None) == INVALID
    assert call(logits=258) == INVALID and call(logits=257, dtype=1) == INVALID
    assert call(r=rule(score=2)) == INVALID and call(r=rule(group_score=2)) == INVALID
    assert call(r=rule(scale=float("nan"))) == INVALID and call(r=rule(scale=float("inf"))) == INVALID
    assert call(r=rule(groups=3)) == SHAPE and call(r=rule(groups=0)) == SHAPE and call(r=rule(groups=64, top_groups=64)) == SHAPE
    assert call(r=rule(groups=8, top_groups=9)) == SHAPE and call(r=rule(groups=8, top_groups=0)) == SHAPE
    assert call(r=rule(groups=16, top_groups=1)) == SHAPE  # k = 8 of 4 experts
    assert lib.moe_route_scores(256, 0, 64, None, 4, 64, 8, None, 256, 256, None, None, None) == INVALID


def test_route_backward_and_logits_refusals(lib):
    def call(logits=256, dtype=0, ld=64, T=4, E=64, k=8, ids=256, dw=256, dl=256, ldd=64):
        return lib.moe_route_scores_backward(logits, dtype, ld, T, E, k, rule(), ids, dw, None, dl, ldd, None)
    assert call(T=0) == B.MOE_OK
    assert call(ld=63) == SHAPE and call(ldd=63) == SHAPE and call(k=0) == SHAPE and call(dtype=-1) == INVALID
    for name in ("logits", "ids", "dw", "dl"):
        assert call(**{name: None}) == INVALID
    assert call(dl=258) == INVALID
    assert lib.moe_route_logits(256, 256, None, 4, 100, 8, 256, None) == SHAPE
    assert lib.moe_route_logits(264, 256, None, 4, 128, 8, 256, None) == INVALID
    assert lib.moe_route_logits(256, 256, None, 4, 128, 8, None, None) == INVALID
    assert lib.moe_route_logits(None, None, None, 0, 128, 8, None, None) == B.MOE_OK


def test_combine_backward_refusals(lib):
    def call(dy=256, yp=256, inv=256, w=256, T=4, k=2, d=256, dw=256, dyp=256):
        return lib.moe_combine_backward(dy, yp, inv, w, T, k, d, dw, dyp, None)
    assert call(T=0) == B.MOE_OK
    assert call(d=12) == SHAPE and call(k=33) == SHAPE and call(k=0) == SHAPE and call(T=-1) == SHAPE
    assert call(dy=None) == INVALID and call(inv=None) == INVALID and call(dw=None, dyp=None) == INVALID
    assert call(yp=None) == INVALID and call(w=None) == INVALID and call(dy=264) == INVALID and call(dyp=264) == INVALID


def test_nvfp4_sizes_and_refusals(lib):
    assert B.moe_nvfp4_operand_codes(1, 1) == 128 * 128 and B.moe_nvfp4_operand_scales(1, 1) == 2048
    assert B.moe_nvfp4_operand_codes(129, 257) == 256 * 256 and B.moe_nvfp4_operand_codes(0, 256) == 0
    assert B.moe_nvfp4_operand_codes(4, 0) == 0 and B.moe_nvfp4_operand_codes(-1, 256) == 0
    # the tensor-core copies of packed weights have the same sizes
    assert B.moe_nvfp4_operand_scales(256, 512) == B.moe_mxfp4_mma_scale_bytes(256, 2 * 512)
    assert B.moe_nvfp4_workspace_size(4, 256, 0) == 0 and B.moe_nvfp4_workspace_size(1 << 30, 256, 256) == 0
    big = 1 << 40
    op = B.moe_nvfp4_operand(256, 256, 256, 1)

    def quant(x=256, dtype=1, R=4, C=64, ld=64, rows=op, cols=None, given=0, ws=None, n=0):
        return lib.moe_nvfp4_quantize(x, dtype, R, C, ld, rows, cols, given, ws, n, None)
    assert quant(R=0) == B.MOE_OK
    assert quant(C=0) == SHAPE and quant(ld=63) == SHAPE and quant(R=-1) == SHAPE
    assert quant(dtype=5) == INVALID and quant(x=None) == INVALID and quant(x=257) == INVALID and quant(rows=None) == INVALID
    assert quant(rows=B.moe_nvfp4_operand(264, 256, 256, 1)) == INVALID
    assert quant(rows=B.moe_nvfp4_operand(256, None, 256, 1)) == INVALID
    assert quant(rows=B.moe_nvfp4_operand(256, 256, 256, 0)) == INVALID  # one scale for rows that are to get their own
    assert quant(cols=op) == WS and quant(cols=op, ws=256, n=8192) == WS and quant(cols=op, ws=128, n=big) == WS

    def matmul(A=op, Bo=op, M=4, N=64, K=64, y=256, dtype=1, ldy=64, ws=256, n=big):
        return lib.moe_nvfp4_matmul(A, Bo, M, N, K, y, dtype, ldy, ws, n, None)
    assert matmul(M=0) == B.MOE_OK and matmul(N=0) == B.MOE_OK
    assert matmul(K=0) == SHAPE and matmul(M=-1) == SHAPE and matmul(ldy=63) == SHAPE and matmul(M=1 << 27, N=1 << 27) == SHAPE
    assert matmul(y=None) == INVALID and matmul(y=257) == INVALID and matmul(dtype=9) == INVALID and matmul(A=None) == INVALID
    assert matmul(ws=None) == WS and matmul(n=100) == WS

    def linear(x=256, M=4, K=64, ldx=64, W=op, N=64, y=256, ldy=64, ws=256, n=big):
        return lib.moe_nvfp4_linear(x, 1, M, K, ldx, W, N, y, 1, ldy, ws, n, None)
    assert linear(M=0) == B.MOE_OK and linear(ldx=63) == SHAPE and linear(x=None) == INVALID and linear(x=257) == INVALID
    assert linear(W=None) == INVALID and linear(n=8192) == WS
    assert lib.moe_nvfp4_operand_values(op, 4, 64, None, None) == INVALID


def test_torch_level_refusals():
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ops.route_scores(cpu, 8, ops.route_rule())
    with pytest.raises(ValueError):
        ops.route_rule("tanh")
    with pytest.raises(ValueError):
        ops.route_rule(group_score="mean")
    with pytest.raises(ValueError):
        ops.route_rule(scale=float("nan"))
    with pytest.raises(ValueError):
        ops.nvfp4_workspace(4, 64, 0)
    with pytest.raises(ValueError):
        ops.Nvfp4Operand(4, 64, torch.zeros(5, dtype=torch.uint8), torch.zeros(5, dtype=torch.uint8), torch.zeros(4))


@pytest.mark.parametrize("name", ["moe_route_rule", "moe_nvfp4_operand"])
def test_struct_offsets_equal_the_c_compilers(name, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    cls = getattr(B, name)
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe.h"', "int main(void) {",
             '  printf("%%zu\\n", sizeof(%s));' % name]
    lines += ['  printf("%%zu\\n", offsetof(%s, %s));' % (name, f) for f, _ in cls._fields_]
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


def test_enums_mirror_the_header():
    src = open(os.path.join(ROOT, "include", "moe.h")).read()
    for name in ("MOE_F32", "MOE_BF16", "MOE_F16", "MOE_SCORE_SIGMOID", "MOE_SCORE_SOFTMAX", "MOE_GROUP_MAX", "MOE_GROUP_TOP2"):
        assert int(re.search(r"\b%s = (\d+)" % name, src).group(1)) == getattr(B, name)


def test_reference_gradient_against_differences():
    """The tests' own 64-bit gradient against central differences of their 64-bit forward."""
    import ops_reference as R
    rng = np.random.default_rng(3)
    l = rng.standard_normal((2, 12))
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            ids, _, _ = R.route(l, 4, score=score, renormalize=renorm, scale=1.5)
            dw, dsc = rng.standard_normal((2, 4)), rng.standard_normal((2, 12))

            def loss(x):
                out = 0.0
                for t in range(2):
                    s = 1 / (1 + np.exp(-x[t])) if score == "sigmoid" else np.exp(x[t]) / np.exp(x[t]).sum()
                    u = s[ids[t]]
                    out += (1.5 * (u / u.sum() if renorm else u) * dw[t]).sum() + (s * dsc[t]).sum()
                return out
            dl, _ = R.route_backward(l, ids, dw, score, renorm, 1.5, dsc)
            for t in range(2):
                for e in range(12):
                    h = np.zeros_like(l)
                    h[t, e] = 1e-5
                    assert abs((loss(l + h) - loss(l - h)) / 2e-5 - dl[t, e]) < 1e-8
