"""Routing rules, their gradients and dense NVFP4 products on torch tensors.

Each function checks its tensors, allocates its results and makes one call of the library, in an extension module; the work is
the library's kernels, on torch's current stream.  None of them synchronises.  Tensors of another device than the current one are
refused (`with torch.cuda.device(...)` makes theirs the current one).  None of them takes part in autograd: gradients come from the
calls that compute them, and backward() through a result raises an error rather than leave its gradient out.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _build
from . import binding as B

_SCORES = {"sigmoid": B.MOE_SCORE_SIGMOID, "softmax": B.MOE_SCORE_SOFTMAX}
_GROUP_SCORES = {"max": B.MOE_GROUP_MAX, "top2": B.MOE_GROUP_TOP2}
_SCALAR_TYPES = {torch.float32: 6, torch.float16: 5, torch.bfloat16: 15}  # torch's own numbers of these types

_module = None


def _calls():
    """The extension module (csrc/torch_ops.cpp), which checks the tensors, allocates the results and calls the library."""
    global _module
    if _module is None:
        import importlib.util
        _build.build()  # (where the library or the module is not there, or older than what it is made of)
        B.load()
        spec = importlib.util.spec_from_file_location("moe_torch_ops", _build.TORCH_OPS)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_error(B.MoeError)
        _module = module
    return _module


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _need_current(device: torch.device, what: str) -> None:
    _need(device.index is None or device.index == torch.cuda.current_device(), "%s: on another device than the current one" % what)


class _Tied(torch.autograd.Function):
    """A result that hangs on inputs which require a gradient, without a formula for it."""

    @staticmethod
    def forward(ctx, hint, result, *inputs):
        ctx.hint = hint
        return result.detach()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("no autograd formula: %s" % ctx.hint)


def tied(hint: str, result: torch.Tensor, *inputs: Optional[torch.Tensor]) -> torch.Tensor:
    """`result`, which backward() does not get past where one of the inputs requires a gradient: an error with the hint."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        return _Tied.apply(hint, result, *inputs)
    return result


# ------------------------------------------------------------------ routing rules

def route_rule(score: str = "sigmoid", groups: int = 1, top_groups: int = 1, group_score: str = "top2",
               renormalize: bool = True, scale: float = 1.0) -> B.moe_route_rule:
    """A routing rule: scores by "sigmoid" or "softmax"; experts in `groups` equal groups, of which the `top_groups` with
    the best group score ("max": the largest ranking value, "top2": the sum of the two largest) are open to a token;
    weights divided by their sum when `renormalize`, times `scale`."""
    _need(score in _SCORES, "score: %r" % (score,))
    _need(group_score in _GROUP_SCORES, "group_score: %r" % (group_score,))
    _need(math.isfinite(scale), "scale: a finite number expected")
    return B.moe_route_rule(_SCORES[score], groups, top_groups, _GROUP_SCORES[group_score], int(bool(renormalize)), scale)


def route_logits(x: torch.Tensor, W_r: torch.Tensor, b: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp32 router logits [T, E] of bf16 x [T, d] and fp32 W_r [E, d] in the layer's fixed order, b added."""
    _need(x.dim() == 2 and x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous(), "x: contiguous bf16 [T, d] expected")
    _need_current(x.device, "x")
    T, d = x.shape
    _need(W_r.dim() == 2 and W_r.shape[1] == d and W_r.dtype == torch.float32 and W_r.device == x.device and W_r.is_contiguous(),
          "W_r: contiguous fp32 [E, d] expected")
    E = W_r.shape[0]
    _need(b is None or (b.shape == (E,) and b.dtype == torch.float32 and b.device == x.device and b.is_contiguous()),
          "b: contiguous fp32 [E] expected")
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    B.moe_route_logits(x, W_r, b, T, d, E, logits)
    return tied("route_logits' gradients are products of dlogits with x and W_r", logits, x, W_r, b)


def route_scores(logits: torch.Tensor, k: int, rule: B.moe_route_rule, bias: Optional[torch.Tensor] = None,
                 scores: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """ids int32 [T, k] (ascending) and weights fp32 [T, k] of logits [T, E] under `rule`; `bias` fp32 [E] takes part in the
    choice only (+inf: picked first, -inf: last).  Logits of -inf take an expert out of service.  scores fp32 [T, E] and counts int32 [E], when given, receive
    all the scores and the picks per expert."""
    ids, w = (_module or _calls()).route_scores(logits, k, rule, bias, scores, counts)
    if logits.requires_grad:
        w = tied("route_scores' gradient is route_scores_backward", w, logits)
    return ids, w


def route_scores_backward(logits: torch.Tensor, ids: torch.Tensor, dw: torch.Tensor, rule: B.moe_route_rule,
                          dscores: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits (their type) from that of the weights, dw fp32 [T, k], and of the scores, dscores fp32 [T, E];
    the choice `ids` is held fixed."""
    return (_module or _calls()).route_scores_backward(logits, ids, dw, rule, dscores)


def combine_backward(dy: torch.Tensor, y_perm: Optional[torch.Tensor], inv_pos: torch.Tensor, w: torch.Tensor,
                     need_dw: bool = True, need_dy_perm: bool = True
                     ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of the weighted sum y[t] = sum_j w[t, j] y_perm[inv_pos[t k + j]]: dw fp32 [T, k] and dy_perm bf16 [T k, d]
    (None where not needed) from dy bf16 [T, d].  Rows of dy_perm that no entry of inv_pos names are not written."""
    return (_module or _calls()).combine_backward(dy, y_perm, inv_pos, w, need_dw, need_dy_perm)


# ------------------------------------------------------------------ dense NVFP4 products

class Nvfp4Operand:
    """A matrix [rows, K] in NVFP4 as the tensor cores read it, contracting along K: code tiles q and scale atoms s (uint8, the
    sizes of binding.moe_nvfp4_operand_codes / _scales) and fp32 scales gs, one per row or one for all."""

    def __init__(self, rows: int, K: int, q: torch.Tensor, s: torch.Tensor, gs: torch.Tensor):
        nq, ns = B.moe_nvfp4_operand_codes(rows, K), B.moe_nvfp4_operand_scales(rows, K)
        _need(rows >= 0 and K >= 1 and (nq > 0 or rows == 0), "unsupported operand shape [%d, %d]" % (rows, K))
        for t, n, dtype, what in ((q, nq, torch.uint8, "q"), (s, ns, torch.uint8, "s"), (gs, gs.numel(), torch.float32, "gs")):
            _need(t.is_cuda and t.shape == (n,) and t.dtype == dtype and t.device == q.device and t.is_contiguous(),
                  "%s: contiguous CUDA %s [%d] expected" % (what, dtype, n))
        _need(gs.numel() in (1, rows), "gs: one scale per row, or one")
        self.rows, self.K, self.q, self.s, self.gs = rows, K, q, s, gs
        self.device = q.get_device()
        self.struct = B.moe_nvfp4_operand(q.data_ptr(), s.data_ptr(), gs.data_ptr(), int(gs.numel() == rows))

    def values(self) -> torch.Tensor:
        """The numbers it stands for, fp32 [rows, K]."""
        _need_current(self.q.device, "operand")
        v = torch.empty((self.rows, self.K), dtype=torch.float32, device=self.q.device)
        B.moe_nvfp4_operand_values(self.struct, self.rows, self.K, v)
        return v


def nvfp4_operand(rows: int, K: int, device="cuda") -> Nvfp4Operand:
    """Room for an operand [rows, K] with a scale per row."""
    on = torch.device(device)
    _need(on.type == "cuda", "device: a CUDA device expected")
    index = on.index if on.index is not None else torch.cuda.current_device()
    op = object.__new__(Nvfp4Operand)  # (its tensors are right as they come)
    op.q, op.s, op.gs, q, s, gs = (_module or _calls()).nvfp4_room(rows, K, index)
    op.rows, op.K, op.device = rows, K, index
    op.struct = B.moe_nvfp4_operand(q, s, gs, 1)
    return op


def nvfp4_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of nvfp4_linear, nvfp4_matmul and nvfp4_quantize at these sizes, initialised."""
    n = B.moe_nvfp4_workspace_size(M, N, K)
    _need(n > 0, "unsupported shape M=%d N=%d K=%d" % (M, N, K))
    _need_current(torch.device(device), "workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    B.moe_workspace_init(ws)
    return ws


def nvfp4_quantize(x: torch.Tensor, rows: Optional[Nvfp4Operand] = None, cols: Optional[Nvfp4Operand] = None,
                   workspace: Optional[torch.Tensor] = None, scales_given: bool = False) -> None:
    """Operands of x [R, C]: `rows` [R, C] receives that of x, `cols` [C, R] that of its transpose; both from one call when both are
    given.  The row scales are computed from the rows, or taken from the operands (scales_given)."""
    r = (None, 0, 0, 0) if rows is None else (rows.struct, rows.rows, rows.K, rows.device)
    c = (None, 0, 0, 0) if cols is None else (cols.struct, cols.rows, cols.K, cols.device)
    (_module or _calls()).nvfp4_quantize(x, *r, *c, workspace, scales_given)


def nvfp4_matmul(a: Nvfp4Operand, b: Nvfp4Operand, dtype: torch.dtype, workspace: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] of dtype (into `out` when given)."""
    code = _SCALAR_TYPES.get(dtype)
    if code is None:
        raise TypeError("fp32, bf16 or fp16 expected, got %s" % (dtype,))
    return (_module or _calls()).nvfp4_matmul(a.struct, a.rows, a.K, a.device, b.struct, b.rows, b.K, b.device, a.q, code, workspace, out)


def nvfp4_linear(x: torch.Tensor, W: Nvfp4Operand, workspace: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] times W [N, K] transposed, x quantised row by row: [M, N] of x's type (or of `out`'s)."""
    y = (_module or _calls()).nvfp4_linear(x, W.struct, W.rows, W.K, W.device, workspace, out)
    if x.requires_grad and out is None:
        y = tied("nvfp4_linear's gradients are nvfp4_matmul of transposed operands", y, x)
    return y
