"""Routing rules, their gradients and dense NVFP4 products on torch tensors.

Each function checks its tensors, allocates its results and makes one call of the library (binding.py); the work is the
library's kernels, on torch's current stream.  None of them synchronises.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import binding as B

_DTYPES = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_F16}
_SCORES = {"sigmoid": B.MOE_SCORE_SIGMOID, "softmax": B.MOE_SCORE_SOFTMAX}
_GROUP_SCORES = {"max": B.MOE_GROUP_MAX, "top2": B.MOE_GROUP_TOP2}


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s: fp32, bf16 or fp16 expected, got %s" % (what, t.dtype))
    return code


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _matrix(t: torch.Tensor, what: str) -> int:
    """Row stride of a 2-D CUDA tensor whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError("%s: a CUDA matrix expected" % what)
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError("%s: contiguous rows expected" % what)
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError("%s: rows may not overlap" % what)
    return ld


def _plain(t: torch.Tensor, shape: tuple, dtype: torch.dtype, like: torch.Tensor, what: str) -> None:
    """A contiguous tensor of this shape and type on `like`'s device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError("%s: contiguous %s of %s on %s expected" % (what, shape, dtype, like.device))


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
    T, d = x.shape
    E = W_r.shape[0]
    _plain(W_r, (E, d), torch.float32, x, "W_r")
    if b is not None:
        _plain(b, (E,), torch.float32, x, "b")
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    B.moe_route_logits(x, W_r, b, T, d, E, logits)
    return logits


def route_scores(logits: torch.Tensor, k: int, rule: B.moe_route_rule, bias: Optional[torch.Tensor] = None,
                 scores: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """ids int32 [T, k] (ascending) and weights fp32 [T, k] of logits [T, E] under `rule`; `bias` fp32 [E] takes part in the
    choice only.  Logits of -inf take an expert out of service.  scores fp32 [T, E] and counts int32 [E], when given, receive
    all the scores and the picks per expert."""
    ld, code = _matrix(logits, "logits"), _dtype(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _plain(bias, (E,), torch.float32, logits, "bias")
    if scores is not None:
        _plain(scores, (T, E), torch.float32, logits, "scores")
    if counts is not None:
        _plain(counts, (E,), torch.int32, logits, "counts")
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    B.moe_route_scores(logits, code, ld, bias, T, E, k, rule, ids, w, scores, counts)
    return ids, w


def route_scores_backward(logits: torch.Tensor, ids: torch.Tensor, dw: torch.Tensor, rule: B.moe_route_rule,
                          dscores: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits (their type) from that of the weights, dw fp32 [T, k], and of the scores, dscores fp32 [T, E];
    the choice `ids` is held fixed."""
    ld, code = _matrix(logits, "logits"), _dtype(logits, "logits")
    T, E = logits.shape
    _need(ids.dim() == 2, "ids: [T, k] expected")
    k = ids.shape[1]
    _plain(ids, (T, k), torch.int32, logits, "ids")
    _plain(dw, (T, k), torch.float32, logits, "dw")
    if dscores is not None:
        _plain(dscores, (T, E), torch.float32, logits, "dscores")
    dlogits = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    B.moe_route_scores_backward(logits, code, ld, T, E, k, rule, ids, dw, dscores, dlogits, E)
    return dlogits


def combine_backward(dy: torch.Tensor, y_perm: Optional[torch.Tensor], inv_pos: torch.Tensor, w: torch.Tensor,
                     need_dw: bool = True, need_dy_perm: bool = True
                     ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of the weighted sum y[t] = sum_j w[t, j] y_perm[inv_pos[t k + j]]: dw fp32 [T, k] and dy_perm bf16 [T k, d]
    (None where not needed) from dy bf16 [T, d]."""
    _need(dy.dim() == 2 and dy.is_cuda and dy.dtype == torch.bfloat16 and dy.is_contiguous(), "dy: contiguous bf16 [T, d] expected")
    _need(w.dim() == 2, "w: [T, k] expected")
    T, d = dy.shape
    k = w.shape[1]
    _plain(w, (T, k), torch.float32, dy, "w")
    _plain(inv_pos, (T * k,), torch.int32, dy, "inv_pos")
    if need_dw:
        _need(y_perm is not None, "y_perm: needed for dw")
        _plain(y_perm, (T * k, d), torch.bfloat16, dy, "y_perm")
    dw = torch.empty((T, k), dtype=torch.float32, device=dy.device) if need_dw else None
    dy_perm = torch.empty((T * k, d), dtype=torch.bfloat16, device=dy.device) if need_dy_perm else None
    if need_dw or need_dy_perm:
        B.moe_combine_backward(dy, y_perm if need_dw else None, inv_pos, w, T, k, d, dw, dy_perm)
    return dw, dy_perm


# ------------------------------------------------------------------ dense NVFP4 products

class Nvfp4Operand:
    """A matrix [rows, K] in NVFP4 as the tensor cores read it, contracting along K: code tiles q and scale atoms s (uint8, the
    sizes of binding.moe_nvfp4_operand_codes / _scales) and fp32 scales gs, one per row or one for all."""

    def __init__(self, rows: int, K: int, q: torch.Tensor, s: torch.Tensor, gs: torch.Tensor):
        nq, ns = B.moe_nvfp4_operand_codes(rows, K), B.moe_nvfp4_operand_scales(rows, K)
        _need(rows >= 0 and K >= 1 and (nq > 0 or rows == 0), "unsupported operand shape [%d, %d]" % (rows, K))
        _plain(q, (nq,), torch.uint8, q, "q")
        _plain(s, (ns,), torch.uint8, q, "s")
        _need(q.is_cuda, "q: a CUDA tensor expected")
        _need(gs.numel() in (1, rows), "gs: one scale per row, or one")
        _plain(gs, (gs.numel(),), torch.float32, q, "gs")
        self.rows, self.K, self.q, self.s, self.gs = rows, K, q, s, gs
        self.struct = B.moe_nvfp4_operand(q.data_ptr(), s.data_ptr(), gs.data_ptr(), int(gs.numel() == rows))

    def values(self) -> torch.Tensor:
        """The numbers it stands for, fp32 [rows, K]."""
        v = torch.empty((self.rows, self.K), dtype=torch.float32, device=self.q.device)
        B.moe_nvfp4_operand_values(self.struct, self.rows, self.K, v)
        return v


def nvfp4_operand(rows: int, K: int, device="cuda") -> Nvfp4Operand:
    """Room for an operand [rows, K] with a scale per row."""
    u8 = dict(dtype=torch.uint8, device=device)
    return Nvfp4Operand(rows, K, torch.empty(B.moe_nvfp4_operand_codes(rows, K), **u8),
                        torch.empty(B.moe_nvfp4_operand_scales(rows, K), **u8),
                        torch.empty(rows, dtype=torch.float32, device=device))


def nvfp4_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of nvfp4_linear, nvfp4_matmul and nvfp4_quantize at these sizes, initialised."""
    n = B.moe_nvfp4_workspace_size(M, N, K)
    _need(n > 0, "unsupported shape M=%d N=%d K=%d" % (M, N, K))
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    B.moe_workspace_init(ws)
    return ws


def _on(op: Nvfp4Operand, rows: int, K: int, t: torch.Tensor, what: str) -> None:
    _need((op.rows, op.K) == (rows, K), "%s: an operand [%d, %d] expected, got [%d, %d]" % (what, rows, K, op.rows, op.K))
    _need(op.q.get_device() == t.get_device(), "%s: on %s, the others on %s" % (what, op.q.device, t.device))


def nvfp4_quantize(x: torch.Tensor, rows: Optional[Nvfp4Operand] = None, cols: Optional[Nvfp4Operand] = None,
                   workspace: Optional[torch.Tensor] = None, scales_given: bool = False) -> None:
    """Operands of x [R, C]: `rows` [R, C] receives that of x, `cols` [C, R] that of its transpose; both from one call when both are
    given.  The row scales are computed from the rows, or taken from the operands (scales_given)."""
    ld, code = _matrix(x, "x"), _dtype(x, "x")
    R, C = x.shape
    _need(rows is not None or cols is not None, "rows or cols: an operand to fill")
    if rows is not None:
        _on(rows, R, C, x, "rows")
    if cols is not None:
        _on(cols, C, R, x, "cols")
    B.moe_nvfp4_quantize(x, code, R, C, ld, None if rows is None else rows.struct, None if cols is None else cols.struct,
                         scales_given, workspace)


def nvfp4_matmul(a: Nvfp4Operand, b: Nvfp4Operand, dtype: torch.dtype, workspace: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] of dtype (into `out` when given)."""
    _on(b, b.rows, a.K, a.q, "b")
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.q.device)
    _need(out.shape == (a.rows, b.rows) and out.dtype == dtype and out.get_device() == a.q.get_device(), "out: [M, N] of dtype expected")
    B.moe_nvfp4_matmul(a.struct, b.struct, a.rows, b.rows, a.K, out, _dtype(out, "out"), _matrix(out, "out"), workspace)
    return out


def nvfp4_linear(x: torch.Tensor, W: Nvfp4Operand, workspace: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] times W [N, K] transposed, x quantised row by row: [M, N] of x's type (or of `out`'s)."""
    ld, code = _matrix(x, "x"), _dtype(x, "x")
    M, K = x.shape
    _on(W, W.rows, K, x, "W")
    if out is None:
        out = torch.empty((M, W.rows), dtype=x.dtype, device=x.device)
    _need(out.shape == (M, W.rows) and out.get_device() == x.get_device(), "out: [M, N] expected")
    B.moe_nvfp4_linear(x, code, M, K, ld, W.struct, W.rows, out, _dtype(out, "out"), _matrix(out, "out"), workspace)
    return out
