"""Routing rules, their gradients and dense NVFP4 products on torch tensors.

Each function checks its tensors, allocates its results and makes one call of the library (binding.py); the work is the
library's kernels, on torch's current stream.  None of them synchronises.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import binding as B

# Calls at decode sizes cost the host more than the GPU: the functions below test with few attribute reads and call the
# library's functions directly (binding.py's wrappers would convert every tensor again).
_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = B.load()
    return _lib


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
    status = _library().moe_route_logits(x.data_ptr(), W_r.data_ptr(), None if b is None else b.data_ptr(), T, d, E,
                                         logits.data_ptr(), B._current_stream())
    if status:
        raise B.MoeError("moe_route_logits", status)
    return logits


def route_scores(logits: torch.Tensor, k: int, rule: B.moe_route_rule, bias: Optional[torch.Tensor] = None,
                 scores: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """ids int32 [T, k] (ascending) and weights fp32 [T, k] of logits [T, E] under `rule`; `bias` fp32 [E] takes part in the
    choice only.  Logits of -inf take an expert out of service.  scores fp32 [T, E] and counts int32 [E], when given, receive
    all the scores and the picks per expert."""
    ld = _matrix(logits, "logits")
    code = _dtype(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        _plain(bias, (E,), torch.float32, logits, "bias")
    if scores is not None:
        _plain(scores, (T, E), torch.float32, logits, "scores")
    if counts is not None:
        _plain(counts, (E,), torch.int32, logits, "counts")
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    status = _library().moe_route_scores(logits.data_ptr(), code, ld, None if bias is None else bias.data_ptr(), T, E, k, rule,
                                         ids.data_ptr(), w.data_ptr(), None if scores is None else scores.data_ptr(),
                                         None if counts is None else counts.data_ptr(), B._current_stream())
    if status:
        raise B.MoeError("moe_route_scores", status)
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
    status = _library().moe_route_scores_backward(logits.data_ptr(), code, ld, T, E, k, rule, ids.data_ptr(), dw.data_ptr(),
                                                  None if dscores is None else dscores.data_ptr(), dlogits.data_ptr(), E,
                                                  B._current_stream())
    if status:
        raise B.MoeError("moe_route_scores_backward", status)
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
        status = _library().moe_combine_backward(dy.data_ptr(), y_perm.data_ptr() if need_dw else None, inv_pos.data_ptr(),
                                                 w.data_ptr(), T, k, d, None if dw is None else dw.data_ptr(),
                                                 None if dy_perm is None else dy_perm.data_ptr(), B._current_stream())
        if status:
            raise B.MoeError("moe_combine_backward", status)
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
        self.device = q.get_device()
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
    if op.rows != rows or op.K != K or op.device != t.get_device():
        raise ValueError("%s: an operand [%d, %d] on %s expected, got [%d, %d] on %s" % (what, rows, K, t.device, op.rows, op.K,
                                                                                        op.q.device))


def _output(out: torch.Tensor, M: int, N: int, like: torch.Tensor) -> int:
    _need(out.shape == (M, N) and out.get_device() == like.get_device(), "out: [%d, %d] on %s expected" % (M, N, like.device))
    return _matrix(out, "out")


def _space(ws: Optional[torch.Tensor]) -> tuple:
    return (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)


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
    status = _library().moe_nvfp4_quantize(x.data_ptr(), code, R, C, ld, None if rows is None else rows.struct,
                                           None if cols is None else cols.struct, int(scales_given),
                                           *_space(workspace), B._current_stream())
    if status:
        raise B.MoeError("moe_nvfp4_quantize", status)


def nvfp4_matmul(a: Nvfp4Operand, b: Nvfp4Operand, dtype: torch.dtype, workspace: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] of dtype (into `out` when given)."""
    M, N = a.rows, b.rows
    _on(b, N, a.K, a.q, "b")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=a.q.device)
        ld = N
    else:
        ld = _output(out, M, N, a.q)
        _need(out.dtype == dtype, "out: %s expected" % (dtype,))
    status = _library().moe_nvfp4_matmul(a.struct, b.struct, M, N, a.K, out.data_ptr(), _dtype(out, "out"), ld,
                                         *_space(workspace), B._current_stream())
    if status:
        raise B.MoeError("moe_nvfp4_matmul", status)
    return out


def nvfp4_linear(x: torch.Tensor, W: Nvfp4Operand, workspace: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] times W [N, K] transposed, x quantised row by row: [M, N] of x's type (or of `out`'s)."""
    ld, code = _matrix(x, "x"), _dtype(x, "x")
    M, K = x.shape
    N = W.rows
    _on(W, N, K, x, "W")
    if out is None:
        out, ldy, ycode = torch.empty((M, N), dtype=x.dtype, device=x.device), N, code
    else:
        ldy, ycode = _output(out, M, N, x), _dtype(out, "out")
    status = _library().moe_nvfp4_linear(x.data_ptr(), code, M, K, ld, W.struct, N, out.data_ptr(), ycode, ldy,
                                         *_space(workspace), B._current_stream())
    if status:
        raise B.MoeError("moe_nvfp4_linear", status)
    return out
