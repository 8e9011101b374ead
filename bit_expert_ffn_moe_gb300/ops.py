"""Routing rules, their gradients, dense NVFP4 products, rows between tokens and experts and products in 8-bit integers on torch tensors.

Each function checks its tensors, allocates its results and makes one call of the library, in an extension module; the work is
the library's kernels, on torch's current stream.  None of them synchronises.  Tensors of another device than the current one are
refused (`with torch.cuda.device(...)` makes theirs the current one).  None of them takes part in autograd: gradients come from the
calls that compute them, and backward() through a result raises an error rather than leave its gradient out.  Results in tensors that
were given, weights of int8_weights and the operand of nvfp4_linear are constants.
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
        self.of: Optional[torch.Tensor] = None  # the tensor that it was made of, where it requires a gradient
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
    op.rows, op.K, op.device, op.of = rows, K, index, None
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
    of = x if x.requires_grad and torch.is_grad_enabled() else None
    if rows is not None:
        rows.of = of
    if cols is not None:
        cols.of = of


def nvfp4_matmul(a: Nvfp4Operand, b: Nvfp4Operand, dtype: torch.dtype, workspace: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] of dtype (into `out` when given)."""
    code = _SCALAR_TYPES.get(dtype)
    if code is None:
        raise TypeError("fp32, bf16 or fp16 expected, got %s" % (dtype,))
    y = (_module or _calls()).nvfp4_matmul(a.struct, a.rows, a.K, a.device, b.struct, b.rows, b.K, b.device, a.q, code, workspace, out)
    if out is None and (a.of is not None or b.of is not None):
        y = tied("nvfp4_matmul's gradients are nvfp4_matmul of transposed operands", y, a.of, b.of)
    return y


def nvfp4_linear(x: torch.Tensor, W: Nvfp4Operand, workspace: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] times W [N, K] transposed, x quantised row by row: [M, N] of x's type (or of `out`'s)."""
    y = (_module or _calls()).nvfp4_linear(x, W.struct, W.rows, W.K, W.device, workspace, out)
    if x.requires_grad and out is None:
        y = tied("nvfp4_linear's gradients are nvfp4_matmul of transposed operands", y, x)
    return y


# ------------------------------------------------------------------ rows between tokens and experts

class ExpertOrder:
    """Pairs (token, slot) in the order of (expert, token, slot): offsets int32 [E + 1], inv int32 [T, k] the row of a pair in that
    order, -1 without an expert."""
    __slots__ = ("T", "k", "E", "offsets", "inv")

    def __init__(self, E: int, offsets: torch.Tensor, inv: torch.Tensor):
        self.E, self.offsets, self.inv = E, offsets, inv
        self.T, self.k = inv.shape


def expert_order(ids: torch.Tensor, E: int) -> ExpertOrder:
    """The order by expert of ids int32 [T, k]; an id outside [0, E) has no expert and its pair no row."""
    return ExpertOrder(E, *(_module or _calls()).expert_order(ids, E))


def _asks(*tensors: Optional[torch.Tensor]) -> bool:
    return any(t is not None and t.requires_grad for t in tensors)


def tokens_to_experts(x: torch.Tensor, order: ExpertOrder, w: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows [T k, d] of x [T, d] (bf16, fp16, fp32) in expert order, times w fp32 [T, k] when given.  Rows behind the last pair with an
    expert are not written."""
    rows = (_module or _calls()).move_rows(True, x, order.inv, w, out)
    if out is None and _asks(x, w):
        rows = tied("tokens_to_experts' gradients are tokens_to_experts_backward", rows, x, w)
    return rows


def tokens_to_experts_backward(drows: torch.Tensor, order: ExpertOrder, x: Optional[torch.Tensor] = None,
                               w: Optional[torch.Tensor] = None, need_dx: bool = True
                               ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of tokens_to_experts: dx [T, d] and, where x and w are given, dw fp32 [T, k] (else None)."""
    return (_module or _calls()).move_backward(False, drows, order.inv, x, w, need_dx)


def experts_to_tokens(rows: torch.Tensor, order: ExpertOrder, w: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T, d]: the sum over a token's slots of its rows [T k, d] (bf16, fp16, fp32), times w fp32 [T, k] when given."""
    y = (_module or _calls()).move_rows(False, rows, order.inv, w, out)
    if out is None and _asks(rows, w):
        y = tied("experts_to_tokens' gradients are experts_to_tokens_backward", y, rows, w)
    return y


def experts_to_tokens_backward(dy: torch.Tensor, order: ExpertOrder, rows: Optional[torch.Tensor] = None,
                               w: Optional[torch.Tensor] = None, need_drows: bool = True
                               ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of experts_to_tokens: drows [T k, d] (rows behind the last pair with an expert are not written) and, where rows and w are
    given, dw fp32 [T, k] (else None)."""
    return (_module or _calls()).move_backward(True, dy, order.inv, rows, w, need_drows)


# ------------------------------------------------------------------ products in 8-bit integers

_DTYPES = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_F16}


class Int8Weights:
    """One matrix [N, K] of 8-bit whole numbers, or those of E experts, as the products read them: tiles q (int8 or uint8,
    binding.moe_int8_weights_bytes a matrix) and fp32 scales s, one for each row.  int8_weights makes them of matrices."""

    def __init__(self, N: int, K: int, q: torch.Tensor, s: torch.Tensor):
        n = B.moe_int8_weights_bytes(N, K)
        _need(n > 0, "unsupported shape [%d, %d]" % (N, K))
        _need(q.is_cuda and q.dtype in (torch.int8, torch.uint8) and q.is_contiguous() and q.numel() > 0 and q.numel() % n == 0,
              "q: contiguous CUDA bytes, a multiple of %d, expected" % n)
        self.E = q.numel() // n
        _need(s.dtype == torch.float32 and s.device == q.device and s.is_contiguous() and s.numel() == self.E * N,
              "s: contiguous fp32 [%d, %d] expected" % (self.E, N))
        self.N, self.K, self.q, self.s = N, K, q, s
        self.struct = B.moe_int8_weights(q.data_ptr(), s.data_ptr())
        self.args = (self.struct, self.E, N, K, q.get_device())  # as the extension module takes them

    def values(self) -> torch.Tensor:
        """The numbers they stand for, fp32 [E, N, K]."""
        KT, NT = -(-self.K // 64), -(-self.N // 128)
        t = self.q.view(torch.int8).view(self.E, NT, KT, 4, 128, 16).permute(0, 1, 4, 2, 3, 5)
        return t.reshape(self.E, NT * 128, KT * 64)[:, :self.N, :self.K].float() * self.s.view(self.E, self.N, 1)


def int8_weights(w: torch.Tensor, scales: Optional[torch.Tensor] = None, up: Optional[torch.Tensor] = None,
                 up_scales: Optional[torch.Tensor] = None) -> Int8Weights:
    """Weights of w [N, K] or [E, N, K]: int8 with fp32 scales [.., N], or fp32, bf16 or fp16, which are quantised row by row.  With
    `up` (of w's shape, type) they are those of a gated product: w the gate, 2 N rows in all."""
    parts = [(w, scales)] if up is None else [(w, scales), (up, up_scales)]
    _need(w.dim() in (2, 3) and w.is_cuda, "w: a CUDA tensor [N, K] or [E, N, K] expected")
    _need_current(w.device, "w")
    E, (N, K) = (1 if w.dim() == 2 else w.shape[0]), w.shape[-2:]
    bytes_ = B.moe_int8_weights_bytes(N * len(parts), K)
    _need(bytes_ > 0 and N > 0 and E > 0, "unsupported shape %s" % (tuple(w.shape),))
    _need(up is not None or up_scales is None, "up_scales without up")
    W = Int8Weights(N * len(parts), K, torch.empty(E * bytes_, dtype=torch.uint8, device=w.device),
                    torch.empty(E * N * len(parts), dtype=torch.float32, device=w.device))
    for i, (m, s) in enumerate(parts):
        _need(m.shape == w.shape and m.dtype == w.dtype and m.device == w.device and m.is_contiguous(), "up: contiguous, as w, expected")
        if m.dtype == torch.int8:
            _need(s is not None and s.shape == w.shape[:-1] and s.dtype == torch.float32 and s.device == w.device and s.is_contiguous(),
                  "scales: contiguous fp32 %s expected" % (tuple(w.shape[:-1]),))
            B.moe_int8_weights_layout(m, s, E, N, K, K, i, len(parts), W.N, W.struct)
        else:
            _need(m.dtype in _DTYPES and s is None, "w: int8 with scales, or fp32, bf16 or fp16 without, expected")
            B.moe_int8_weights_quantize(m, _DTYPES[m.dtype], E, N, K, K, i, len(parts), W.N, W.struct)
    return W


class Int8Rows:
    """Rows [M, K] of activations in 8 bits, of no expert or in an order's: what int8_quantize makes and int8_matmul takes."""

    def __init__(self, M: int, K: int, order: Optional[ExpertOrder], device: int):
        self.M, self.K, self.order = M, K, order
        self.q, self.s, q, s, self.room = (_module or _calls()).int8_room(M, order.E if order else 0, K, device)
        self.struct = B.moe_int8_rows(q, s, self.room)
        self.of: Optional[torch.Tensor] = None  # the tensor that they were made of, where it requires a gradient

    def values(self) -> torch.Tensor:
        """The numbers they stand for, fp32 [room, K] (rows that no row was put into: anything)."""
        r = torch.arange(self.room, device=self.q.device)
        at = torch.arange(8, device=self.q.device)[None, :] ^ (r[:, None] % 8)
        t = self.q.view(-1, self.room, 8, 8)
        t = t.gather(2, at[None, :, :, None].expand_as(t))
        return t.permute(1, 0, 2, 3).reshape(self.room, -1)[:, :self.K].float() * self.s[:, None]


def int8_quantize(x: torch.Tensor, order: Optional[ExpertOrder] = None, ordered: bool = False) -> Int8Rows:
    """Rows of x [M, K] in 8 bits; with an order those of its tokens x [T, K], spread into expert order, or, `ordered`, of x [T k, K] in
    expert order already."""
    _need(x.dim() == 2 and x.is_cuda, "x: a CUDA matrix expected")
    M = x.shape[0] if order is None else order.T * order.k
    _need(order is None or x.shape[0] == (M if ordered else order.T), "x: another number of rows than the order's expected")
    rows = Int8Rows(M, x.shape[1], order, x.get_device())
    inv, offsets, E = (None, None, 0) if order is None else (None if ordered else order.inv, order.offsets, order.E)
    (_module or _calls()).int8_quantize(x, inv, offsets, E, rows.struct)
    if x.requires_grad and torch.is_grad_enabled():
        rows.of = x
    return rows


def int8_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of int8_linear and int8_matmul for up to M rows, initialised."""
    n = B.moe_int8_workspace_size(M, N, K)
    _need(n > 0, "unsupported shape M=%d N=%d K=%d" % (M, N, K))
    _need_current(torch.device(device), "workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    B.moe_workspace_init(ws)
    return ws


def int8_matmul(rows: Int8Rows, W: Int8Weights, dtype: torch.dtype, workspace: torch.Tensor, gated: bool = False,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rows [M, K] times W [N, K] transposed, or each expert's rows times its matrix: [M, N] of dtype, gated [M, N / 2] (rows behind the last
    pair with an expert are not written).  Sums are exact where they stay within 2^24 on their way, always for K <= 1032, and beyond that
    fp32 sums: a row's last bits can then depend on how many rows there are."""
    code = _SCALAR_TYPES.get(dtype)
    if code is None:
        raise TypeError("fp32, bf16 or fp16 expected, got %s" % (dtype,))
    offsets, E = (None, 0) if rows.order is None else (rows.order.offsets, rows.order.E)
    y = (_module or _calls()).int8_matmul(rows.struct, rows.s, rows.M, rows.K, offsets, E, *W.args, code, workspace, gated, out)
    if out is None and rows.of is not None:
        y = tied("int8_matmul's input gradient is a product with the transposed weights", y, rows.of)
    return y


def int8_linear(x: torch.Tensor, W: Int8Weights, workspace: torch.Tensor, gated: bool = False,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] times W [N, K] transposed, x quantised row by row: [M, N] of x's type (or of `out`'s), gated [M, N / 2]."""
    y = (_module or _calls()).int8_linear(x, *W.args, workspace, gated, out)
    if out is None and x.requires_grad:
        y = tied("int8_linear's input gradient is int8_linear of the transposed weights", y, x)
    return y


def int8_experts_workspace(T: int, k: int, d: int, I: int, E: int, dtype: torch.dtype = torch.bfloat16,  # noqa: E741
                           device="cuda") -> torch.Tensor:
    """Workspace of int8_experts for up to T tokens of k slots, initialised."""
    n = B.moe_int8_experts_workspace_size(T, d, E, k, I, _DTYPES[dtype])
    _need(n > 0, "unsupported shape T=%d k=%d d=%d I=%d E=%d" % (T, k, d, I, E))
    _need_current(torch.device(device), "workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    B.moe_workspace_init(ws)
    return ws


def int8_experts(x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, up: Int8Weights, down: Int8Weights, workspace: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A sparse layer behind its router: y [T, d] of x [T, d], ids int32 [T, k] and w fp32 [T, k]; `up` the gated weights [E, 2 I, d],
    `down` [E, d, I].  The same as int8_quantize, int8_matmul (gated, in x's type), int8_quantize, int8_matmul and experts_to_tokens."""
    y = (_module or _calls()).int8_experts(x, ids, w, *up.args, *down.args, workspace, out)
    if out is None and _asks(x, w):
        y = tied("int8_experts computes no gradients; the weights' is experts_to_tokens_backward", y, x, w)
    return y
