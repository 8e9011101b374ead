"""A latent sparse block: an NVFP4 projection narrows the tokens, a routing rule sends them to frozen 4-bit experts, a second
NVFP4 projection widens the weighted sum -- and the router's gradient, to tune it over those experts.

The shared latent projections are those of the Muse Spark Open explainer, section 9, in the experts' own format; the routed
part runs the library's step calls with the ids and weights that the rule chose.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B
from . import ops
from .layer import DeviceLayer, make_workspace


class Nvfp4Linear:
    """y = x W^T with W [N, K] quantised once, row by row; with `gradients` also its transpose, for dx = dy W."""

    def __init__(self, W: torch.Tensor, max_rows: int, gradients: bool = False):
        self.N, self.K = W.shape
        self.workspace = ops.nvfp4_workspace(max_rows, self.N, self.K, W.device)
        self.forward_operand = ops.nvfp4_operand(self.N, self.K, W.device)
        self.transposed = ops.nvfp4_operand(self.K, self.N, W.device) if gradients else None
        ops.nvfp4_quantize(W, self.forward_operand, self.transposed, self.workspace)
        self.back_workspace = ops.nvfp4_workspace(max_rows, self.K, self.N, W.device) if gradients else None

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return ops.nvfp4_linear(x, self.forward_operand, self.workspace)

    def input_gradient(self, dy: torch.Tensor) -> torch.Tensor:
        if self.transposed is None:
            raise ValueError("input_gradient: built without gradients")
        return ops.nvfp4_linear(dy, self.transposed, self.back_workspace)


class LatentBlock:
    """W_out experts(W_in x): `layer` holds the experts and the router's matrix (d, E, k, I; the bias of its logits is not used), `rule`
    the routing rule, `balance` an fp32 [E] bias of the choice, which balance_step moves in place.  Calls take up to max_tokens tokens; the
    expert path is that of MXFP4 activations."""

    def __init__(self, layer: DeviceLayer, rule: B.moe_route_rule, W_in: torch.Tensor, W_out: torch.Tensor, max_tokens: int,
                 balance: Optional[torch.Tensor] = None, gradients: bool = False):
        cfg = layer.cfg
        self.layer, self.rule, self.balance = layer, rule, balance
        self.narrow = Nvfp4Linear(W_in, max_tokens)
        self.widen = Nvfp4Linear(W_out, max_tokens, gradients)
        if self.narrow.N != cfg.d or self.widen.K != cfg.d:
            raise ValueError("W_in [%d, .] and W_out [., %d] expected" % (cfg.d, cfg.d))
        self.W_r = layer.W_r.clone()
        self.counts = torch.zeros(cfg.E, dtype=torch.int32, device=W_in.device)
        self.max_tokens = max_tokens
        T, k, E = max_tokens, cfg.k, cfg.E
        rows = B.moe_padded_rows(T, k, E)
        i32, u8 = dict(dtype=torch.int32, device=W_in.device), dict(dtype=torch.uint8, device=W_in.device)
        self.ws = make_workspace(T, cfg.d, E, k, cfg.I, B.MOE_ACT_MXFP4, W_in.device)
        self.offsets, self.perm, self.inv = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
        self.picked = torch.empty(E, **i32)
        self.xa, self.xa_s = torch.empty((rows, cfg.d // 2), **u8), torch.empty(B.moe_mxfp4_mma_scale_bytes(rows, cfg.d), **u8)
        self.h, self.h_s = torch.empty((rows, cfg.I // 2), **u8), torch.empty(B.moe_mxfp4_mma_scale_bytes(rows, cfg.I), **u8)

    def experts(self, z: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        """Outputs bf16 [T k, d] of the chosen experts, grouped by expert (self.inv: the row of each (token, slot))."""
        cfg, W, T = self.layer.cfg, self.layer.weights, z.shape[0]
        shape = (T, cfg.d, cfg.E, cfg.k, cfg.I)
        y_perm = torch.empty((T * cfg.k, cfg.d), dtype=torch.bfloat16, device=z.device)
        if T == 0:
            return y_perm
        B.moe_permute(z, ids, T, cfg.d, cfg.E, cfg.k, B.MOE_ACT_MXFP4, self.picked, self.offsets, self.perm, self.inv, self.xa,
                      self.xa_s, self.ws)
        B.moe_expert_up_swiglu(None, self.xa, self.xa_s, B.MOE_ACT_MXFP4, self.perm, self.offsets, *shape, W, self.h, self.h_s,
                               self.ws)
        B.moe_expert_down(self.h, self.h_s, B.MOE_ACT_MXFP4, self.perm, self.offsets, *shape, W, y_perm, self.ws)
        return y_perm

    def __call__(self, x: torch.Tensor) -> Tuple[torch.Tensor, dict]:
        """y bf16 [T, D] of bf16 x [T, D], and what router_gradient needs of this pass."""
        y, past = self._pass(x)
        return ops.tied("LatentBlock computes its router's gradient alone (router_gradient)", y, x), past

    @torch.no_grad()
    def _pass(self, x: torch.Tensor) -> Tuple[torch.Tensor, dict]:
        cfg, T = self.layer.cfg, x.shape[0]
        if T > self.max_tokens:
            raise ValueError("at most %d tokens, got %d" % (self.max_tokens, T))
        z = self.narrow(x)
        logits = ops.route_logits(z, self.W_r)
        ids, w = ops.route_scores(logits, cfg.k, self.rule, self.balance, counts=self.counts)
        y_perm = self.experts(z, ids)
        s = torch.empty((T, cfg.d), dtype=torch.bfloat16, device=x.device)
        B.moe_combine(y_perm, self.inv, w, T, cfg.k, cfg.d, s)
        return self.widen(s), dict(z=z, logits=logits, ids=ids, w=w, y_perm=y_perm, inv=self.inv[:T * cfg.k].clone())

    @torch.no_grad()
    def router_gradient(self, dy: torch.Tensor, past: dict) -> torch.Tensor:
        """Gradient fp32 [E, d] of the router's matrix from that of y, experts and projections held fixed."""
        ds = self.widen.input_gradient(dy)
        dw, _ = ops.combine_backward(ds, past["y_perm"], past["inv"], past["w"], need_dy_perm=False)
        dlogits = ops.route_scores_backward(past["logits"], past["ids"], dw, self.rule)
        return dlogits.T @ past["z"].float()

    def balance_step(self, rate: float) -> None:
        """Moves the balance bias against the load of the last pass: up for experts below the mean, down above."""
        if self.balance is None:
            raise ValueError("balance_step: built without a balance bias")
        load = self.counts.float()
        self.balance += rate * torch.sign(load.mean() - load)


class Int8Linear:
    """y = x W^T with W [N, K] (int8 with a scale per row, or numbers to quantise), x quantised row by row."""

    def __init__(self, W: torch.Tensor, max_rows: int, scales: Optional[torch.Tensor] = None):
        self.weights = ops.int8_weights(W, scales)
        self.workspace = ops.int8_workspace(max_rows, self.weights.N, self.weights.K, W.device)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return ops.int8_linear(x, self.weights, self.workspace)


class Int8Experts:
    """A sparse layer in 8-bit integers behind any routing rule: `up` the gated weights [E, 2 I, d], `down` [E, d, I]
    (ops.int8_weights).  Calls take up to max_tokens tokens of k slots, of dtype (or another type of no more bytes)."""

    def __init__(self, up: ops.Int8Weights, down: ops.Int8Weights, max_tokens: int, k: int, dtype: torch.dtype = torch.bfloat16):
        if up.E != down.E or up.K != down.N or up.N != 2 * down.K:
            raise ValueError("up [E, 2 I, d] and down [E, d, I] expected")
        self.up, self.down, self.max_tokens, self.k = up, down, max_tokens, k
        self.workspace = ops.int8_experts_workspace(max_tokens, k, up.K, down.K, up.E, dtype, up.q.device)

    def _check(self, x: torch.Tensor, ids: torch.Tensor) -> None:
        if x.shape[0] > self.max_tokens or ids.dim() != 2 or ids.shape[1] != self.k:
            raise ValueError("at most %d tokens of %d slots expected" % (self.max_tokens, self.k))

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
        """y [T, d] of x [T, d] and the routing ids int32 [T, k], w fp32 [T, k]."""
        self._check(x, ids)
        return ops.int8_experts(x, ids, w, self.up, self.down, self.workspace)

    def outputs(self, x: torch.Tensor, ids: torch.Tensor) -> Tuple[torch.Tensor, ops.ExpertOrder]:
        """The experts' outputs [T k, d] in expert order, and that order: the layer without its weighted sum, for the gradient of the
        routing weights (ops.experts_to_tokens_backward)."""
        self._check(x, ids)
        order = ops.expert_order(ids, self.up.E)
        h = ops.int8_matmul(ops.int8_quantize(x, order), self.up, x.dtype, self.workspace, gated=True)
        return ops.int8_matmul(ops.int8_quantize(h, order, ordered=True), self.down, x.dtype, self.workspace), order
