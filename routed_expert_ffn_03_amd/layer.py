"""One routed-expert layer call on caller-owned buffers: the C entry points
in order on one stream.  Buffers are allocated once per shape with
torch (device memory only); the call itself allocates nothing.
"""
from __future__ import annotations

import torch

from . import binding as B


class MoELayerBuffers:
    """Outputs, intermediates and workspace of one layer shape."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, wfmt: int = B.MOE_WFMT_BF16,
                 device: str | torch.device = "cuda"):
        self.T, self.E, self.k, self.H, self.I, self.wfmt = T, E, k, H, I, wfmt
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_ids = torch.empty((T, k), **i32)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.expert_counts = torch.empty((E,), **i32)
        self.expert_offsets = torch.empty((E + 1,), **i32)
        self.sorted_pair = torch.empty((T * k,), **i32)
        self.pair_to_sorted = torch.empty((T * k,), **i32)
        self.y_sorted = torch.empty((T * k, H), dtype=torch.float16, device=device)
        self.out = torch.empty((T, H), dtype=torch.float32, device=device)
        ws = B.moe_workspace_size(T, E, k, H, I, wfmt)
        if ws == 0:
            raise ValueError("unsupported layer shape")
        self.workspace = torch.empty((ws,), dtype=torch.uint8, device=device)

    def forward(self, logits: torch.Tensor, x: torch.Tensor, w: dict, fat_threshold: int = B.DEFAULT_FAT_THRESHOLD,
                stream=None) -> torch.Tensor:
        """route -> permute -> grouped FFN -> combine; returns ``out`` (fp32 [T, H]).

        Decode-sized batches (T <= 64) run route, permute and the FFN plan as
        one launch (moe_route_permute_plan); the results are the same."""
        if self.T <= 64:
            B.moe_route_permute_plan(logits, self.k, self.H, self.I, self.topk_ids, self.topk_w, self.expert_counts,
                                     self.expert_offsets, self.sorted_pair, self.pair_to_sorted, self.workspace,
                                     fat_threshold=fat_threshold, wfmt=self.wfmt, stream=stream)
            B.moe_ffn_gate_up(x, w["gate"], w["up"], self.sorted_pair, self.E, self.k, self.workspace,
                              s_gate=w.get("gate_scale"), s_up=w.get("up_scale"), fat_threshold=fat_threshold,
                              wfmt=self.wfmt, stream=stream)
            B.moe_ffn_down(w["down"], self.T, self.E, self.k, self.I, self.y_sorted, self.workspace,
                           s_down=w.get("down_scale"), fat_threshold=fat_threshold, wfmt=self.wfmt, stream=stream)
        else:
            B.moe_route_topk(logits, self.k, self.topk_ids, self.topk_w, self.expert_counts, stream)
            B.moe_permute(self.topk_ids, self.E, self.expert_offsets, self.sorted_pair, self.pair_to_sorted,
                          self.workspace, stream)
            B.moe_grouped_ffn(x, w["gate"], w["up"], w["down"], self.expert_offsets, self.sorted_pair, self.k,
                              self.y_sorted, self.workspace, s_gate=w.get("gate_scale"), s_up=w.get("up_scale"),
                              s_down=w.get("down_scale"), fat_threshold=fat_threshold, wfmt=self.wfmt, stream=stream)
        B.moe_combine(self.y_sorted, self.topk_w, self.pair_to_sorted, self.out, stream)
        return self.out


class RouterGradBuffers:
    """Outputs and workspace of one router training step on a ``MoELayerBuffers`` layer whose
    experts are frozen: the balance loss of its routing, and the gradient of the layer's output
    and of that loss with respect to the router logits."""

    def __init__(self, layer: MoELayerBuffers, groups: int = 1, expert_grad: bool = False):
        T, E, k = layer.T, layer.E, layer.k
        dev = layer.out.device
        f32 = dict(dtype=torch.float32, device=dev)
        self.layer = layer
        self.expert_counts = torch.empty((groups, E), dtype=torch.int32, device=dev)
        self.prob_mean = torch.empty((groups, E), **f32)
        self.group_scale = torch.empty((groups,), **f32)
        self.loss = torch.empty((1,), **f32)
        self.d_topk_w = torch.empty((T, k), **f32)
        self.d_logits = torch.empty((T, E), **f32)
        self.d_y_sorted = torch.empty_like(layer.y_sorted) if expert_grad else None
        ws = B.moe_balance_workspace_size(T, E, groups)
        if ws == 0:
            raise ValueError("unsupported groups: they must divide the tokens")
        self.workspace = torch.empty((ws,), dtype=torch.uint8, device=dev)

    def balance_loss(self, logits: torch.Tensor, coef: float, token_mask: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
        """The balance loss (fp32 [1]) of the layer's last ``forward`` on ``logits``."""
        B.moe_balance_loss(logits, self.layer.topk_ids, self.expert_counts, self.prob_mean, self.group_scale,
                           self.loss, self.workspace, token_mask=token_mask, coef=coef, stream=stream)
        return self.loss

    def backward(self, logits: torch.Tensor, d_out: torch.Tensor, d_loss: torch.Tensor | None = None,
                 token_mask: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """``d_logits`` (fp32 [T, E]) from the gradient of the layer's output ``d_out`` (fp32 [T, H]) and,
        where ``d_loss`` (fp32 [1]) is given, of the balance loss last computed by ``balance_loss`` with
        the same ``token_mask``.  With ``expert_grad`` also fills ``d_y_sorted``."""
        b = self.layer
        B.moe_combine_backward(d_out, b.y_sorted, b.topk_w, b.pair_to_sorted, d_y_sorted=self.d_y_sorted,
                               d_topk_w=self.d_topk_w, stream=stream)
        on = d_loss is not None
        B.moe_route_backward(logits, b.topk_ids, b.topk_w, self.d_logits, d_topk_w=self.d_topk_w,
                             expert_counts=self.expert_counts if on else None,
                             group_scale=self.group_scale if on else None, d_loss=d_loss,
                             token_mask=token_mask if on else None, stream=stream)
        return self.d_logits
