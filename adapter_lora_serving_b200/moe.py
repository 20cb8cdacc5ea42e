"""One adapted mixture-of-experts layer, from routing logits to the layer's output,
over the library's entry points.

Sources: spark_model/lora/expert_apply.rs, module text (the order of a routed
layer: router delta before top-k; base grouped product, fold of gate/up, silu_mul,
down product, fold of down, weighted un-permute), and spark_model/lora/target.rs
(the router, expert gate/up and expert down targets).

    logits  += router delta                       lora_apply_router
    ids, w   = top-k of the scores                lora_route_experts
    rows     = (token, choice) pairs by expert    lora_group_experts
    x_s, x_q = x of every row, in bf16 and 4 bits lora_mx_quantize
    gu       = x_q  W_gate_up[e]^T                lora_mx_expert_linear
    gu      += adapters' delta of x_s             lora_expert_apply
    a, a_q   = silu(gate) * up, in both           lora_mx_quantize
    y        = a_q  W_down[e]^T                   lora_mx_expert_linear
    y       += adapters' delta of a               lora_expert_apply
    out      = residual + sum_j w y               lora_combine_experts

Only argument marshalling and the layer's buffers live here; the arithmetic is the
library's kernels.  Nothing synchronises with the host and the buffers are the
layer's own, so a call can be captured in a CUDA graph; calls that share a layer
must be ordered (one stream, or events).
"""
from __future__ import annotations

from . import lora as L


class ExpertAdapters:
    """The expert adapters of a layer's slots for one projection: the pair pool
    a [num_pairs, S*R, in], b [num_pairs, out, R] (bf16), pair_index
    [slots * num_experts] (int32, -1 = not adapted), ranks and scalings [slots],
    as lora_expert_apply takes them."""

    def __init__(self, a, b, pair_index, ranks, scalings):
        self.a, self.b, self.pair_index = a, b, pair_index
        self.ranks, self.scalings = ranks, scalings
        self.num_pairs, self.R = int(b.shape[0]), int(b.shape[2])
        self.slots = int(ranks.numel())


class RouterAdapters:
    """The router adapters of a layer's slots: a [slots, R, hidden], b [slots,
    num_experts, R] (bf16), ranks and scalings [slots], as lora_apply_router takes
    them."""

    def __init__(self, a, b, ranks, scalings):
        self.a, self.b, self.ranks, self.scalings = a, b, ranks, scalings
        self.slots, self.R = int(a.shape[0]), int(a.shape[1])


class MoeLayer:
    """Weights, adapters and buffers of one routed layer for at most max_tokens
    tokens a call.

    gate_up: (codes [E, 2 * inter, hidden / 2], scales [E, 2 * inter, hidden / 32]),
    down: (codes [E, hidden, inter / 2], scales [E, hidden, inter / 32]), uint8 on
    the device, as lora_mx_quantize writes them; rows of gate_up: gate, then up.
    gate_up_adapters, down_adapters: ExpertAdapters or None; router_adapters:
    RouterAdapters or None.  routing: keyword arguments of lora_route_experts
    (score, bias, num_groups, top_groups, group_score, renormalize, scale)."""

    def __init__(self, max_tokens, hidden, inter, num_experts, top_k, gate_up, down,
                 gate_up_adapters=None, down_adapters=None, router_adapters=None, **routing):
        import torch
        if max_tokens <= 0 or top_k <= 0 or num_experts <= 0:
            raise ValueError("max_tokens, top_k and num_experts must be positive")
        if hidden <= 0 or inter <= 0 or hidden % 32 or inter % 32:
            raise ValueError(f"hidden {hidden} and inter {inter} must be positive multiples of 32")
        self.max_tokens, self.hidden, self.inter = max_tokens, hidden, inter
        self.num_experts, self.top_k = num_experts, top_k
        self.gate_up, self.down = gate_up, down
        self.gate_up_adapters, self.down_adapters = gate_up_adapters, down_adapters
        self.router_adapters = router_adapters
        self.bias = routing.pop("bias", None)
        self.routing = routing
        self.device = gate_up[0].device
        for ad, slices, n_in, out in ((gate_up_adapters, 2, hidden, 2 * inter),
                                      (down_adapters, 1, inter, hidden)):
            if ad is not None:
                self._check_adapters(ad, "expert", ad.num_pairs * slices * ad.R * n_in,
                                     ad.num_pairs * out * ad.R, ad.slots * num_experts)
        if router_adapters is not None:
            n = router_adapters.slots * router_adapters.R
            self._check_adapters(router_adapters, "router", n * hidden, n * num_experts, 0)
        rows = max_tokens * top_k

        def empty(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=self.device)

        bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
        self.topk_ids, self.topk_weights = empty(i32, rows), empty(torch.float32, rows)
        self.expert_offsets = empty(i32, num_experts + 1)
        self.row_token, self.pair_row, self.row_slot = (empty(i32, rows) for _ in range(3))
        self.x_sorted = empty(bf16, rows, hidden)
        self.x_codes, self.x_scales = empty(u8, rows, hidden // 2), empty(u8, rows, hidden // 32)
        self.gate_up_out = empty(bf16, rows, 2 * inter)
        self.act = empty(bf16, rows, inter)
        self.act_codes, self.act_scales = empty(u8, rows, inter // 2), empty(u8, rows, inter // 32)
        self.down_out = empty(bf16, rows, hidden)
        # the expert folds' and the router fold's workspaces (the latter's first
        # 4096 bytes must start out zeroed)
        need = [L.lora_workspace_bytes(L.LORA_OP_EXPERT_APPLY, rows, num_experts, ad.R, slices)
                for ad, slices in ((gate_up_adapters, 2), (down_adapters, 1)) if ad is not None]
        self.fold_bytes = max(need, default=0)
        self.fold_ws = empty(u8, self.fold_bytes) if self.fold_bytes else None
        self.router_bytes = 0
        if router_adapters is not None:
            # by the number of tokens: the regime, and with it the need, changes
            self.router_bytes = max(
                L.lora_workspace_bytes(L.LORA_OP_APPLY_LINEAR, t, router_adapters.slots,
                                       router_adapters.R, 1)
                for t in {max_tokens, min(max_tokens, 8192), min(max_tokens, 1024)})
        self.router_ws = (torch.zeros(self.router_bytes, dtype=u8, device=self.device)
                          if self.router_bytes else None)

    def _check_adapters(self, ad, what, of_a, of_b, of_index):
        """The folds' entry points take addresses: what stands behind these is looked
        at here, once."""
        import torch
        bf16 = torch.bfloat16
        for name, dtype, n in (("a", bf16, of_a), ("b", bf16, of_b),
                               ("ranks", torch.int32, ad.slots),
                               ("scalings", torch.float32, ad.slots),
                               ("pair_index", torch.int32, of_index)):
            t = getattr(ad, name, None)
            if t is None or t.__class__ is int:
                continue
            if t.dtype is not dtype or not t.is_contiguous() or t.numel() < n or t.device != self.device:
                raise ValueError(f"{name} of the {what} adapters: {t.dtype} {tuple(t.shape)} on "
                                 f"{t.device}, not {n} contiguous {dtype} on {self.device}")

    def _check_inputs(self, T, x, gate_logits, out, token_slot, token_order, slot_indptr,
                      residual, flags):
        """Every argument, before the first kernel: the router fold, which runs first,
        takes addresses."""
        op, E = "MoeLayer.forward", self.num_experts
        if x.numel() != T * self.hidden:
            L._refuse(op, f"x has {x.numel() // T} features a token, the layer {self.hidden}")
        for name, t, n in (("gate_logits", gate_logits, E), ("out", out, self.hidden),
                           ("residual", residual, self.hidden)):
            if t is not None and t.__class__ is not int and t.dim() == 2 and t.shape[1] != n:
                L._refuse(op, f"{name} has rows of {t.shape[1]}, not of {n}")
        bf16, i32, rt = L.LORA_TYPE_BF16, "int32", self.router_adapters
        of_logits = bf16
        if rt is None:   # the routing takes logits of any LORA_TYPE_*
            of_logits = L._type_of(op, "gate_logits", gate_logits, None)
            token_order = slot_indptr = None
        n = T * self.hidden
        L._pointers(op, (x, gate_logits, out, residual, token_slot, token_order, slot_indptr, flags),
                    (bf16, of_logits, bf16, bf16, i32, i32, i32, i32),
                    (n, T * E, n, n, T, 0, rt.slots + 1 if rt is not None else 0, 1),
                    ("x", "gate_logits", "out", "residual", "token_slot", "token_order",
                     "slot_indptr", "err_flags"))

    def forward(self, x, gate_logits, out, token_slot=None, token_order=None, slot_indptr=None,
                residual=None, err_flags=None, stream=None):
        """out [T, hidden] = residual + the layer of x [T, hidden] (bf16) routed by
        gate_logits [T, num_experts] (bf16, and the router delta is added in place;
        without router adapters fp16 or fp32 too).
        token_slot [T] int32 (-1 = no adapter) is needed with expert adapters;
        token_order and slot_indptr (CSR by slot) with router adapters."""
        import torch
        T, k, E = int(x.shape[0]), self.top_k, self.num_experts
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, and room for {self.max_tokens}")
        if x.device != self.device:
            raise ValueError(f"x is on {x.device}, the layer on {self.device}")
        if token_slot is None and (self.gate_up_adapters or self.down_adapters):
            raise ValueError("expert adapters need token_slot")
        if (token_order is None or slot_indptr is None) and self.router_adapters:
            raise ValueError("router adapters need token_order and slot_indptr")
        if T == 0:
            return out
        self._check_inputs(T, x, gate_logits, out, token_slot, token_order, slot_indptr, residual,
                           err_flags)
        with torch.cuda.device(self.device):
            self._forward(x, gate_logits, out, T, k, E, token_slot, token_order, slot_indptr,
                          residual, err_flags, stream)
        return out

    def _forward(self, x, gate_logits, out, T, k, E, token_slot, token_order, slot_indptr,
                 residual, flags, stream):
        rows = T * k
        kw = dict(err_flags=flags, stream=stream)
        rt = self.router_adapters
        if rt is not None:
            L.lora_apply_router(x, gate_logits, rt.a, rt.b, rt.ranks, rt.scalings, token_order,
                                slot_indptr, T, self.hidden, rt.slots, rt.R, E,
                                workspace=self.router_ws, workspace_bytes=self.router_bytes, **kw)
        L.lora_route_experts(gate_logits, self.bias, self.topk_ids, self.topk_weights, T, E, k,
                             **self.routing, **kw)
        L.lora_group_experts(self.topk_ids, token_slot, self.expert_offsets, self.row_token,
                             self.pair_row, self.row_slot if token_slot is not None else None, T,
                             k, E, **kw)
        count = self.expert_offsets[E:]
        L.lora_mx_quantize(x, self.x_codes, self.x_scales, rows, self.hidden,
                           row_index=self.row_token, row_count=count, rows_out=self.x_sorted, **kw)
        self._product(self.x_codes, self.x_scales, self.gate_up, self.gate_up_out, rows,
                      self.hidden, 2 * self.inter, kw)
        self._fold(self.gate_up_adapters, self.x_sorted, self.gate_up_out, rows, self.hidden,
                   (self.inter, self.inter), kw)
        L.lora_mx_quantize(self.gate_up_out, self.act_codes, self.act_scales, rows, self.inter,
                           row_count=count, rows_out=self.act, activation=L.LORA_ACT_SILU_MUL, **kw)
        self._product(self.act_codes, self.act_scales, self.down, self.down_out, rows, self.inter,
                      self.hidden, kw)
        self._fold(self.down_adapters, self.act, self.down_out, rows, self.inter, (self.hidden,),
                   kw)
        L.lora_combine_experts(self.down_out, self.pair_row, self.topk_weights, residual, out, T,
                               k, rows, self.hidden, **kw)

    def _product(self, codes, scales, weight, y, rows, n_in, n_out, kw):
        L.lora_mx_expert_linear(codes, scales, weight[0], weight[1], self.expert_offsets, y, rows,
                                n_in, n_out, self.num_experts, **kw)

    def _fold(self, ad, x, y, rows, n_in, out_slices, kw):
        if ad is None:
            return
        L.lora_expert_apply(x, y, ad.a, ad.b, ad.pair_index, ad.ranks, ad.scalings, self.row_slot,
                            self.expert_offsets, rows, n_in, self.num_experts, ad.slots,
                            ad.num_pairs, ad.R, out_slices, workspace=self.fold_ws,
                            workspace_bytes=self.fold_bytes, **kw)
