"""A transformer block's feed-forward half around the MoE layer: the norm
before it, the layer, and the end of the block (post norm, gate, residual and
the norm that follows), as a training step and as a step over the few tokens
of a decode batch with 4-bit expert weights.

    h   = N(x; w_pre)
    y   = moe_layer(h)                       routed by h w_router + offset
    out = res_scale * x + gate * N(y; w_post)
    h_next = N(out; w_next)

The arithmetic is in the library's kernels (include/moe.h); this module only
sequences them and owns their buffers.  The router's own linear backward (two
plain matrix products) uses torch.

The kernels read a tensor's elements one after another from its address.  So
a tensor that is not contiguous, or has another type, another number of
elements or another device than the block's is refused with a ValueError.
"""
from __future__ import annotations

import torch

from . import (MOE_F32, MOE_GATE_CHANNEL, MOE_GATE_FULL, MOE_GATE_NONE,
               MOE_GATE_TOKEN, MOE_MODE_FALLBACK_LAYER,
               MOE_WS_BLOCK_BACKWARD, MOE_WS_LAYER, MOE_WS_LAYER_BACKWARD,
               alloc_step_buffers, alloc_w4, layer_workspace,
               moe_block_out, moe_block_out_backward, moe_combine_block_out,
               moe_gmm_swiglu_w4, moe_layer, moe_layer_backward, moe_norm,
               moe_norm_backward, moe_permute, moe_route, moe_router_logits,
               moe_w4_bytes, moe_w4_pack, moe_w4_quantize)


def _row_type(cfg):
    return torch.float32 if cfg.dtype == MOE_F32 else torch.bfloat16


def _check(name, t, n, dtype, device):
    """Refuses a tensor whose n elements are not where a kernel reads them."""
    if not (t.is_contiguous() and t.numel() == n and t.dtype == dtype
            and t.device.type == device.type):
        raise ValueError(
            f"{name}: needs {n} contiguous elements of {dtype} on "
            f"{device.type}, not {tuple(t.shape)} of {t.dtype} on "
            f"{t.device.type}, strides {t.stride()}")


def _check_columns(cfg, w, device):
    for n in ("w_pre", "w_post", "w_next"):
        if n == "w_pre" or w[n] is not None:
            _check(n, w[n], cfg.H, torch.float32, device)


def _check_rows(cfg, device, **rows):
    for name, t in rows.items():
        if t is not None:
            _check(name, t, cfg.T * cfg.H, _row_type(cfg), device)


def _check_router(cfg, w, offset, device):
    _check("w_router", w["w_router"], cfg.H * cfg.E, _row_type(cfg), device)
    if offset is not None:
        _check("logit_offset", offset, cfg.T * cfg.E, torch.float32, device)


def _check_gate(cfg, opt, gate, device):
    """The gate's form is opt's; a gate that opt does not name, a missing one
    and an unknown form are left for the library to refuse."""
    if gate is None:
        return
    forms = {MOE_GATE_TOKEN: (cfg.T, torch.float32),
             MOE_GATE_CHANNEL: (cfg.H, torch.float32),
             MOE_GATE_FULL: (cfg.T * cfg.H, _row_type(cfg))}
    if opt.gate_kind in forms:
        _check("gate", gate, *forms[opt.gate_kind], device)


class TrainBlock:
    """One training step's forward and backward over cfg.T tokens.

    ``weights``: w_pre, w_post, w_next [H] float32 (w_post, w_next or both
    may be None), w_router [H, E], w_gate, w_up [E, H, F], w_down [E, F, H].
    ``opt`` is make_block_norm()'s; its gate kind says what ``gate`` is.
    """

    def __init__(self, cfg, opt, weights, logit_offset=None,
                 mode=MOE_MODE_FALLBACK_LAYER, device="cuda"):
        self.cfg, self.opt, self.mode = cfg, opt, mode
        self.w, self.offset = weights, logit_offset
        self.device = torch.device(device)
        _check_columns(cfg, weights, self.device)
        for n in ("w_gate", "w_up", "w_down"):
            _check(n, weights[n], cfg.E * cfg.H * cfg.F, _row_type(cfg),
                   self.device)
        _check_router(cfg, weights, logit_offset, self.device)
        rows = dict(dtype=_row_type(cfg), device=device)
        f32 = dict(dtype=torch.float32, device=device)
        T, H = cfg.T, cfg.H
        self.h, self.y, self.out = (torch.empty((T, H), **rows)
                                    for _ in range(3))
        self.h_next = None if weights["w_next"] is None else \
            torch.empty((T, H), **rows)
        self.logits = torch.empty((T, cfg.E), **f32)
        self.rstd_x, self.rstd_y, self.rstd_out = (torch.empty(T, **f32)
                                                   for _ in range(3))
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = layer_workspace(cfg, MOE_WS_LAYER, device)
        self.ws_layer_back = layer_workspace(cfg, MOE_WS_LAYER_BACKWARD,
                                             device)
        self.ws_block_back = layer_workspace(cfg, MOE_WS_BLOCK_BACKWARD,
                                             device)

    def forward(self, x, gate=None):
        """(out, h_next), h_next None without w_next; keeps what backward()
        needs."""
        c, w = self.cfg, self.w
        _check_rows(c, self.device, x=x)
        _check_gate(c, self.opt, gate, self.device)
        self.x, self.gate = x, gate
        moe_norm(c, self.opt, x, w["w_pre"], self.h, self.rstd_x)
        moe_router_logits(c, self.h, w["w_router"], self.offset, self.logits,
                          self.status)
        self.info = moe_layer(c, self.h, self.logits, w["w_gate"], w["w_up"],
                              w["w_down"], self.y, self.mode, self.ws,
                              self.status)
        moe_block_out(c, self.opt, x, self.y, w["w_post"], gate, w["w_next"],
                      self.out, self.h_next, self.rstd_y, self.rstd_out)
        return self.out, self.h_next

    def backward(self, dout=None, dh_next=None):
        """Gradients of <dout, out> + <dh_next, h_next>: a dict with dx and
        one entry for each weight and the gate."""
        c, w = self.cfg, self.w
        _check_rows(c, self.device, dout=dout, dh_next=dh_next)
        like = torch.empty_like
        columns = {n: None if w[n] is None else like(w[n])
                   for n in ("w_pre", "w_post", "w_next")}
        dgate = None if self.gate is None else like(self.gate)
        dres, dy, dh = like(self.x), like(self.y), like(self.h)
        moe_block_out_backward(
            c, self.opt, self.y, w["w_post"], self.gate, self.rstd_y,
            self.out, w["w_next"], self.rstd_out, dout, dh_next, dres, dy,
            columns["w_post"], dgate, columns["w_next"], False,
            self.ws_block_back)
        dlogits = like(self.logits)
        experts = {n: torch.empty(w[n].shape, dtype=torch.float32,
                                  device=w[n].device)
                   for n in ("w_gate", "w_up", "w_down")}
        moe_layer_backward(c, self.h, self.logits, w["w_gate"], w["w_up"],
                           w["w_down"], dy, dh, dlogits, experts["w_gate"],
                           experts["w_up"], experts["w_down"], self.mode,
                           self.ws_layer_back, self.status)
        dh = (dh.float() + dlogits @ w["w_router"].float().T).to(dh.dtype)
        dx = like(self.x)
        moe_norm_backward(c, self.opt, self.x, w["w_pre"], self.rstd_x, dh,
                          dres, dx, columns["w_pre"], False,
                          self.ws_block_back)
        return {"dx": dx, "gate": dgate, "w_router":
                self.h.float().T @ dlogits, **columns, **experts}


def quantize_experts(w4, w):
    """Packed 4-bit matrices of expert weights w [E, K, N] (contiguous; a
    transposed view is refused)."""
    E, K, N = w.shape
    _check("w", w, E * K * N, w.dtype, torch.device("cuda"))
    G = -(-K // w4.group_size)
    codes = torch.empty((E, K // 2, N), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, G, N), dtype=torch.bfloat16, device=w.device)
    zeros = torch.empty((E, G, N), dtype=torch.uint8, device=w.device) \
        if w4.zero_points else None
    packed = alloc_w4(w4, E, K, N, w.device)
    moe_w4_quantize(w4, E, K, N, w, codes, scales, zeros)
    moe_w4_pack(w4, E, K, N, codes, scales, zeros, packed)
    return packed


class DecodeBlock:
    """The block over cfg.T tokens with 4-bit experts (w_gate, w_up, w_down
    packed; the other weights as TrainBlock's).  The step enqueues its calls
    and waits for nothing, so torch.cuda.graph can capture it."""

    def __init__(self, cfg, opt, w4, weights, logit_offset=None,
                 device="cuda"):
        self.cfg, self.opt, self.w4 = cfg, opt, w4
        self.w, self.offset = weights, logit_offset
        self.device = torch.device(device)
        _check_columns(cfg, weights, self.device)
        _check_router(cfg, weights, logit_offset, self.device)
        for n, K, N in (("w_gate", cfg.H, cfg.F), ("w_up", cfg.H, cfg.F),
                        ("w_down", cfg.F, cfg.H)):
            _check(n, weights[n], moe_w4_bytes(w4, cfg.E, K, N), torch.uint8,
                   self.device)
        self.b = alloc_step_buffers(cfg, device)
        rows = dict(dtype=_row_type(cfg), device=device)
        self.h, self.out = (torch.empty((cfg.T, cfg.H), **rows)
                            for _ in range(2))
        self.h_next = None if weights["w_next"] is None else \
            torch.empty((cfg.T, cfg.H), **rows)
        self.logits = torch.empty((cfg.T, cfg.E), dtype=torch.float32,
                                  device=device)

    def step(self, x, gate=None):
        """(out, h_next) of rows x [T, H], in this object's buffers; h_next is
        None without w_next."""
        c, w, b = self.cfg, self.w, self.b
        _check_rows(c, self.device, x=x)
        _check_gate(c, self.opt, gate, self.device)
        moe_norm(c, self.opt, x, w["w_pre"], self.h)
        moe_router_logits(c, self.h, w["w_router"], self.offset, self.logits,
                          b["status"])
        moe_route(c, self.logits, b["topk_idx"], b["topk_w"], b["status"])
        moe_permute(c, self.h, b["topk_idx"], False, b["x_sorted"],
                    b["row_of"], b["sorted_token"], b["group_offsets"],
                    b["uniq_offsets"], b["uniq_tokens"], b["expand_idx"],
                    b["n_dropped"], b["permute_ws"])
        moe_gmm_swiglu_w4(c, self.w4, b["x_sorted"], b["group_offsets"],
                          w["w_gate"], w["w_up"], w["w_down"], b["h"],
                          b["y_sorted"], b["status"])
        moe_combine_block_out(c, self.opt, b["y_sorted"], b["row_of"],
                              b["topk_w"], x, w["w_post"], gate, w["w_next"],
                              None, self.out, self.h_next)
        return self.out, self.h_next


__all__ = ["DecodeBlock", "TrainBlock", "quantize_experts",
           "MOE_GATE_CHANNEL", "MOE_GATE_FULL", "MOE_GATE_NONE",
           "MOE_GATE_TOKEN"]
