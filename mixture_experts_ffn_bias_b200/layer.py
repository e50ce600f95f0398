"""Device-side buffers for one MoE layer and calls into the C ABI.

PyTorch supplies device memory and streams only; every step of the layer runs
in libmoe_b200.so.  ``MoELayer`` uploads a workload's host arrays (as produced
by :mod:`.inputs`), owns the output buffers and the workspace, and exposes the
calls of the ABI with those buffers filled in.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import binding as B
from .inputs import DTYPE_BF16, MoEShape

_WEIGHT_KEYS = ("w1", "w3", "w2", "ws1", "ws3", "ws2")


def act_dtype(shape: MoEShape) -> torch.dtype:
    return torch.bfloat16 if shape.dtype == DTYPE_BF16 else torch.float32


def to_device(a: np.ndarray, dtype: torch.dtype, device) -> torch.Tensor:
    """Host float32 array (bf16-exact for bf16) -> contiguous device tensor."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(device=device)
    return t.to(dtype).contiguous()


class MoELayer:
    def __init__(self, shape: MoEShape, host: Dict[str, np.ndarray], device="cuda",
                 groups: Optional[B.MoEGroupOpts] = None):
        """groups (binding.make_group_opts): route with moe_route_groups."""
        self.shape = shape
        self.groups = groups
        self.device = torch.device(device)
        self.cfg = B.config_from_shape(shape)
        st = B.moe_check_config(self.cfg)
        if st != B.MOE_OK:
            raise B.MoEError(st, "configuration rejected: " + B.status_string(st))
        dt = act_dtype(shape)
        self.dtype = dt
        self.x = to_device(host["x"], dt, self.device)
        self.w_router = to_device(host["w_router"], dt, self.device)
        self.weights = {k: to_device(host[k], dt, self.device) for k in _WEIGHT_KEYS if k in host}
        self.sel_bias = (to_device(host["sel_bias"], torch.float32, self.device)
                         if "sel_bias" in host else None)
        self.logit_offset = (to_device(host["logit_offset"], torch.float32, self.device)
                             if "logit_offset" in host else None)
        T, d, E, k = shape.T, shape.d_model, shape.n_experts, shape.top_k
        kw = dict(device=self.device)
        self.out = torch.empty((T, d), dtype=dt, **kw)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, **kw)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, **kw)
        self.counts = torch.empty((E,), dtype=torch.int32, **kw)
        self.ws = torch.empty((max(B.moe_workspace_size(self.cfg), 256),), dtype=torch.uint8, **kw)
        self.ows = []

    # ----------------------------------------------------------------- calls
    def forward(self, x: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None, gather_rows: bool = False, fold_combine: bool = False,
                scatter_in_gemm: bool = False,
                token_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The layer forward (moe_forward; moe_forward_ex with gather_rows,
        fold_combine or scatter_in_gemm; moe_forward_grouped for a layer with
        groups, which also takes a token_mask [T] uint8 or bool, 0 for
        padding)."""
        if self.groups is not None:
            if gather_rows or fold_combine or scatter_in_gemm:
                raise B.MoEError(B.MOE_ERR_UNSUPPORTED,
                                 "a layer with groups has the default expert path only")
            B.moe_forward_grouped(self.cfg, self.groups, self.x if x is None else x,
                                  self.w_router, self.sel_bias, self.logit_offset, token_mask,
                                  self.weights, self.out if out is None else out, self.topk_idx,
                                  self.topk_w, self.counts, self.ws, stream=stream)
            return self.out if out is None else out
        if token_mask is not None:
            raise B.MoEError(B.MOE_ERR_UNSUPPORTED, "token_mask needs a layer with groups")
        args = (self.cfg, self.x if x is None else x, self.w_router, self.sel_bias,
                self.logit_offset, self.weights, self.out if out is None else out,
                self.topk_idx, self.topk_w, self.counts, self.ws)
        if gather_rows or fold_combine or scatter_in_gemm:
            B.moe_forward_ex(*args, gather_rows=int(gather_rows),
                             fold_combine=int(fold_combine),
                             scatter_in_gemm=int(scatter_in_gemm), stream=stream)
        else:
            B.moe_forward(*args, stream=stream)
        return self.out if out is None else out

    def dispatch_view(self):
        """(offsets, slot_pos, perm_src) of the last forward, read from the
        workspace (int32 device views; valid until the next call on it)."""
        return B.moe_forward_dispatch_view(self.cfg, self.ws)

    def backward(self, dout: torch.Tensor, stream=None) -> Dict[str, torch.Tensor]:
        """Gradients of <dout, out> for the last forward (bf16 layers): dx,
        dw_router (fp32) and dw1, dw3, dw2 (and the shared expert's)."""
        if not hasattr(self, "bws"):
            n = B.moe_backward_workspace_size(self.cfg)
            if n == 0:
                raise B.MoEError(B.MOE_ERR_UNSUPPORTED, "backward needs a bf16 layer")
            self.bws = torch.empty((n,), dtype=torch.uint8, device=self.device)
        g = {"dx": torch.empty_like(self.x),
             "dw_router": torch.empty(self.w_router.shape, dtype=torch.float32,
                                      device=self.device)}
        for k, v in self.weights.items():
            g["d" + k] = torch.empty_like(v)
        args = (self.x, self.w_router, self.logit_offset, self.weights, self.topk_idx,
                self.topk_w, dout, g["dx"], g["dw_router"], g, self.ws, self.bws, stream)
        if self.groups is not None:
            B.moe_backward_grouped(self.cfg, self.groups, *args)
        else:
            B.moe_backward(self.cfg, *args)
        return g

    def orthogonalize(self, grads: Dict[str, torch.Tensor], steps=5, coeffs=B.MUON_COEFFS,
                      eps=1e-7, scale=1.0, stream=None) -> Dict[str, torch.Tensor]:
        """Muon's update directions (moe_orthogonalize) of the weight gradients or
        momenta in ``grads`` (the dw* of backward(), by their names), each in
        its own dtype; a stacked [E, out, in] tensor is E matrices.  The layer's
        calls share one workspace: not on two streams at once.  It grows to the
        largest set of gradients a call has had, and outgrown ones are kept with
        the layer (a captured graph may use them): pass the largest set first."""
        jobs, need = [], 0
        for k, g in grads.items():
            if not k.startswith("dw"):
                continue
            b, r, c = (1,) * (3 - g.dim()) + tuple(g.shape)
            dt = B.DTYPE_BF16 if g.dtype == torch.bfloat16 else B.DTYPE_F32
            cfg = B.make_ortho_config(b, r, c, dt, dt, steps, coeffs, eps, scale)
            need = max(need, B.moe_orthogonalize_workspace_size(cfg))
            jobs.append((k, g, cfg))
        out, here = {}, torch.cuda.current_stream(self.device)
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(
                stream if isinstance(stream, int) else stream.cuda_stream, device=self.device)
        # allocated on the stream that writes: a block of the current one's may
        # still be in use by what that has queued
        with torch.cuda.stream(here if stream is None else stream):
            if jobs and (not self.ows or self.ows[-1].numel() < need):
                # the outgrown ones stay: a captured graph, or work queued on
                # another stream, may still use them
                self.ows.append(torch.empty((max(need, 256),), dtype=torch.uint8,
                                            device=self.device))
            for k, g, cfg in jobs:
                out[k] = torch.empty_like(g)
                B.moe_orthogonalize(cfg, g, out[k], self.ows[-1])
        if stream is not None and stream != here:
            for u in out.values():
                u.record_stream(here)
        return out

    def bias_update(self, counts: Optional[torch.Tensor] = None, rate=1e-3, starved_frac=0.1,
                    starved_add=0.5, clamp=10.0, stream=None):
        if self.sel_bias is None:
            self.sel_bias = torch.zeros(self.shape.n_experts, dtype=torch.float32,
                                        device=self.device)
        B.moe_bias_update(self.cfg, self.counts if counts is None else counts, self.sel_bias,
                          rate, starved_frac, starved_add, clamp, stream)

    def device_status(self, stream=None):
        return B.moe_device_status(self.ws, stream)
