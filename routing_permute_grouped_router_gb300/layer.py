"""A mixture-of-experts layer, and the transformer sub-block around it, held on one GPU.

``MoELayer`` owns the device copies of the weights, the saved routing state,
the float32 gradient buffers and the workspace (allocated with torch), and
calls ``moe_layer_fwd`` / ``moe_layer_bwd``.  ``MoEBlock`` puts the layer norm in
front of it and the residual dropout behind it, for training, and runs the
serving step of a few tokens with ``moe_layer_decode``.  Neither does arithmetic
itself.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import (MOE_BF16, MOE_DECODE_MAX_T, MoeConfig, _stream_of, allocate_grads, allocate_saved, moe_decode_workspace_size,
               moe_dropout_add, moe_dropout_bwd, moe_layer_bwd, moe_layer_decode, moe_layer_fwd, moe_max_rows,
               moe_norm_bwd, moe_norm_fwd, norm_workspace, workspace)


class MoELayer:
    def __init__(self, cfg: MoeConfig, W_r: torch.Tensor, bias: Optional[torch.Tensor], W1: torch.Tensor,
                 W3: torch.Tensor, W2: torch.Tensor, training: bool = True, recompute: bool = False):
        self.cfg = cfg
        self.device = W1.device
        self.act_dtype = torch.bfloat16 if cfg.dtype == MOE_BF16 else torch.float32
        self.weights = dict(W_r=W_r.contiguous(), bias=None if bias is None else bias.contiguous(),
                            W1=W1.contiguous(), W3=W3.contiguous(), W2=W2.contiguous())
        self.training = training
        self.max_rows = moe_max_rows(cfg)
        self.recompute = training and recompute  # keep no a, b, h: the backward recomputes them
        self.saved = allocate_saved(cfg, self.device, self.recompute) if training else None
        self.grads = allocate_grads(cfg, self.device) if training else None
        self.ws = workspace(cfg, (2 if self.recompute else 1) if training else 0, self.device)
        T, d = max(cfg.T, 1), cfg.d_model
        self.y = torch.empty(T, d, dtype=self.act_dtype, device=self.device)
        self.dx = torch.empty(T, d, dtype=self.act_dtype, device=self.device) if training else None

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        moe_layer_fwd(self.cfg, self.weights, x, self.y, self.saved, self.ws, stream)
        return self.y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, accumulate: bool, stream=None) -> torch.Tensor:
        if not self.training:
            raise RuntimeError("layer was built without training buffers")
        moe_layer_bwd(self.cfg, self.weights, x, dy, self.saved, self.dx, self.grads, int(accumulate), self.ws,
                      stream)
        return self.dx


class MoEBlock:
    """out = x + dropout(layer(norm(x))), its backward, and the same for a few tokens without dropout.

    ``layer`` is a ``MoELayer``; gamma and beta [d] float32 are the norm's weights, whose gradients are in
    ``dgamma`` and ``dbeta``.  The dropout's mask is a function of (seed, offset): the backward is given the
    forward's.  Give each layer and step its own offset.
    """

    def __init__(self, layer: MoELayer, gamma: torch.Tensor, beta: torch.Tensor, p: float = 0.0, eps: float = 1e-5):
        self.layer, self.p, self.eps = layer, p, eps
        self.gamma, self.beta = gamma.contiguous(), beta.contiguous()
        cfg, dev = layer.cfg, layer.device
        T, d = cfg.T, cfg.d_model
        # the layer's calls want valid pointers for no tokens too: what they are given has a row at least
        rows = dict(size=(max(T, 1), d), dtype=layer.act_dtype, device=dev)
        self._h = torch.empty(**rows)
        self.h = self._h[:T]
        self.out = torch.empty_like(self.h)
        self._decode = {}  # (stream, tokens) -> config, h, out and workspace
        self._decode_ws = {}  # stream -> workspace, large enough for any number of tokens
        if layer.training:
            f32 = dict(dtype=torch.float32, device=dev)
            self.mean, self.rstd = torch.empty(T, **f32), torch.empty(T, **f32)
            self.dgamma, self.dbeta = torch.zeros(d, **f32), torch.zeros(d, **f32)
            self._dy = torch.empty(**rows)
            self.dy = self._dy[:T]
            self.dx = torch.empty_like(self.h)
            self.ws = norm_workspace(T, d, dev)
        else:
            self.mean = self.rstd = None

    def forward(self, x: torch.Tensor, seed: int = 0, offset: int = 0, stream=None) -> torch.Tensor:
        moe_norm_fwd(x, self.gamma, self.beta, self.eps, self.h, self.mean, self.rstd, stream)
        y = self.layer.forward(self._h, stream)[:self.layer.cfg.T]
        moe_dropout_add(y, x, self.out, self.p if self.layer.training else 0.0, seed, offset, stream)
        return self.out

    def backward(self, x: torch.Tensor, dout: torch.Tensor, accumulate: bool, seed: int = 0, offset: int = 0,
                 stream=None) -> torch.Tensor:
        if not self.layer.training:
            raise RuntimeError("block's layer was built without training buffers")
        moe_dropout_bwd(dout, self.dy, self.p, seed, offset, stream)
        dh = self.layer.backward(self._h, self._dy, accumulate, stream)[:self.layer.cfg.T]
        moe_norm_bwd(x, dh, self.gamma, self.mean, self.rstd, dout, self.dx, self.dgamma, self.dbeta, accumulate,
                     self.ws, stream)
        return self.dx

    def decode(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """x + layer(norm(x)) for at most 64 tokens, in two kernels.

        The result is a buffer of the block's, written again by the next call of as many tokens on the same stream.
        Buffers belong to one stream each and live as long as the block, so calls on several streams may overlap and
        graphs may be captured, for any numbers of tokens in any order.  A graph uses the buffers of the stream that
        it was captured on: its replays, and other calls on that stream, follow one another.
        """
        key = _stream_of(self.gamma, stream), x.shape[0]
        if key not in self._decode:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                self._decode[key] = self._decode_buffers(*key)
        cfg, h, out, ws = self._decode[key]
        moe_norm_fwd(x, self.gamma, self.beta, self.eps, h, None, None, stream)
        moe_layer_decode(cfg, self.layer.weights, h, x, out, None, None, ws, stream)
        return out if out.shape == x.shape else out.view(x.shape)

    def _decode_config(self, T: int) -> MoeConfig:
        c = self.layer.cfg
        return MoeConfig(T, c.d_model, c.d_ff, c.E, c.k, c.capacity_factor, c.capacity, c.dtype, 0.0)

    def _decode_buffers(self, raw_stream: int, T: int):
        """Made on the stream that uses them: memory that the allocator hands out again is free in that order.  Their
        sizes and type are the layer's, whatever was passed."""
        cfg = self._decode_config(T)
        moe_decode_workspace_size(cfg)  # refuses what the layer would
        ws = self._decode_ws.get(raw_stream)
        if ws is None:
            size = max(moe_decode_workspace_size(self._decode_config(t)) for t in range(1, MOE_DECODE_MAX_T + 1))
            ws = self._decode_ws[raw_stream] = torch.empty(size, dtype=torch.uint8, device=self.layer.device)
        h, out = (torch.empty(T, cfg.d_model, dtype=self.layer.act_dtype, device=self.layer.device) for _ in range(2))
        return cfg, h, out, ws


def from_workload(wl, device="cuda", training: bool = True, T: Optional[int] = None,
                  aux_loss_coeff: float = 0.0, recompute: bool = False) -> MoELayer:
    """Upload a ``workload.Workload``'s weights and build the layer."""
    from . import config_of

    cfg = config_of(wl.shape, T, aux_loss_coeff)
    bias = None if wl.bias is None else torch.from_numpy(wl.bias).to(device)
    return MoELayer(cfg, torch.from_numpy(wl.W_r).to(device), bias, wl.W1.torch(device), wl.W3.torch(device),
                    wl.W2.torch(device), training=training, recompute=recompute)
