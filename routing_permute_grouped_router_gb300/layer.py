"""A mixture-of-experts layer, the transformer sub-block around it, and a stack of blocks with its loss, held on one GPU.

``MoELayer`` owns the device copies of the weights, the saved routing state,
the float32 gradient buffers and the workspace (allocated with torch), and
calls ``moe_layer_fwd`` / ``moe_layer_bwd``.  ``MoEBlock`` puts the layer norm in
front of it and the residual dropout behind it, for training, and runs the
serving step of a few tokens with ``moe_layer_decode``.  ``MoEStack`` joins layers by
residual paths with norms and gates, puts the vocabulary loss behind them, and
clips the gradients of a step.  None does arithmetic itself.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import (MOE_BF16, MOE_DECODE_MAX_T, MoeConfig, _stream_of, allocate_grads, allocate_saved, clip_workspace,
               grad_list, moe_clip_grads, moe_decode_workspace_size, moe_dropout_add, moe_dropout_bwd, moe_layer_bwd,
               moe_layer_decode, moe_layer_fwd, moe_max_rows, moe_norm_bwd, moe_norm_fwd, moe_residual_norm_bwd,
               moe_residual_norm_fwd, moe_vocab_loss_bwd, moe_vocab_loss_fwd, norm_workspace, residual_norm_workspace,
               vocab_loss_workspace, workspace)


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
        return _tokens(self.layer.cfg, T)

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


class MoEStack:
    """Layers joined by residual paths, and the loss of a vocabulary behind them:

        s = x;  h = norm_0(s)
        for each layer i:  s = residual_scale s + branch_scale gate_i post_norm_i(layer_i(h));  h = norm_(i+1)(s)
        loss = cross entropy of h over the rows of ``head``

    ``layers`` are ``MoELayer`` of one configuration; ``gammas`` has a float32 [d] weight for each layer's norm and the
    last one, ``posts`` and ``gates`` one for each layer, or are None; ``head`` is [V, d] in the layers' type, or None.
    Gradients of the norms, the gates and the head (float32, as the layers') are in ``dgammas``, ``dposts``, ``dgates``
    and ``dhead``.
    """

    def __init__(self, layers, gammas, posts=None, gates=None, head: Optional[torch.Tensor] = None,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6):
        self.layers, n = list(layers), len(layers)
        if n == 0 or len(gammas) != n + 1 or any(v is not None and len(v) != n for v in (posts, gates)):
            raise ValueError("a stack of n layers has n + 1 norms, and n norms and n gates behind the layers or none")
        first = self.layers[0]
        alike = lambda l: (l.cfg.T, l.cfg.d_model, l.cfg.dtype, l.training)  # noqa: E731
        if any(alike(l) != alike(first) for l in self.layers):
            raise ValueError("the layers of a stack have the same tokens, width, type and training flag")
        if len({id(l) for l in self.layers}) != n:  # each keeps its own output and state for the backward
            raise ValueError("a layer is in the stack twice: build two on the same weights")
        self.gammas = [g.contiguous() for g in gammas]
        self.posts = [None] * n if posts is None else [p.contiguous() for p in posts]
        self.gates = [None] * n if gates is None else [g.contiguous() for g in gates]
        self.head = None if head is None else head.contiguous()
        self.residual_scale, self.branch_scale, self.eps = residual_scale, branch_scale, eps
        self.training, dev, cfg = first.training, first.device, first.cfg
        T, d = cfg.T, cfg.d_model
        # the layers' calls want valid pointers for no tokens too: what they are given has a row at least
        rows = dict(size=(max(T, 1), d), dtype=first.act_dtype, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self._h = [torch.empty(**rows) for _ in range(n + 1)]
        self.h = [v[:T] for v in self._h]
        self.streams = [torch.empty(**rows)[:T] for _ in range(n)]
        self.rstd_post = [None if p is None or not self.training else torch.empty(T, **f32) for p in self.posts]
        self.rstd = [torch.empty(T, **f32) if self.training else None for _ in range(n + 1)]
        if self.head is not None:
            self.loss, self.lse, self.total = torch.empty(T, **f32), torch.empty(T, **f32), torch.empty(2, **f32)
            self.loss_ws = vocab_loss_workspace(T, d, self.head.shape[0], first.act_dtype, self.training, dev)
        self._decode = {}  # (stream, tokens) -> configs, s, h, y, out and workspace
        self._decode_ws = {}  # stream -> workspace, large enough for any number of tokens and layer
        if not self.training:
            return
        zeros = lambda w: None if w is None else torch.zeros(w.numel(), **f32)  # noqa: E731
        self.dgammas, self.dposts, self.dgates = ([zeros(w) for w in v] for v in (self.gammas, self.posts, self.gates))
        self.dhead = None if self.head is None else torch.zeros(self.head.shape, **f32)
        self.dh, self.dx = torch.empty(**rows)[:T], torch.empty(**rows)[:T]
        self._dy = torch.empty(**rows)
        self.ws = residual_norm_workspace(T, d, dev)
        self.norm = torch.zeros(1, **f32)
        grads = self.gradients()
        self._grad_list, self._clip_ws = grad_list(grads, grads), clip_workspace(len(grads), dev)

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """The last norm's output [T, d], a buffer of the stack's."""
        T = self.layers[0].cfg.T
        moe_residual_norm_fwd(x, None, None, self.h[0], None, self.gammas[0], eps=self.eps, rstd_next=self.rstd[0], stream=stream)
        s = x
        for i, layer in enumerate(self.layers):
            y = layer.forward(self._h[i], stream)[:T]
            moe_residual_norm_fwd(s, y, self.streams[i], self.h[i + 1], self.posts[i], self.gammas[i + 1], self.gates[i], None,
                                  self.residual_scale, self.branch_scale, self.eps, self.rstd_post[i], self.rstd[i + 1], stream)
            s = self.streams[i]
        return self.h[-1]

    def forward_loss(self, x: torch.Tensor, labels: torch.Tensor, stream=None) -> torch.Tensor:
        """(sum of the losses, labelled tokens) as two floats; each token's loss is in ``loss``."""
        if self.head is None:
            raise RuntimeError("stack was built without a head")
        self.forward(x, stream)
        moe_vocab_loss_fwd(self.h[-1], self.head, labels, self.loss, self.lse, self.loss_ws, self.total, stream)
        return self.total

    def backward(self, x: torch.Tensor, labels: torch.Tensor, accumulate: bool, dloss: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """Gradients after ``forward_loss`` of the same x and labels: of the losses' mean, or of sum(dloss * loss).
        Returns that of x."""
        if not self.training:
            raise RuntimeError("stack's layers were built without training buffers")
        if self.head is None:
            raise RuntimeError("stack was built without a head")
        T = self.layers[0].cfg.T
        moe_vocab_loss_bwd(self.h[-1], self.head, labels, self.lse, dloss, self.dh, self.dhead, accumulate, self.loss_ws, stream)
        dh, ds, dy = self.dh, None, self._dy[:T]
        for i in reversed(range(len(self.layers))):
            layer = self.layers[i]
            grads = dict(dgamma_post=self.dposts[i], dgamma_next=self.dgammas[i + 1], dgate=self.dgates[i])
            moe_residual_norm_bwd(self.streams[i], layer.y[:T], dh, ds, self.posts[i], self.gammas[i + 1], self.gates[i], None,
                                  self.residual_scale, self.branch_scale, self.rstd_post[i], self.rstd[i + 1], self.dx, dy,
                                  grads, accumulate, self.ws, stream)
            dh, ds = layer.backward(self._h[i], self._dy, accumulate, stream)[:T], self.dx
        moe_residual_norm_bwd(x, None, dh, ds, None, self.gammas[0], None, None, 1.0, 1.0, None, self.rstd[0], self.dx, None,
                              dict(dgamma_next=self.dgammas[0]), accumulate, self.ws, stream)
        return self.dx

    def gradients(self) -> list:
        """Every gradient tensor of the stack."""
        grads = [l.grads[n] for l in self.layers for n in ("dW_r", "dW1", "dW3", "dW2")]
        return grads + [g for v in (self.dgammas, self.dposts, self.dgates, [self.dhead]) for g in v if g is not None]

    def clip(self, max_norm: float, stream=None) -> torch.Tensor:
        """Clips the gradients in place to a norm of ``max_norm`` all together; their norm before it, one float."""
        if not self.training:
            raise RuntimeError("stack's layers were built without training buffers")
        moe_clip_grads(self._grad_list, max_norm, self.norm, self._clip_ws, stream)
        return self.norm

    def decode(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """The last norm's output for at most 64 tokens, two kernels a layer.  Buffers as in ``MoEBlock.decode``."""
        key = _stream_of(self.gammas[0], stream), x.numel() // self.layers[0].cfg.d_model
        if key not in self._decode:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                self._decode[key] = self._decode_buffers(*key)
        cfgs, s, h, y, out, ws = self._decode[key]
        moe_residual_norm_fwd(x, None, None, h, None, self.gammas[0], eps=self.eps, stream=stream)
        before, last = x, len(self.layers) - 1
        for i, layer in enumerate(self.layers):
            moe_layer_decode(cfgs[i], layer.weights, h, None, y, None, None, ws, stream)
            # x may be the last call's result: nothing but the last path writes there
            moe_residual_norm_fwd(before, y, s, out if i == last else h, self.posts[i], self.gammas[i + 1], self.gates[i],
                                  None, self.residual_scale, self.branch_scale, self.eps, stream=stream)
            before = s
        return out if out.shape == x.shape else out.view(x.shape)

    def _decode_buffers(self, raw_stream: int, T: int):
        cfgs = [_tokens(l.cfg, T) for l in self.layers]
        for c in cfgs:
            moe_decode_workspace_size(c)  # refuses what the layer would
        ws = self._decode_ws.get(raw_stream)
        first = self.layers[0]
        if ws is None:
            size = max(moe_decode_workspace_size(_tokens(l.cfg, t)) for l in self.layers for t in range(1, MOE_DECODE_MAX_T + 1))
            ws = self._decode_ws[raw_stream] = torch.empty(size, dtype=torch.uint8, device=first.device)
        rows = [torch.empty(T, first.cfg.d_model, dtype=first.act_dtype, device=first.device) for _ in range(4)]
        return (cfgs, *rows, ws)


def _tokens(c: MoeConfig, T: int) -> MoeConfig:
    """The configuration for T tokens, without training's terms."""
    return MoeConfig(T, c.d_model, c.d_ff, c.E, c.k, c.capacity_factor, c.capacity, c.dtype, 0.0)


def from_workload(wl, device="cuda", training: bool = True, T: Optional[int] = None,
                  aux_loss_coeff: float = 0.0, recompute: bool = False) -> MoELayer:
    """Upload a ``workload.Workload``'s weights and build the layer."""
    from . import config_of

    cfg = config_of(wl.shape, T, aux_loss_coeff)
    bias = None if wl.bias is None else torch.from_numpy(wl.bias).to(device)
    return MoELayer(cfg, torch.from_numpy(wl.W_r).to(device), bias, wl.W1.torch(device), wl.W3.torch(device),
                    wl.W2.torch(device), training=training, recompute=recompute)
