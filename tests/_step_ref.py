"""64-bit plain forms of the operators that join blocks to a training step, for their tests (torch, on any device)."""
import torch


def f64(t):
    return None if t is None else t.detach().double()


def join_fwd(x, y, post=None, nxt=None, gate=None, row=None, rs=1.0, bs=1.0, eps=1e-6):
    """(out, h, ry, ro); None where there is none."""
    x, y, post, nxt, gate, row = (f64(v) for v in (x, y, post, nxt, gate, row))
    out, ry = rs * x, None
    if y is not None:
        u = y
        if post is not None:
            ry = (y.square().mean(1) + eps).rsqrt()
            u = y * ry[:, None] * post
        out = out + bs * (1.0 if row is None else row[:, None]) * (1.0 if gate is None else gate) * u
    if nxt is None:
        return out, None, ry, None
    ro = (out.square().mean(1) + eps).rsqrt()
    return out, out * ro[:, None] * nxt, ry, ro


def join_bwd(out, y, dh, dout, post, nxt, gate, row, rs, bs, ry, ro):
    """dict of dx, dy, dgamma_post, dgamma_next, dgate, drow_gate (those there are)."""
    out, y, dh, dout, post, nxt, gate, row, ry, ro = (f64(v) for v in (out, y, dh, dout, post, nxt, gate, row, ry, ro))
    r = {}
    D = 0.0 if dout is None else dout
    if nxt is not None:
        n, v = out * ro[:, None], dh * nxt
        D = D + ro[:, None] * (v - n * (v * n).mean(1, keepdim=True))
        r["dgamma_next"] = (dh * n).sum(0)
    r["dx"] = rs * D
    if y is None:
        return r
    row = torch.ones(len(D), dtype=D.dtype, device=D.device) if row is None else row
    one = torch.ones(D.shape[1], dtype=D.dtype, device=D.device)
    g, w = one if gate is None else gate, one if post is None else post
    m = y if post is None else y * ry[:, None]
    G = bs * row[:, None] * g * D
    r["dgate"] = (bs * row[:, None] * D * m * w).sum(0)
    r["drow_gate"] = (bs * g * D * m * w).sum(1)
    r["dgamma_post"] = (G * m).sum(0)
    r["dy"] = G if post is None else ry[:, None] * (G * w - m * (G * w * m).mean(1, keepdim=True))
    return r


def loss_fwd(x, W, labels):
    """(loss, lse, z of the labelled tokens); 0 for the others."""
    V = W.shape[0]
    at = torch.nonzero((labels >= 0) & (labels < V))[:, 0]
    z = x[at].double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    full = torch.zeros(len(labels), dtype=torch.float64, device=x.device)
    loss = lse - z.gather(1, labels[at].long()[:, None])[:, 0]
    return full.index_copy(0, at, loss), full.index_copy(0, at, lse), z


def loss_bwd(x, W, labels, lse, dloss):
    """(dx, dW, dz of the labelled tokens, their indexes)."""
    V = W.shape[0]
    at = torch.nonzero((labels >= 0) & (labels < V))[:, 0]
    xs, Wd = x[at].double(), W.double()
    g = torch.full((len(at),), 1.0 / max(1, len(at)), dtype=torch.float64, device=x.device) if dloss is None else dloss[at].double()
    dz = torch.exp(xs @ Wd.t() - lse[at].double()[:, None])
    dz[torch.arange(len(at), device=x.device), labels[at].long()] -= 1
    dz *= g[:, None]
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device).index_copy(0, at, dz @ Wd)
    return dx, dz.t() @ xs, dz, at
