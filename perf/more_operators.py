"""Cases, plain forms and work of the operators that join the blocks to a training step:

  join_fwd   the residual path between two blocks: RMS norm behind a block, its gates and residual scale, RMS norm in
             front of the next block
  join_bwd   its backward pass, with the gradients of the norms' weights and of the gates
  clip       the global norm of many gradient tensors, and the clipped gradients
  loss_fwd   softmax cross entropy over a large vocabulary: the loss and log-sum-exp of each token
  loss_bwd   its gradient: of the tokens and of the vocabulary's weights

``run`` computes the plain form in elementary torch operations in 32 bits, or, where ``own`` is true, makes the
library's calls.  ``exact`` computes the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
IGNORED = -100


# ----------------------------- cases -------------------------------------- #
def _join(op, rows, d, dtype, post=True, following=True, gate="channel", rs=1.0, bs=1.0, dout=True):
    return dict(op=op, rows=rows, d=d, dtype=dtype, post=post, following=following, gate=gate, rs=rs, bs=bs, dout=dout)


def _clip(sizes, dtype, ratio, tensors=0, elements=0):
    return dict(op="clip", sizes=sizes, dtype=dtype, ratio=ratio, tensors=tensors, elements=elements)


def _loss(op, T, d, V, dtype, ignored=0.0, dw="f32", mean=False):
    return dict(op=op, T=T, d=d, V=V, dtype=dtype, ignored=ignored, dw=dw, mean=mean)


def listed():
    return [
        # between two blocks of a decoding batch: launch latency
        dict(name="join_fwd_16_rows", **_join("join_fwd", 16, 4096, "bf16")),
        # between two blocks in training, at the dropless layer's micro-batch
        dict(name="join_fwd_train", **_join("join_fwd", 32768, 4096, "bf16", rs=1.0, bs=0.5)),
        # its backward pass: both norms, the channel gate, the residual stream's own gradient
        dict(name="join_bwd_train", **_join("join_bwd", 32768, 4096, "bf16", rs=1.0, bs=0.5)),
        # float32 rows of an odd length with a gate of each token, so no row but the first is aligned
        dict(name="join_bwd_odd_f32", **_join("join_bwd", 4099, 1021, "f32", gate="row", rs=0.8)),
        # the float32 gradients of the 16-expert layer (W_r, W1, W3, W2) past their largest norm
        dict(name="clip_train_e16", **_clip("layer_2048_4096_16", "f32", 0.25)),
        # the norm alone of the dropless 32-expert layer's gradients, as a training step logs it
        dict(name="norm_dropless_e32", **_clip("layer_4096_1536_32", "f32", math.inf)),
        # some hundred small tensors, bf16 and float32, at odd offsets of one flat buffer: norms, gates, routers
        dict(name="clip_300_small", **_clip("flat", "both", 0.5, tensors=300, elements=700000)),
        # scoring one token over a large vocabulary: the weights are read once
        dict(name="loss_fwd_one_token", **_loss("loss_fwd", 1, 4096, 128000, "bf16")),
        # a training micro-batch of the 16-expert layer over a vocabulary of an odd size
        dict(name="loss_fwd_train", **_loss("loss_fwd", 8192, 2048, 50257, "bf16", ignored=0.02)),
        # its gradient, the weights' in float32 as gradients are accumulated
        dict(name="loss_bwd_train", **_loss("loss_bwd", 8192, 2048, 50257, "bf16", ignored=0.02, mean=True)),
        # a long micro-batch at the dropless layer's width, prompts masked out, the weights' gradient in bf16
        dict(name="loss_bwd_large", **_loss("loss_bwd", 16384, 4096, 65536, "bf16", ignored=0.25, dw="bf16")),
        # a small float32 model: nothing is a multiple of a tile
        dict(name="loss_bwd_odd_f32", **_loss("loss_bwd", 777, 1000, 10007, "f32", ignored=0.1)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join_fwd", "join_bwd", "clip", "loss_fwd", "loss_bwd", "loss_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("join"):
        step = rng.choice([1, 8])
        d = step * _log(rng, 64 // step, 8192 // step)
        rows = min(_log(rng, 1, 32768), 32768 * 4096 // d // (2 if dtype == "f32" else 1))
        post, following = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        return _join(op, rows, d, dtype, post, following, rng.choice(["none", "channel", "row", "both"]),
                     rng.choice([1.0, 0.8]), rng.choice([1.0, 0.5]), rng.random() < 0.7 or not following)
    if op == "clip":
        if rng.random() < 0.5:
            d, f, E = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512), rng.choice([1, 4, 7, 8, 16, 32])
            while E * d * f > 32 * 4096 * 1536:
                E = max(1, E // 2)
            return _clip(f"layer_{d}_{f}_{E}", dtype, rng.choice([0.1, 0.9, 1.5, math.inf]))
        n = _log(rng, 1, 400)
        return _clip("flat", rng.choice(["bf16", "f32", "both"]), rng.choice([0.3, 2.0]), n, n * _log(rng, 16, 50000))
    if dtype == "bf16":
        d, V, most = 8 * _log(rng, 8, 512), _log(rng, 500, 131072), 16384 * 4096 * 65536
    else:
        d, V, most = 4 * _log(rng, 16, 512), _log(rng, 500, 32768), 1024 * 1024 * 32768
    T = max(1, min(_log(rng, 1, 16384), most // (d * V)))
    return _loss(op, T, d, V, dtype, rng.choice([0.0, 0.05, 0.5]), rng.choice(["f32", "bf16"]) if dtype == "bf16" else "f32",
                 rng.random() < 0.5)


# ----------------------------- inputs ------------------------------------- #
def _flat_sizes(case):
    """Lengths of the tensors of a flat buffer, from a few elements up, odd ones among them; and whether each is bf16."""
    n = case["tensors"]
    r = torch.Generator().manual_seed(n + case["elements"])
    u = torch.exp(5 * torch.rand(n, generator=r, dtype=torch.float64))
    sizes = (u / u.sum() * case["elements"]).long().clamp_(min=1).tolist()
    return sizes, [case["dtype"] == "bf16" or (case["dtype"] == "both" and i % 3 == 1) for i in range(n)]


def _layer_shapes(case):
    d, f, E = (int(v) for v in case["sizes"].split("_")[1:])
    return [(d, E), (E, d, f), (E, d, f), (E, f, d)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * seed + 29)
    f32 = torch.float32

    def normal(*shape, scale=1.0, dtype=f32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=f32).mul_(scale).to(dtype)

    s = dict(case=dict(case))
    if case["op"].startswith("join"):
        t, rows, d = DTYPES[case["dtype"]], case["rows"], case["d"]
        # a residual stream whose rows have their own scale, and a block's output of a smaller one
        x = normal(rows, d) * (0.5 + 1.5 * torch.rand(rows, 1, generator=g, device=DEV))
        x[:, torch.randint(0, d, (max(1, d // 512),), generator=g, device=DEV)] *= 8.0
        s["x"] = x.to(t)
        del x
        s["y"] = normal(rows, d, scale=0.3, dtype=t)
        s["gamma_post"] = 1.0 + normal(d, scale=0.2) if case["post"] else None
        s["gamma_next"] = 1.0 + normal(d, scale=0.2) if case["following"] else None
        s["gate"] = 0.5 + normal(d, scale=0.3) if case["gate"] in ("channel", "both") else None
        s["row_gate"] = torch.rand(rows, generator=g, device=DEV) if case["gate"] in ("row", "both") else None
        if case["op"] == "join_bwd":
            s["dh"] = normal(rows, d, dtype=t) if case["following"] else None
            s["dout"] = normal(rows, d, dtype=t) if case["dout"] else None
            # what the forward pass has kept
            kept = _plain_join_fwd(s)
            s["out"], s["rstd_post"], s["rstd_next"] = kept["out"], kept["rstd_post"], kept["rstd_next"]
        return s
    if case["op"] == "clip":
        if case["sizes"] == "flat":
            sizes, half = _flat_sizes(case)
            # views of one buffer a type, as a data-parallel bucket holds them: offsets of any parity
            for name, t in (("f32", f32), ("bf16", torch.bfloat16)):
                own_sizes = [n for n, h in zip(sizes, half) if h == (name == "bf16")]
                flat = normal(sum(own_sizes), dtype=f32)
                scales = torch.exp(3 * torch.randn(len(own_sizes), generator=g, device=DEV) - 6)
                flat *= scales.repeat_interleave(torch.tensor(own_sizes, device=DEV)) if own_sizes else 1.0
                s["flat_" + name] = flat.to(t)
                s["sizes_" + name] = own_sizes
            total = sum(float(s["flat_" + n].double().square().sum()) for n in ("f32", "bf16"))
        else:
            t = DTYPES[case["dtype"]]
            s["grads"] = [normal(*shape, scale=math.exp(-7 - i), dtype=t) for i, shape in enumerate(_layer_shapes(case))]
            total = sum(float(x.numel()) * math.exp(-7 - i) ** 2 for i, x in enumerate(s["grads"]))
        s["max_norm"] = case["ratio"] * math.sqrt(total)
        return s
    t, T, d, V = DTYPES[case["dtype"]], case["T"], case["d"], case["V"]
    s["W"] = normal(V, d, scale=d ** -0.5, dtype=t)
    # frequent tokens first; the tokens' states lean to their labels as in a model that has learned something
    labels = (V * torch.rand(T, generator=g, device=DEV, dtype=torch.float64) ** 3).long().clamp_(max=V - 1)
    s["x"] = (1.5 * normal(T, d) + 4.0 * s["W"][labels].float()).to(t)
    masked = torch.randperm(T, generator=g, device=DEV)[: int(case["ignored"] * T)]
    labels[masked] = IGNORED
    s["labels"] = labels.int()
    if case["op"] == "loss_bwd":
        s["lse"] = _lse(s)
        s["dloss"] = None if case["mean"] else torch.rand(T, generator=g, device=DEV) / T
    return s


def _lse(s):
    """What the forward pass has kept, for few rows at a time."""
    W = s["W"].float()
    return torch.cat([torch.logsumexp(x.float() @ W.t(), 1) for x in s["x"].split(2048)])


# ----------------------------- plain forms -------------------------------- #
def _branch(s):
    """The block's output, normed: u, its norm before the weight, and 1 / rms."""
    y = s["y"].float()
    if s["gamma_post"] is None:
        return y, y, None
    rstd = 1 / torch.sqrt((y * y).mean(1) + EPS)
    m = y * rstd[:, None]
    return m * s["gamma_post"], m, rstd


def _gated(s, u):
    u = u * s["case"]["bs"]
    if s["gate"] is not None:
        u = u * s["gate"]
    return u if s["row_gate"] is None else u * s["row_gate"][:, None]


def _plain_join_fwd(s):
    t = s["x"].dtype
    u, _, rstd_post = _branch(s)
    out = s["x"].float() * s["case"]["rs"] + _gated(s, u)
    if s["gamma_next"] is None:
        return dict(out=out.to(t), h=None, rstd_post=rstd_post, rstd_next=None)
    rstd = 1 / torch.sqrt((out * out).mean(1) + EPS)
    h = out * rstd[:, None] * s["gamma_next"]
    return dict(out=out.to(t), h=h.to(t), rstd_post=rstd_post, rstd_next=rstd)


def _plain_join_bwd(s):
    c, t = s["case"], s["x"].dtype
    grads = {}
    D = 0.0 if s["dout"] is None else s["dout"].float()
    if s["gamma_next"] is not None:
        n, dh = s["out"].float() * s["rstd_next"][:, None], s["dh"].float()
        grads["dgamma_next"] = (dh * n).sum(0)
        v = dh * s["gamma_next"]
        D = D + (v - n * (v * n).mean(1, keepdim=True)) * s["rstd_next"][:, None]
    y = s["y"].float()
    m = y if s["rstd_post"] is None else y * s["rstd_post"][:, None]
    u = m if s["gamma_post"] is None else m * s["gamma_post"]
    if s["gate"] is not None:
        rows = 1.0 if s["row_gate"] is None else s["row_gate"][:, None]
        grads["dgate"] = (D * c["bs"] * rows * u).sum(0)
    if s["row_gate"] is not None:
        grads["drow_gate"] = (D * c["bs"] * (u if s["gate"] is None else u * s["gate"])).sum(1)
    dy = _gated(s, D)
    if s["gamma_post"] is not None:
        grads["dgamma_post"] = (dy * m).sum(0)
        w = dy * s["gamma_post"]
        dy = (w - m * (w * m).mean(1, keepdim=True)) * s["rstd_post"][:, None]
    return dict(dx=(D * c["rs"]).to(t), dy=dy.to(t), **grads)


def _plain_clip(s):
    grads = s["grads"] if "grads" in s else [s["flat_f32"], s["flat_bf16"]]
    total = torch.stack([x.float().square().sum(dtype=torch.float64) for x in grads]).sum()
    norm = torch.sqrt(total).float()
    if math.isinf(s["max_norm"]):
        return dict(norm=norm)
    scale = torch.where((norm > s["max_norm"]) & torch.isfinite(norm), s["max_norm"] / norm, 1.0)
    return dict(norm=norm, out=[(x.float() * scale).to(x.dtype) for x in grads])


def _logits(s):
    valid = s["labels"] >= 0
    x = torch.where(valid[:, None], s["x"].float(), 0.0)  # an ignored token's state may hold anything
    return valid, x, x @ s["W"].float().t()


def _plain_loss_fwd(s):
    valid, _, z = _logits(s)
    top = z.max(1)[0]
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    picked = z.gather(1, s["labels"].long().clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return dict(loss=torch.where(valid, lse - picked, zero), lse=torch.where(valid, lse, zero))


def _plain_loss_bwd(s):
    c = s["case"]
    valid, x, z = _logits(s)
    dloss = 1.0 / valid.sum().clamp(min=1) if s["dloss"] is None else s["dloss"]
    dz = torch.exp(z.sub_(s["lse"][:, None]))
    del z
    at = s["labels"].long().clamp(min=0)[:, None]
    dz.scatter_(1, at, dz.gather(1, at) - 1)
    dz *= torch.where(valid, dloss, 0.0)[:, None]
    return dict(dx=(dz @ s["W"].float()).to(s["x"].dtype), dW=(dz.t() @ x).to(DTYPES[c["dw"]]))


# ----------------------------- the library's calls ------------------------ #
def _plan(s):
    """The buffers that a user's program keeps from call to call."""
    import routing_permute_grouped_router_gb300 as pkg

    c = s["case"]
    vec = dict(dtype=torch.float32, device=DEV)

    def empty(n, wanted=True):
        return torch.empty(n, **vec) if wanted else None

    if c["op"] == "join_fwd":
        return dict(pkg=pkg, out=torch.empty_like(s["x"]), h=torch.empty_like(s["x"]) if c["following"] else None,
                    rstd_post=empty(c["rows"], c["post"]), rstd_next=empty(c["rows"], c["following"]))
    if c["op"] == "join_bwd":
        grads = dict(dgamma_post=empty(c["d"], c["post"]), dgamma_next=empty(c["d"], c["following"]),
                     dgate=empty(c["d"], s["gate"] is not None), drow_gate=empty(c["rows"], s["row_gate"] is not None))
        return dict(pkg=pkg, dx=torch.empty_like(s["x"]), dy=torch.empty_like(s["x"]), grads=grads,
                    ws=pkg.residual_norm_workspace(c["rows"], c["d"], DEV))
    if c["op"] == "clip":
        flat = "grads" not in s
        grads = [s["flat_f32"], s["flat_bf16"]] if flat else s["grads"]
        out = None if math.isinf(s["max_norm"]) else [torch.empty_like(x) for x in grads]
        src, dst = grads, out
        if flat:
            sizes = (s["sizes_f32"], s["sizes_bf16"])
            src = [v for x, n in zip(grads, sizes) for v in x.split(n)]
            dst = None if out is None else [v for x, n in zip(out, sizes) for v in x.split(n)]
        return dict(pkg=pkg, list=pkg.grad_list(src, dst), out=out, norm=torch.empty(1, **vec),
                    ws=pkg.clip_workspace(len(src), DEV))
    ws = pkg.vocab_loss_workspace(c["T"], c["d"], c["V"], s["x"].dtype, c["op"] == "loss_bwd", DEV)
    if c["op"] == "loss_fwd":
        return dict(pkg=pkg, ws=ws, loss=empty(c["T"]), lse=empty(c["T"]))
    return dict(pkg=pkg, ws=ws, dx=torch.empty_like(s["x"]),
                dW=torch.empty(c["V"], c["d"], dtype=DTYPES[c["dw"]], device=DEV))


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    pkg, c = p["pkg"], s["case"]
    if c["op"] == "join_fwd":
        pkg.moe_residual_norm_fwd(s["x"], s["y"], p["out"], p["h"], s["gamma_post"], s["gamma_next"], s["gate"],
                                  s["row_gate"], c["rs"], c["bs"], EPS, p["rstd_post"], p["rstd_next"])
        return dict(out=p["out"], h=p["h"], rstd_post=p["rstd_post"], rstd_next=p["rstd_next"])
    if c["op"] == "join_bwd":
        pkg.moe_residual_norm_bwd(s["out"], s["y"], s["dh"], s["dout"], s["gamma_post"], s["gamma_next"], s["gate"],
                                  s["row_gate"], c["rs"], c["bs"], s["rstd_post"], s["rstd_next"], p["dx"], p["dy"],
                                  p["grads"], False, p["ws"])
        return dict(dx=p["dx"], dy=p["dy"], **{n: v for n, v in p["grads"].items() if v is not None})
    if c["op"] == "clip":
        pkg.moe_clip_grads(p["list"], s["max_norm"], p["norm"], p["ws"])
        norm = p["norm"][0]
        return dict(norm=norm) if p["out"] is None else dict(norm=norm, out=p["out"])
    if c["op"] == "loss_fwd":
        pkg.moe_vocab_loss_fwd(s["x"], s["W"], s["labels"], p["loss"], p["lse"], p["ws"])
        return dict(loss=p["loss"], lse=p["lse"])
    pkg.moe_vocab_loss_bwd(s["x"], s["W"], s["labels"], s["lse"], s["dloss"], p["dx"], p["dW"], False, p["ws"])
    return dict(dx=p["dx"], dW=p["dW"])


_PLAIN = dict(join_fwd=_plain_join_fwd, join_bwd=_plain_join_bwd, clip=_plain_clip, loss_fwd=_plain_loss_fwd,
              loss_bwd=_plain_loss_bwd)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ----------------------------- work --------------------------------------- #
def work(case):
    op = case["op"]
    if op == "clip":
        if case["sizes"] == "flat":
            sizes, half = _flat_sizes(case)
            n, b = sum(sizes), sum(k * (2 if h else 4) for k, h in zip(sizes, half))
        else:
            n = sum(math.prod(s) for s in _layer_shapes(case))
            b = n * (2 if case["dtype"] == "bf16" else 4)
        # the norm's sum; a clipped gradient is written as well
        return dict(bytes=b if math.isinf(case["ratio"]) else 2 * b, flops=2 * n if math.isinf(case["ratio"]) else 3 * n)
    es = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("join"):
        n, rows, d = case["rows"] * case["d"], case["rows"], case["d"]
        post, following = int(case["post"]), int(case["following"])
        vectors = 4 * d * (post + following + int(case["gate"] in ("channel", "both")))
        per_row = 4 * rows * (post + following + int(case["gate"] in ("row", "both")))
        if op == "join_fwd":
            return dict(bytes=(3 + following) * n * es + vectors + per_row, flops=(4 + 4 * post + 4 * following) * n)
        # dh with out, dout and y are read, dx and dy written
        tensors = 2 * following + int(case["dout"]) + 1 + 2
        return dict(bytes=tensors * n * es + 2 * vectors + per_row, flops=(4 + 10 * post + 10 * following) * n)
    T, d, V = case["T"], case["d"], case["V"]
    T -= int(case["ignored"] * T)
    if op == "loss_fwd":
        return dict(bytes=(T * d + V * d) * es + 12 * case["T"], flops=2.0 * T * d * V + 3.0 * T * V)
    dw = 2 if case["dw"] == "bf16" else 4
    return dict(bytes=(T * d + case["T"] * d + V * d) * es + V * d * dw + 12 * case["T"],
                flops=6.0 * T * d * V + 3.0 * T * V)


# ----------------------------- 64 bits ------------------------------------ #
def _mul(*factors):
    r = None
    for v in factors:
        if v is not None:
            r = v if r is None else r * v
    return r


def _exact_join(c, s):
    x, y, d = s["x"].double(), s["y"].double(), c["d"]
    post, nxt, gate = (None if s[n] is None else s[n].double() for n in ("gamma_post", "gamma_next", "gate"))
    row = None if s["row_gate"] is None else s["row_gate"].double()[:, None]
    scale = _mul(torch.full((1, 1), c["bs"], dtype=torch.float64, device=x.device), gate, row)
    if c["op"] == "join_fwd":
        ry = None if post is None else torch.rsqrt(torch.einsum("rd,rd->r", y, y) / d + EPS)
        u = y if post is None else torch.einsum("rd,r,d->rd", y, ry, post)
        out = torch.addcmul(x * c["rs"], scale.expand_as(u), u)
        if nxt is None:
            return dict(out=out, h=None, rstd_post=ry, rstd_next=None)
        ro = torch.rsqrt(torch.einsum("rd,rd->r", out, out) / d + EPS)
        return dict(out=out, h=torch.einsum("rd,r,d->rd", out, ro, nxt), rstd_post=ry, rstd_next=ro)
    res = {}
    D = torch.zeros_like(x) if s["dout"] is None else s["dout"].double()
    if nxt is not None:
        ro, dh, out = s["rstd_next"].double(), s["dh"].double(), s["out"].double()
        res["dgamma_next"] = torch.einsum("rd,rd,r->d", dh, out, ro)
        along = torch.einsum("rd,rd,d->r", dh, out, nxt) * ro ** 3 / d
        D = D + torch.einsum("rd,r,d->rd", dh, ro, nxt) - along[:, None] * out
    ry = None if post is None else s["rstd_post"].double()
    u = y if post is None else torch.einsum("rd,r,d->rd", y, ry, post)
    if gate is not None:
        res["dgate"] = c["bs"] * (D * u if row is None else D * u * row).sum(0)
    if row is not None:
        res["drow_gate"] = c["bs"] * (D * u if gate is None else D * u * gate).sum(1)
    du = D * scale
    if post is None:
        dy = du
    else:
        res["dgamma_post"] = torch.einsum("rd,rd,r->d", du, y, ry)
        along = torch.einsum("rd,rd,d->r", du, y, post) * ry ** 3 / d
        dy = torch.einsum("rd,r,d->rd", du, ry, post) - along[:, None] * y
    return dict(dx=D * c["rs"], dy=dy, **res)


def _exact_clip(c, s):
    grads = s["grads"] if "grads" in s else [s["flat_f32"], s["flat_bf16"]]
    norm = math.hypot(*(float(torch.linalg.vector_norm(p.double())) for g in grads for p in g.reshape(-1).split(1 << 26)))
    n = torch.tensor(norm, dtype=torch.float64)
    if math.isinf(s["max_norm"]):
        return dict(norm=n)
    scale = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
    return dict(norm=n, out=[g.double() * scale for g in grads])


def _exact_loss(c, s):
    valid = torch.nonzero(s["labels"] >= 0)[:, 0]
    x, at = s["x"][valid].double(), s["labels"][valid].long()
    T, dev = c["T"], x.device
    if c["op"] == "loss_fwd":
        lse = torch.full((len(valid),), -math.inf, dtype=torch.float64, device=dev)
        for W in s["W"].split(8192):
            lse = torch.logaddexp(lse, torch.logsumexp(x @ W.double().t(), 1))
        picked = torch.einsum("td,td->t", x, s["W"][at].double())
        zero = torch.zeros(T, dtype=torch.float64, device=dev)
        return dict(loss=zero.index_copy(0, valid, lse - picked), lse=zero.index_copy(0, valid, lse))
    g = (torch.full((len(valid),), 1.0 / max(1, len(valid)), dtype=torch.float64, device=dev) if s["dloss"] is None
         else s["dloss"][valid].double())
    # the softmax's part, a piece of the vocabulary at a time; then the labels' part
    dx, dW = torch.zeros_like(x), []
    for W in s["W"].split(8192):
        Wd = W.double()
        p = torch.exp(x @ Wd.t() - s["lse"][valid].double()[:, None]) * g[:, None]
        dx += p @ Wd
        dW.append(p.t() @ x)
    dx -= g[:, None] * s["W"][at].double()
    dW = torch.cat(dW).index_add(0, at, -g[:, None] * x)
    return dict(dx=torch.zeros(T, c["d"], dtype=torch.float64, device=dev).index_copy(0, valid, dx), dW=dW)


def exact(case, seed):
    if case["op"].startswith("loss"):
        # 64-bit products at about 1e12 operations a second
        if work(case)["flops"] > 1.2e13:
            return None
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(case, s)
    return (_exact_join if case["op"].startswith("join") else _exact_loss)(case, s)
