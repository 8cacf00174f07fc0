"""Cases, plain forms and work of the operators around one mixture-of-experts layer of a transformer block:

  decode       the whole layer for a few tokens (router, top-k, capacity, SwiGLU experts, combine), as a serving step calls it
  norm_fwd     layer norm in front of the layer: y, and the row mean and 1/std that training keeps
  norm_bwd     its backward pass: dx (with the gradient of the residual branch added), dgamma, dbeta
  dropout_fwd  out = residual + dropout(y) behind the layer, the mask drawn from a counter and never stored
  dropout_bwd  the same mask drawn again for the gradient

``run`` computes the plain form in elementary torch operations in 32 bits, or, where ``own`` is true, makes the
library's calls.  ``exact`` computes the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ----------------------------- cases -------------------------------------- #
def _decode(T, d, f, E, k, cf, zipf, dtype, residual):
    return dict(op="decode", T=T, d=d, f=f, E=E, k=k, cf=cf, zipf=zipf, dtype=dtype, residual=residual)


def _rows(op, rows, d, dtype, **more):
    return dict(op=op, rows=rows, d=d, dtype=dtype, **more)


def listed():
    return [
        # one token of one request through the dropless top-4 layer: the four picked experts' weights, and latency
        dict(name="decode_one_token", **_decode(1, 4096, 1536, 32, 4, 0.0, 1.3, "bf16", True)),
        # a batch of 16 requests through the skewed 64-expert layer, whose capacity of one row an expert drops picks
        dict(name="decode_16_zipf_e64", **_decode(16, 2048, 2048, 64, 2, 1.0, 1.1, "bf16", False)),
        # the largest batch of the few-token form: nearly every expert is read
        dict(name="decode_64_dropless_e32", **_decode(64, 4096, 1536, 32, 4, 0.0, 1.3, "bf16", True)),
        # a float32 layer, seven tokens, top-2 of eight experts with capacity factor 1.25
        dict(name="decode_7_top2_f32", **_decode(7, 1024, 4096, 8, 2, 1.25, 0.0, "f32", False)),
        # the norm of a decoding batch: launch latency
        dict(name="norm_fwd_16_rows", **_rows("norm_fwd", 16, 4096, "bf16")),
        # the norm of a training micro-batch of the dropless layer
        dict(name="norm_fwd_train", **_rows("norm_fwd", 32768, 4096, "bf16")),
        # its backward pass, with the residual branch's gradient
        dict(name="norm_bwd_train", **_rows("norm_bwd", 32768, 4096, "bf16", residual=True)),
        # a short micro-batch: few rows to spread the weight's gradient over
        dict(name="norm_bwd_333_rows", **_rows("norm_bwd", 333, 2048, "bf16", residual=False)),
        # float32 rows of an odd length, so no row but the first is aligned
        dict(name="norm_bwd_odd_f32", **_rows("norm_bwd", 4099, 1021, "f32", residual=True)),
        # residual dropout of a training micro-batch of the dropless layer
        dict(name="dropout_fwd_train", **_rows("dropout_fwd", 32768, 4096, "bf16", p=0.1, residual=True)),
        # its gradient at the size of the 16-expert layer's micro-batch
        dict(name="dropout_bwd_train", **_rows("dropout_bwd", 8192, 2048, "bf16", p=0.1)),
        # a small float32 tensor whose length is no multiple of a draw's eight elements
        dict(name="dropout_fwd_odd_f32", **_rows("dropout_fwd", 257, 129, "f32", p=0.5, residual=True)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, step, hi):
    """A multiple of step up to hi, spread over its logarithm; 12 * 256 is left to its neighbour."""
    n = step * _log(rng, max(1, 64 // step), hi // step)
    return n + step if n == 12 * 256 else n


def draw(rng):
    op = rng.choice(["decode", "decode", "norm_fwd", "norm_bwd", "dropout_fwd", "dropout_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "decode":
        E = rng.choice([4, 7, 8, 16, 32, 48, 64, 128])
        if dtype == "bf16":
            d, f = _size(rng, 256, 4096), _size(rng, 256, 4096)
        else:
            d, f = _size(rng, 4, 2048), _size(rng, 4, 2048)
        while E > 4 and E * d * f > 32 * 4096 * 1536 // (1 if dtype == "bf16" else 4):
            E //= 2
        k = rng.randint(1, min(E, 8))
        return _decode(_log(rng, 1, 64), d, f, E, k, rng.choice([0.0, 1.0, 1.25]), rng.choice([0.0, 1.1, 1.3]),
                       dtype, rng.random() < 0.5)
    d = _size(rng, rng.choice([1, 8]), 8192)
    rows = min(_log(rng, 1, 32768), 32768 * 4096 // d // (2 if dtype == "f32" else 1))
    if op == "norm_fwd":
        return _rows(op, rows, d, dtype)
    if op == "norm_bwd":
        return _rows(op, rows, d, dtype, residual=rng.random() < 0.5)
    p = round(rng.uniform(0.02, 0.6), 3)
    if op == "dropout_fwd":
        return _rows(op, rows, d, dtype, p=p, residual=rng.random() < 0.7)
    return _rows(op, rows, d, dtype, p=p)


# ----------------------------- inputs ------------------------------------- #
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)

    s = dict(case=dict(case))
    if case["op"] == "decode":
        T, d, f, E, k = (case[n] for n in ("T", "d", "f", "E", "k"))
        s["W_r"] = normal(d, E, scale=d ** -0.5, dtype=torch.float32)
        s["bias"] = None
        if case["zipf"] > 0:  # the router's picks follow (e + 1)^-zipf
            s["bias"] = -case["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
        for n, shape, scale in (("W1", (E, d, f), d ** -0.5), ("W3", (E, d, f), d ** -0.5), ("W2", (E, f, d), f ** -0.5)):
            w = torch.empty(*shape, device=DEV, dtype=t)
            for e in range(E):
                w[e] = normal(*shape[1:], scale=scale)
            s[n] = w
        # tokens whose picks no rounding of the scores can change: gaps of 1e-3 among the top k + 1
        x = normal(3 * T + 64, d)
        top = (x.double() @ s["W_r"].double() + (0 if s["bias"] is None else s["bias"].double())).sort(1, True)[0]
        top = top[:, : min(k + 1, E)]
        near = ((top[:, :-1] - top[:, 1:]) < 1e-3).any(1) if top.shape[1] > 1 else torch.zeros(len(x), dtype=torch.bool, device=DEV)
        s["x"] = x[near.int().sort(stable=True)[1][:T]].contiguous()
        s["residual"] = normal(T, d) if case["residual"] else None
        return s
    rows, d = case["rows"], case["d"]
    if case["op"].startswith("norm"):
        # rows of a residual stream: their own scale and mean, a few channels far larger than the others
        x = normal(rows, d, dtype=torch.float32)
        x *= 0.5 + 1.5 * torch.rand(rows, 1, generator=g, device=DEV)
        x += 0.2 * normal(rows, 1, dtype=torch.float32)
        x[:, torch.randint(0, d, (max(1, d // 512),), generator=g, device=DEV)] *= 8.0
        s["x"] = x.to(t)
        del x
        s["gamma"] = 1.0 + normal(d, scale=0.2, dtype=torch.float32)
        s["beta"] = normal(d, scale=0.1, dtype=torch.float32)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, d)
            s["dres"] = normal(rows, d) if case["residual"] else None
            # what the forward pass has kept
            s["mean"] = s["x"].double().mean(1).float() if rows * d <= 1 << 24 else s["x"].float().mean(1)
            c = s["x"].float() - s["mean"][:, None]
            s["rstd"] = torch.rsqrt((c * c).mean(1) + EPS)
        return s
    s["y"] = normal(rows, d)
    s["residual"] = normal(rows, d) if case.get("residual") else None
    # a training program's seed, and its step as the offset
    s["seed"] = (0x5DEECE66D * (seed + 1) + 0xB) & (2 ** 62 - 1)
    s["offset"] = 2 ** 33 + 7 * seed
    return s


# ----------------------------- plain forms -------------------------------- #
def _plain_decode(s):
    c, x, W_r = s["case"], s["x"].float(), s["W_r"]
    T, E, k = c["T"], c["E"], c["k"]
    scores = x @ W_r if s["bias"] is None else x @ W_r + s["bias"]
    ids = torch.sort(scores, dim=1, descending=True, stable=True)[1][:, :k]
    probs = torch.exp(scores - scores.max(1, keepdim=True)[0])
    probs = probs / probs.sum(1, keepdim=True)
    gates = probs.gather(1, ids)
    if k > 1:
        gates = gates / gates.sum(1, keepdim=True)
    # an expert's rows: first choices in token order, then second choices, ...; those past its capacity are dropped
    kept = gates
    if c["cf"] > 0:
        cap = math.ceil(float(np.float32(c["cf"])) * T * k / E)
        one = (ids.t().reshape(-1, 1) == torch.arange(E, device=ids.device)).int()
        slot = ((one.cumsum(0) - 1) * one).sum(1).reshape(k, T).t()
        kept = gates * (slot < cap)
    if T * k < E:  # the picked experts' weights alone
        at = ids.reshape(-1)
        xs = x.repeat_interleave(k, 0)[:, None, :]
        a, b = torch.bmm(xs, s["W1"][at].float()), torch.bmm(xs, s["W3"][at].float())
        h = a / (1 + torch.exp(-a)) * b
        y = (torch.bmm(h, s["W2"][at].float()).reshape(T, k, -1) * kept[:, :, None]).sum(1)
    else:  # every expert for every token, the unpicked ones with weight 0
        a, b = torch.matmul(x, s["W1"].float()), torch.matmul(x, s["W3"].float())
        h = a / (1 + torch.exp(-a)) * b
        w = torch.zeros_like(scores).scatter_(1, ids, kept)
        y = (torch.matmul(h, s["W2"].float()) * w.t()[:, :, None]).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return dict(y=y.to(s["x"].dtype), ids=ids.int(), gates=gates)


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_bwd(s):
    n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    dgamma, dbeta = (dy * n).sum(0), dy.sum(0)
    dn = dy * s["gamma"]
    dx = (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["x"].dtype), dgamma=dgamma, dbeta=dbeta)


def _mul32(a, m):
    """High and low 32 bits of a * m for a in [0, 2^32) held in int64."""
    lo, hi = a * (m & 0xFFFF), a * (m >> 16)
    return (hi + (lo >> 16)) >> 16, (a * m) & 0xFFFFFFFF


def _plain_keep(n, p, seed, offset, device):
    """Which of n elements are kept: 16 bits for each, eight elements to a Philox-4x32-10 block (Salmon et al., 2011)
    with the counter (block, offset) and the key seed.  Also the scale of the kept ones."""
    cut = int(p * 65536 + 0.5)
    b = torch.arange((n + 7) // 8, device=device, dtype=torch.int64)
    c0, c1 = b & 0xFFFFFFFF, b >> 32
    c2, c3 = torch.full_like(b, offset & 0xFFFFFFFF), torch.full_like(b, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):  # the generator's ten rounds
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = torch.stack([c0, c1, c2, c3], 1)
    u = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    return u >= cut, 65536 / (65536 - cut)


def _plain_dropout(s):
    c, y = s["case"], s["y"]
    keep, scale = _plain_keep(y.numel(), c["p"], s["seed"], s["offset"], y.device)
    out = torch.where(keep.reshape(y.shape), y.float() * scale, 0.0)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return dict(out=out.to(y.dtype))


# ----------------------------- the library's calls ------------------------ #
def _plan(s):
    """The buffers that a user's program keeps from call to call."""
    import routing_permute_grouped_router_gb300 as pkg

    c = s["case"]
    if c["op"] == "decode":
        cfg = pkg.config(c["T"], c["d"], c["f"], c["E"], c["k"], c["cf"], -1,
                         pkg.MOE_BF16 if c["dtype"] == "bf16" else pkg.MOE_F32)
        return dict(pkg=pkg, cfg=cfg, ws=pkg.decode_workspace(cfg, DEV),
                    weights=dict(W_r=s["W_r"], bias=s["bias"], W1=s["W1"], W3=s["W3"], W2=s["W2"]),
                    y=torch.empty_like(s["x"]), ids=torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV),
                    gates=torch.empty(c["T"], c["k"], dtype=torch.float32, device=DEV))
    vec = dict(dtype=torch.float32, device=DEV)
    if c["op"] == "norm_fwd":
        return dict(pkg=pkg, y=torch.empty_like(s["x"]), mean=torch.empty(c["rows"], **vec),
                    rstd=torch.empty(c["rows"], **vec))
    if c["op"] == "norm_bwd":
        return dict(pkg=pkg, dx=torch.empty_like(s["x"]), dgamma=torch.empty(c["d"], **vec),
                    dbeta=torch.empty(c["d"], **vec), ws=pkg.norm_workspace(c["rows"], c["d"], DEV))
    return dict(pkg=pkg, out=torch.empty_like(s["y"]))


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    pkg, c = p["pkg"], s["case"]
    if c["op"] == "decode":
        pkg.moe_layer_decode(p["cfg"], p["weights"], s["x"], s["residual"], p["y"], p["ids"], p["gates"], p["ws"])
        return dict(y=p["y"], ids=p["ids"], gates=p["gates"])
    if c["op"] == "norm_fwd":
        pkg.moe_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, p["y"], p["mean"], p["rstd"])
        return dict(y=p["y"], mean=p["mean"], rstd=p["rstd"])
    if c["op"] == "norm_bwd":
        pkg.moe_norm_bwd(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], s["dres"], p["dx"], p["dgamma"], p["dbeta"],
                         False, p["ws"])
        return dict(dx=p["dx"], dgamma=p["dgamma"], dbeta=p["dbeta"])
    if c["op"] == "dropout_fwd":
        pkg.moe_dropout_add(s["y"], s["residual"], p["out"], c["p"], s["seed"], s["offset"])
    else:
        pkg.moe_dropout_bwd(s["y"], p["out"], c["p"], s["seed"], s["offset"])
    return dict(out=p["out"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "decode":
        return _plain_decode(state)
    if op == "norm_fwd":
        return _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    return _plain_dropout(state)


# ----------------------------- work --------------------------------------- #
def _picked_experts(c):
    """Experts that a step of T tokens picks, on average over draws of the scores."""
    T, E, k = c["T"], c["E"], c["k"]
    rng = np.random.default_rng(5)
    s = rng.standard_normal((32, T, E)) - c["zipf"] * np.log(np.arange(1, E + 1))
    ids = np.argsort(-s, axis=2)[:, :, :k].reshape(32, -1)
    return float(np.mean([len(np.unique(r)) for r in ids]))


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "decode":
        T, d, f, E, k = (case[n] for n in ("T", "d", "f", "E", "k"))
        tokens = T * d * es * (3 if case["residual"] else 2) + T * k * 8
        return dict(bytes=_picked_experts(case) * 3 * d * f * es + d * E * 4 + tokens,
                    flops=2.0 * T * d * E + 2.0 * T * k * 3 * d * f)
    n = case["rows"] * case["d"]
    if case["op"] == "norm_fwd":
        return dict(bytes=2 * n * es + 8 * case["d"] + 8 * case["rows"], flops=8 * n)
    if case["op"] == "norm_bwd":
        return dict(bytes=(4 if case["residual"] else 3) * n * es + 12 * case["d"] + 8 * case["rows"], flops=14 * n)
    # a block of eight draws is ten rounds of two 32-bit products and two three-way exclusive ors
    return dict(bytes=(3 if case.get("residual") else 2) * n * es, flops=(40 / 8 + 3) * n)


# ----------------------------- 64 bits ------------------------------------ #
def _exact_decode(c, s):
    x = s["x"].double()
    score = x @ s["W_r"].double()
    if s["bias"] is not None:
        score += s["bias"].double()
    ids = torch.argsort(score, dim=1, descending=True, stable=True)[:, : c["k"]]
    g = torch.softmax(score, 1).gather(1, ids)
    if c["k"] > 1:
        g = torch.softmax(score.gather(1, ids), 1)
    cap = math.ceil(float(np.float32(c["cf"])) * c["T"] * c["k"] / c["E"]) if c["cf"] > 0 else c["T"] * c["k"]
    used, host = [0] * c["E"], ids.tolist()
    rows = [[] for _ in range(c["E"])]
    for j in range(c["k"]):
        for t in range(c["T"]):
            e = host[t][j]
            if used[e] < cap:
                used[e] += 1
                rows[e].append((t, j))
    y = torch.zeros(c["T"], c["d"], dtype=torch.float64, device=x.device)
    for e, r in enumerate(rows):
        if r:
            t, j = (torch.tensor(v, device=x.device) for v in zip(*r))
            a = x[t] @ s["W1"][e].double()
            h = a * torch.sigmoid(a) * (x[t] @ s["W3"][e].double())
            y[t] += g[t, j][:, None] * (h @ s["W2"][e].double())
    if s["residual"] is not None:
        y += s["residual"].double()
    return dict(y=y, ids=ids.int(), gates=g)


def _exact_keep(n, p, seed, offset):
    cut = np.uint64(int(p * 65536 + 0.5))
    m32, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    c = [i & m32, i >> s32, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> s32) ^ c[1] ^ np.uint64(key[0]), p1 & m32, (p0 >> s32) ^ c[3] ^ np.uint64(key[1]), p0 & m32]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    u = np.stack([c[j // 2] >> np.uint64(16 * (j % 2)) & np.uint64(0xFFFF) for j in range(8)], 1).reshape(-1)[:n]
    return u >= cut


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"].startswith("norm"):
        x, gamma = s["x"].double(), s["gamma"].double()
        if case["op"] == "norm_fwd":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["beta"].double(), x.sub_(mean[:, None]).mul_(rstd[:, None]), gamma)
            return dict(y=y, mean=mean, rstd=rstd)
        rstd = s["rstd"].double()[:, None]
        n = x.sub_(s["mean"].double()[:, None]).mul_(rstd)
        dy = s["dy"].double()
        out = dict(dgamma=torch.einsum("rd,rd->d", dy, n), dbeta=dy.sum(0))
        v = dy.mul_(gamma)
        m1, m2 = v.mean(1, keepdim=True), torch.einsum("rd,rd->r", v, n)[:, None] / case["d"]
        dx = v.sub_(m1).sub_(n.mul_(m2)).mul_(rstd)
        return dict(dx=dx if s["dres"] is None else dx.add_(s["dres"].double()), **out)
    y = s["y"].double().cpu().numpy().reshape(-1)
    cut = int(case["p"] * 65536 + 0.5)
    out = np.where(_exact_keep(y.size, case["p"], s["seed"], s["offset"]), y * (65536 / (65536 - cut)), 0.0)
    if s["residual"] is not None:
        out = out + s["residual"].double().cpu().numpy().reshape(-1)
    return dict(out=out.reshape(case["rows"], case["d"]))
