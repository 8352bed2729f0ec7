"""The operators of a Muon + layer-norm training step, as cases that can be timed.

Each case names one pass of one operator:

* ``norm``      layer norm's forward pass (optionally of x + residual);
* ``norm_grad`` its backward pass with the reduction of the weight's and the
                bias's gradients;
* ``ortho``     the Newton-Schulz orthogonalisation of a batch of update
                matrices;
* ``momentum``  the mean of the N_d gradient contributions, the momentum
                update and the (Nesterov) update matrix;
* ``apply``     the weight update with decoupled decay and the bf16 copy.

``run`` computes the plain form in elementary torch operations in 32 bits
where ``own`` is false, and calls the framework where it is true.
"""

from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
COEFFS = (3.4445, -4.7750, 2.0315)  # Newton-Schulz quintic of the Muon optimiser
STEPS = 5
NORM_EPS, ORTHO_EPS = 1e-5, 1e-7
MU, LR, DECAY, SCALE = 0.95, 0.02, 0.1, 0.2


def listed():
    return [
        # one token's hidden state of a 13B block: the latency of a call
        _norm("norm", "norm-one-token", 1, 5120, "bf16", "bf16", residual=False, pad=0),
        # a pre-norm block's residual add and norm over a 4 x 2048-token batch
        _norm("norm", "norm-batch", 8192, 5120, "bf16", "bf16", residual=True, pad=0),
        # the tail of a ragged micro-batch in full precision, odd width and stride
        _norm("norm_grad", "norm-grad-ragged", 37, 1601, "f32", "f32", residual=False, pad=3),
        # the backward pass of the batch above, its residual gradient joined in
        _norm("norm_grad", "norm-grad-batch", 8192, 5120, "bf16", "bf16", residual=True, pad=0),
        # an adapter's small matrix: latency
        _ortho("ortho-adapter", 1, 96, 128, "f32", pad=0),
        # the matrices of four small blocks, one call
        _ortho("ortho-blocks", 4, 1024, 1024, "bf16", pad=0),
        # an attention projection of the 13B layout, fp32 momentum
        _ortho("ortho-projection", 1, 5120, 5120, "f32", pad=0),
        # a feed-forward matrix of the 13B layout, tall
        _ortho("ortho-feed-forward", 1, 13824, 5120, "bf16", pad=0),
        # one 1024 x 1024 matrix over 4 ranks (the smallest shard of the workloads)
        _momentum("momentum-small", 4, 1 << 20, "bf16"),
        # an attention projection of the 13B layout over 16 ranks
        _momentum("momentum-projection", 16, 5120 * 5120, "f32"),
        # an odd-sized small shard
        _apply("apply-small", 1_000_003),
        # a feed-forward matrix of the 13B layout
        _apply("apply-feed-forward", 5120 * 13824),
    ]


def draw(rng):
    """One more case of the same ranges."""
    def spread(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["norm", "norm_grad", "ortho", "ortho", "momentum", "apply"])
    if op in ("norm", "norm_grad"):
        cols = spread(32, 13824)
        rows = spread(1, min(16384, 8192 * 5120 // cols))
        kind = rng.choice(["f32", "bf16", "f16"])
        return _norm(op, None, rows, cols, kind, rng.choice([kind, "f32"]),
                     residual=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 8]))
    if op == "ortho":
        rows, cols = spread(16, 13824), spread(16, 13824)
        short = min(rows, cols, 5120)
        rows, cols = (short, cols) if rows <= cols else (rows, short)
        most = 5120 * 5120 * 13824 // (short * short * max(rows, cols))
        batch = spread(1, max(1, min(16, most)))
        return _ortho(None, batch, rows, cols, rng.choice(["f32", "bf16", "f16"]),
                      pad=rng.choice([0, 0, 5]))
    if op == "momentum":
        n_d = spread(1, 64)
        return _momentum(None, n_d, spread(1000, 16 * 5120 * 5120 // max(16, n_d)),
                         rng.choice(["f32", "bf16"]))
    return _apply(None, spread(1000, 5120 * 13824))


def _named(name, case):
    return {"name": name, **case} if name else case


def _norm(op, name, rows, cols, kind, params, residual, pad):
    return _named(name, {"op": op, "rows": rows, "cols": cols, "type": kind, "params": params,
                         "residual": residual, "pad": pad})


def _ortho(name, batch, rows, cols, kind, pad):
    return _named(name, {"op": "ortho", "batch": batch, "rows": rows, "cols": cols, "type": kind,
                         "pad": pad})


def _momentum(name, n_d, n, update):
    return _named(name, {"op": "momentum", "n_d": n_d, "n": n, "update": update})


def _apply(name, n):
    return _named(name, {"op": "apply", "n": n})


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        r, d, t, p = case["rows"], case["cols"], SIZE[case["type"]], SIZE[case["params"]]
        if op == "norm":  # x (+ residual) in, y (+ sum) out, gamma and beta, mean and rstd
            return {"bytes": r * d * t * (4 if case["residual"] else 2) + 2 * d * p + 8 * r,
                    "flops": 8 * r * d}
        # dy and x (+ the sum's gradient) in, dx out, gamma in, two gradients out
        return {"bytes": r * d * t * (4 if case["residual"] else 3) + 3 * d * p + 8 * r,
                "flops": 15 * r * d}
    if op == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        # X X^T and A A are symmetric: half of each product is enough
        return {"bytes": case["batch"] * m * n * (SIZE[case["type"]] + 2),
                "flops": case["batch"] * STEPS * (3 * m * m * n + m * m * m)}
    if op == "momentum":
        n, k = case["n"], case["n_d"]
        return {"bytes": n * (2 * k + 8 + SIZE[case["update"]]), "flops": n * (k + 5)}
    return {"bytes": case["n"] * 12, "flops": case["n"] * 4}


def _rows(g, rows, cols, kind, pad, scale=1.0):
    """Rows of a wider buffer when pad > 0 (the row stride is cols + pad)."""
    a = torch.randn(rows, cols + pad, device="cuda", generator=g) * scale
    return a.to(TYPES[kind])[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        r, d, kind, pad = case["rows"], case["cols"], case["type"], case["pad"]
        # hidden states: rows of differing size, a few columns that stand out
        size = torch.exp(0.5 * torch.randn(r, 1, device="cuda", generator=g))
        wide = 1.0 + 9.0 * (torch.rand(d, device="cuda", generator=g) < 0.01)
        x = (torch.randn(r, d + pad, device="cuda", generator=g)[:, :d] * wide + 0.3) * size
        x = torch.nn.functional.pad(x, (0, pad)).to(TYPES[kind])[:, :d]
        ptype = TYPES[case["params"]]
        s["x"] = x
        s["gamma"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(ptype)
        s["beta"] = (0.1 * torch.randn(d, device="cuda", generator=g)).to(ptype)
        if op == "norm":
            s["residual"] = _rows(g, r, d, kind, pad) if case["residual"] else None
        else:
            s["dy"] = _rows(g, r, d, kind, pad)
            s["dsum"] = _rows(g, r, d, kind, pad) if case["residual"] else None
            xf = x.double()
            mean = xf.mean(1)
            var = ((xf - mean[:, None]) ** 2).mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (1.0 / torch.sqrt(var + NORM_EPS)).float()
    elif op == "ortho":
        b, r, c, pad = case["batch"], case["rows"], case["cols"], case["pad"]
        # a momentum matrix: rows of differing size
        size = 1e-3 * torch.exp(0.5 * torch.randn(b, r, 1, device="cuda", generator=g))
        a = torch.randn(b, r, c + pad, device="cuda", generator=g) * size
        s["g"] = a.to(TYPES[case["type"]])[:, :, :c]
    elif op == "momentum":
        n, k = case["n"], case["n_d"]
        stride = (n + 7) // 8 * 8  # every rank's row starts on a 16-byte boundary
        rows = torch.empty(k, stride, device="cuda", dtype=torch.bfloat16)
        for i in range(k):
            rows[i] = (1e-3 * torch.randn(stride, device="cuda", generator=g)).bfloat16()
        s["rows"] = rows[:, :n]
        s["m"] = 1e-2 * torch.randn(n, device="cuda", generator=g)
    else:
        n = case["n"]
        s["master"] = 0.02 * torch.randn(n, device="cuda", generator=g)
        s["o"] = (0.01 * torch.randn(n, device="cuda", generator=g)).bfloat16()
    if own:
        _plan(case, s)
    return s


def _plan(case, s):
    """What a program that uses the framework keeps: owner objects with their
    workspaces, and the buffers that the results go into."""
    import sharded_mixed_precision_zero_amd as Z

    op = case["op"]
    if op in ("norm", "norm_grad"):
        t = TYPES[case["type"]]
        r, d = case["rows"], case["cols"]
        s["plan"] = Z.ZeroLayerNorm(rows=r, cols=d, dtype=t, param_dtype=TYPES[case["params"]],
                                    eps=NORM_EPS)
        s["out"] = torch.empty(r, d, device="cuda", dtype=t)
        if op == "norm":
            s["sum"] = torch.empty_like(s["out"]) if case["residual"] else None
        else:
            s["dgamma"] = torch.empty_like(s["gamma"])
            s["dbeta"] = torch.empty_like(s["beta"])
    elif op == "ortho":
        s["out"] = torch.empty(case["batch"], case["rows"], case["cols"], device="cuda",
                               dtype=torch.bfloat16)
        s["plan"] = Z.ZeroOrtho(batch=case["batch"], rows=case["rows"], cols=case["cols"],
                                dtype=TYPES[case["type"]], steps=STEPS, coeffs=COEFFS,
                                eps=ORTHO_EPS)
    elif op == "momentum":
        s["plan"] = Z.muon_desc(n=case["n"], n_d=case["n_d"], mu=MU, nesterov=True,
                                dtype=TYPES[case["update"]])
        s["table"] = Z.contrib_table(s["rows"])
        s["m_out"] = torch.empty_like(s["m"])
        s["u"] = torch.empty(case["n"], device="cuda", dtype=TYPES[case["update"]])
    else:
        s["plan"] = Z.muon_desc(n=case["n"], n_d=1, weight_decay=DECAY)
        s["master_out"] = torch.empty_like(s["master"])
        s["p"] = torch.empty(case["n"], device="cuda", dtype=torch.bfloat16)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _OWN[op](case, state)
    return _PLAIN[op](case, state)


# ------------------------------------------------------------ the framework

def _own_norm(case, s):
    plan = s["plan"]
    plan.forward(s["x"], s["out"], gamma=s["gamma"], beta=s["beta"], residual=s["residual"],
                 sum_out=s["sum"])
    out = {"y": s["out"], "mean": plan.mean, "rstd": plan.rstd}
    if case["residual"]:
        out["sum"] = s["sum"]
    return out


def _own_norm_grad(case, s):
    s["plan"].backward(s["dy"], s["x"], s["out"], gamma=s["gamma"], dgamma=s["dgamma"],
                       dbeta=s["dbeta"], dsum=s["dsum"], mean=s["mean"], rstd=s["rstd"])
    return {"dx": s["out"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _own_ortho(case, s):
    s["plan"](s["g"], s["out"])
    return {"o": s["out"]}


def _own_momentum(case, s):
    import sharded_mixed_precision_zero_amd as Z

    Z.check(Z.zero_shard_muon_momentum(s["plan"], s["table"], s["m"], s["m_out"], s["u"]))
    return {"m": s["m_out"], "u": s["u"]}


def _own_apply(case, s):
    import sharded_mixed_precision_zero_amd as Z

    Z.check(Z.zero_shard_muon_apply(s["plan"], s["o"], LR, SCALE, s["master"], s["master_out"],
                                    s["p"]))
    return {"master": s["master_out"], "p": s["p"]}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "ortho": _own_ortho,
        "momentum": _own_momentum, "apply": _own_apply}


# ------------------------------------------------------------ the plain form

def _plain_norm(case, s):
    t = TYPES[case["type"]]
    x = s["x"].float()
    out = {}
    if case["residual"]:
        total = (x + s["residual"].float()).to(t)
        x = total.float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1) + NORM_EPS)
    y = centred * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    out = {"y": y.to(t), "mean": mean, "rstd": rstd}
    if case["residual"]:
        out["sum"] = total
    return out


def _plain_norm_grad(case, s):
    t = TYPES[case["type"]]
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    c1 = g.mean(1, keepdim=True)
    c2 = (g * xhat).mean(1, keepdim=True)
    dx = s["rstd"][:, None] * (g - c1 - xhat * c2)
    if case["residual"]:
        dx = dx + s["dsum"].float()
    p = s["gamma"].dtype
    return {"dx": dx.to(t), "dgamma": (dy * xhat).sum(0).to(p), "dbeta": dy.sum(0).to(p)}


def _plain_ortho(case, s):
    a, b, c = COEFFS
    x = s["g"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        x = x.mT
    norm = torch.sqrt((x * x).sum((1, 2), keepdim=True))
    x = (x / (norm + ORTHO_EPS)).contiguous()
    for _ in range(STEPS):
        gram = x @ x.mT.contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.mT
    return {"o": x.to(torch.bfloat16).contiguous()}


def _plain_momentum(case, s):
    gbar = s["rows"].sum(0, dtype=torch.float32) / case["n_d"]
    m = MU * s["m"] + gbar
    return {"m": m, "u": (gbar + MU * m).to(TYPES[case["update"]])}


def _plain_apply(case, s):
    w = s["master"]
    w = w - (LR * DECAY) * w - (LR * SCALE) * s["o"].float()
    return {"master": w, "p": w.to(torch.bfloat16)}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "ortho": _plain_ortho,
          "momentum": _plain_momentum, "apply": _plain_apply}


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False  # inputs only
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    f32 = {k: float(torch.tensor(v)) for k, v in (("mu", MU), ("lr", LR), ("decay", DECAY),
                                                   ("scale", SCALE))}
    if op == "norm":
        x, out = s["x"].double(), {}
        if case["residual"]:
            out["sum"] = (x + s["residual"].double()).to(TYPES[case["type"]]).double()
            x = out["sum"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + NORM_EPS)
        y = torch.addcmul(s["beta"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1),
                          s["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd, **out}
    if op == "norm_grad":
        n = case["cols"]
        dy, rstd = s["dy"].double(), s["rstd"].double().unsqueeze(1)
        xhat = (s["x"].double() - s["mean"].double().unsqueeze(1)) * rstd
        g = dy * s["gamma"].double()
        # the projection of g off the span of 1 and xhat, as inner products
        along = torch.einsum("rd,rd->r", g, xhat).unsqueeze(1) / n
        dx = (g - g.sum(1, keepdim=True) / n - along * xhat) * rstd
        if case["residual"]:
            dx += s["dsum"].double()
        return {"dx": dx, "dgamma": torch.einsum("rd,rd->d", dy, xhat), "dbeta": dy.sum(0)}
    if op == "ortho":
        a, b, c = COEFFS
        out = []
        for i in range(case["batch"]):
            x = s["g"][i].double()
            x = x / (torch.linalg.norm(x) + ORTHO_EPS)
            left = case["rows"] <= case["cols"]
            for _ in range(STEPS):
                gram = x @ x.T if left else x.T @ x
                poly = b * gram + c * (gram @ gram)
                poly.diagonal().add_(a)
                x = poly @ x if left else x @ poly
            out.append(x)
        return {"o": torch.stack(out)}
    if op == "momentum":
        gbar = torch.zeros(case["n"], device="cuda", dtype=torch.float64)
        for i in range(case["n_d"]):
            gbar += s["rows"][i].double()
        gbar /= case["n_d"]
        m = f32["mu"] * s["m"].double() + gbar
        return {"m": m, "u": gbar + f32["mu"] * m}
    w = s["master"].double()
    w = w * (1 - f32["lr"] * f32["decay"]) - f32["lr"] * f32["scale"] * s["o"].double()
    return {"master": w, "p": w}
