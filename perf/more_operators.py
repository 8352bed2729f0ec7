"""The operators around the matrices of a training step, as cases that can be timed.

Each case names one pass of one operator:

* ``seam``         the seam between two blocks: the norm of a block's output, its gate,
                   the scaled residual sum, and the norm before the next block;
* ``seam_grad``    its backward pass, with the gradients of both norms and the gate;
* ``lookup``       the embedding of tokens, scaled;
* ``lookup_grad``  the gradient of the embedding's table;
* ``adamw``        the AdamW step of many tensors, with states in 32 bits, or in 8 (scaled
                   blocks of 256, rounded stochastically), and the norm that clips it.

``run`` computes the plain form in elementary torch operations in 32 bits where ``own`` is
false (in 64 where the rounding of a state to 8 bits depends on it), and calls the framework
where it is true.
"""

from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
EPS = 1e-5
BETA1, BETA2, ADAM_EPS, LR, DECAY, MAX_NORM, T = 0.9, 0.999, 1e-8, 3e-4, 0.1, 1.0, 100
BLOCK = 256  # elements that share a scale in an 8-bit state
WORD = 0xFFFFFFFF


def listed():
    return [
        # one token's hidden state between two 13B blocks: the latency of a call
        _seam("seam", "seam-one-token", 1, 5120, "bf16", "bf16", "rms", "column", 0),
        # the same seam over a 4 x 2048-token batch, gains kept in full precision
        _seam("seam", "seam-batch", 8192, 5120, "bf16", "f32", "layer", "column", 0),
        # the tail of a ragged micro-batch in full precision, odd width and stride
        _seam("seam_grad", "seam-grad-ragged", 37, 1601, "f32", "f32", "layer", "sigmoid", 3),
        # the backward pass over a 4 x 2048-token batch
        _seam("seam_grad", "seam-grad-batch", 8192, 5120, "bf16", "bf16", "rms", "column", 0),
        # the next tokens of 16 sequences: latency
        _lookup("lookup", "lookup-few", 16, 5120, 32000, "bf16", "bf16"),
        # a 32 x 2048-token batch out of one rank's copy of the table
        _lookup("lookup", "lookup-batch", 65536, 5120, 32000, "bf16", "bf16"),
        # a small model's table in full precision, odd width, a ragged micro-batch
        _lookup("lookup_grad", "lookup-grad-ragged", 333, 1601, 1009, "f32", "f32"),
        # the 13B layout's table over a 4 x 2048-token batch
        _lookup("lookup_grad", "lookup-grad-batch", 8192, 5120, 32000, "bf16", "bf16"),
        # the gains of a 40-block model: many short tensors
        _adamw("adamw-gains", 0, 0, 160, 5120, "bf16", clip=False),
        # the 13B layout's table in 8 bits beside its gains, clipped
        _adamw("adamw-table", 1, 32000 * 5120, 81, 5120, "bf16", clip=True),
        # odd-sized tensors with full-precision gradients, in 8 bits
        _adamw("adamw-odd", 24, 1_000_003, 0, 0, "f32", clip=False),
        # the 13B layout's table with its state in 32 bits
        _adamw("adamw-table-32", 0, 0, 1, 32000 * 5120, "bf16", clip=False),
    ]


def draw(rng):
    """One more case of the same ranges."""
    def spread(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["seam", "seam_grad", "lookup", "lookup_grad", "adamw", "adamw"])
    if op in ("seam", "seam_grad"):
        cols = spread(32, 16384)
        rows = spread(1, min(16384, 8192 * 5120 // cols))
        kind = rng.choice(["f32", "bf16", "f16"])
        return _seam(op, None, rows, cols, kind, rng.choice([kind, "f32"]),
                     rng.choice(["rms", "layer"]), rng.choice(["none", "column", "sigmoid"]),
                     pad=rng.choice([0, 0, 3, 8]))
    if op in ("lookup", "lookup_grad"):
        cols = spread(64, 8192)
        tokens = spread(1, min(65536, (65536 if op == "lookup" else 16384) * 5120 // cols))
        vocab = spread(16, min(128000, 32000 * 5120 // cols))
        kind = rng.choice(["f32", "bf16", "f16"])
        return _lookup(op, None, tokens, cols, vocab, kind, rng.choice([kind, "f32"]))
    n8, n32 = spread(256, 32000 * 5120), spread(1, 8_000_000)
    many8 = spread(1, max(1, min(64, 32000 * 5120 // n8)))
    many32 = spread(1, max(1, min(256, 16_000_000 // n32)))
    which = rng.choice(["8", "32", "both"])
    return _adamw(None, 0 if which == "32" else many8, 0 if which == "32" else n8,
                  0 if which == "8" else many32, 0 if which == "8" else n32,
                  rng.choice(["f32", "bf16", "f16"]), clip=rng.random() < 0.5)


def _named(name, case):
    return {"name": name, **case} if name else case


def _seam(op, name, rows, cols, kind, params, norm, gate, pad):
    return _named(name, {"op": op, "rows": rows, "cols": cols, "type": kind, "params": params,
                         "norm": norm, "gate": gate, "pad": pad})


def _lookup(op, name, tokens, cols, vocab, kind, table):
    return _named(name, {"op": op, "tokens": tokens, "cols": cols, "vocab": vocab, "type": kind,
                         "table": table})


def _adamw(name, many8, n8, many32, n32, grad, clip):
    return _named(name, {"op": "adamw", "many8": many8, "n8": n8, "many32": many32, "n32": n32,
                         "grad": grad, "clip": clip})


def work(case):
    op = case["op"]
    if op in ("seam", "seam_grad"):
        r, d, t, p = case["rows"], case["cols"], SIZE[case["type"]], SIZE[case["params"]]
        wide = case["gate"] == "sigmoid"  # a gate for each element
        vectors = 4 + (case["gate"] == "column")
        stats = 4 * r * (4 if case["norm"] == "layer" else 2)
        if op == "seam":  # x, block (, gate) in, sum and y out
            return {"bytes": r * d * t * (4 + wide) + vectors * d * p + stats,
                    "flops": 16 * r * d}
        # dy, dsum, sum, block (, gate) in, dx and dblock (, dgate) out
        return {"bytes": r * d * t * (6 + 2 * wide) + 2 * vectors * d * p + stats,
                "flops": 36 * r * d}
    if op == "lookup":
        n, d, v = case["tokens"], case["cols"], case["vocab"]
        return {"bytes": n * d * SIZE[case["type"]] + min(n, v) * d * SIZE[case["table"]] + 8 * n,
                "flops": n * d}
    if op == "lookup_grad":
        n, d, v = case["tokens"], case["cols"], case["vocab"]
        return {"bytes": n * d * SIZE[case["type"]] + v * d * SIZE[case["table"]] + 8 * n,
                "flops": n * d}
    a, b, g = case["many8"] * case["n8"], case["many32"] * case["n32"], SIZE[case["grad"]]
    # gradient and master in, master and its bf16 copy out, both moments in and out; the norm
    # of what is clipped has to be there before the first element is updated
    each = g + 4 + 4 + 2 + (g if case["clip"] else 0)
    return {"bytes": a * (each + 4) + a // BLOCK * 16 + b * (each + 16), "flops": 20 * (a + b)}


# ------------------------------------------------------------------- inputs

def _rows(g, rows, cols, kind, pad, scale=1.0):
    """Rows of a wider buffer when pad > 0 (the row stride is cols + pad)."""
    a = torch.randn(rows, cols + pad, device="cuda", generator=g) * scale
    return a.to(TYPES[kind])[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("seam", "seam_grad"):
        _prepare_seam(case, s, g)
    elif case["op"] in ("lookup", "lookup_grad"):
        n, d, v = case["tokens"], case["cols"], case["vocab"]
        # a few tokens are frequent, most are rare; one in twenty is padding
        u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
        ids = (v * u ** 3).long().clamp_(max=v - 1)
        pads = torch.rand(n, device="cuda", generator=g) < 0.05
        s["ids"] = torch.where(pads, 0, ids)
        if case["op"] == "lookup":
            s["table"] = _rows(g, v, d, case["table"], 0, 0.02)
        else:
            s["dy"] = _rows(g, n, d, case["type"], 0)
        s["scale"] = float(torch.tensor(d ** 0.5))
    else:
        _prepare_adamw(case, s, g, seed)
    if own:
        _plan(case, s)
    return s


def _prepare_seam(case, s, g):
    r, d, kind, pad = case["rows"], case["cols"], case["type"], case["pad"]
    ptype = TYPES[case["params"]]
    for name in ("x", "block"):
        # hidden states: rows of differing size, a few columns that stand out
        size = torch.exp(0.5 * torch.randn(r, 1, device="cuda", generator=g))
        wide = 1.0 + 9.0 * (torch.rand(d, device="cuda", generator=g) < 0.01)
        a = (torch.randn(r, d, device="cuda", generator=g) * wide + 0.3) * size
        s[name] = torch.nn.functional.pad(a, (0, pad)).to(TYPES[kind])[:, :d]
    for name, mid in (("gamma_post", 1.0), ("beta_post", 0.0), ("gamma", 1.0), ("beta", 0.0)):
        s[name] = (mid + 0.1 * torch.randn(d, device="cuda", generator=g)).to(ptype)
    s["residual_scale"] = 0.75
    if case["gate"] == "column":
        s["gate"] = (0.5 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(ptype)
    else:
        s["gate"] = _rows(g, r, d, kind, pad) if case["gate"] == "sigmoid" else None
    if case["op"] == "seam_grad":
        s["dy"], s["dsum"] = _rows(g, r, d, kind, pad), _rows(g, r, d, kind, pad)
        stats = []
        for a in (s["block"].double(), s["x"].double()):  # x stands for the saved sum here
            mean = a.mean(1) if case["norm"] == "layer" else torch.zeros_like(a[:, 0])
            rstd = 1.0 / torch.sqrt(((a - mean[:, None]) ** 2).mean(1) + EPS)
            stats.append((rstd, mean))
        (r0, m0), (r1, m1) = stats
        rows = [r0, r1] + ([m0, m1] if case["norm"] == "layer" else [])
        s["stats"] = torch.stack(rows).float()


def _prepare_adamw(case, s, g, seed):
    s["key"] = seed & WORD
    for bits in (8, 32):
        many, n = case["many%d" % bits], case["n%d" % bits]
        if not many:
            continue
        blocks = (n + BLOCK - 1) // BLOCK
        # every tensor starts on a multiple of BLOCK elements; zeros behind its end
        live = torch.arange(blocks * BLOCK, device="cuda") < n
        # gradients of differing size from block to block, state like that of such gradients
        size = 1e-3 * torch.exp(torch.randn(many, blocks, 1, device="cuda", generator=g))

        def values(scale):
            a = torch.randn(many, blocks, BLOCK, device="cuda", generator=g) * scale
            return torch.where(live.view(blocks, BLOCK), a, 0.0)

        p = {"grad": values(size).to(TYPES[case["grad"]]), "master": values(0.02)}
        p["m"], p["v"] = values(0.3 * size), (values(0.3 * size) + 0.1 * values(size)) ** 2
        # matrices and gains decay differently: a rate for each tensor
        p["decay"] = torch.tensor(DECAY).expand(many) * (torch.arange(many) % 2 == 0)
        if bits == 8:
            for name, a in (("m", p["m"]), ("v", torch.sqrt(p["v"]))):
                top = a.abs().amax(2)
                scale = torch.where(top > 0, top / 256, 0.0)
                code = torch.where(top[..., None] > 0, a / scale[..., None], 0.0).to(F8)
                p[name], p[name + "_scale"] = code, scale
        s[bits] = p


def _plan(case, s):
    """What a program that uses the framework keeps: owner objects with their workspaces, and
    the buffers that the results go into."""
    import sharded_mixed_precision_zero_amd as Z

    op = case["op"]
    if op in ("seam", "seam_grad"):
        t = TYPES[case["type"]]
        r, d = case["rows"], case["cols"]
        s["plan"] = Z.ZeroBlockNorm(rows=r, cols=d, dtype=t, param_dtype=TYPES[case["params"]],
                                    kind=case["norm"], gate=case["gate"], eps=EPS,
                                    residual_scale=s["residual_scale"])
        names = ("sum", "y") if op == "seam" else ("dx", "dblock")
        s.update({name: torch.empty(r, d, device="cuda", dtype=t) for name in names})
        if op == "seam_grad":
            grads = ["gamma_post", "beta_post", "gamma", "beta"]
            if case["gate"] != "none":
                grads.append("gate")
            s["grads"] = {"d" + name: torch.empty(s[name].shape, device="cuda",
                                                  dtype=s[name].dtype) for name in grads}
    elif op in ("lookup", "lookup_grad"):
        n, d, v = case["tokens"], case["cols"], case["vocab"]
        t, tt = TYPES[case["type"]], TYPES[case["table"]]
        s["plan"] = Z.ZeroEmbedding(tokens=n, vocab=v, cols=d, dtype=t, table_dtype=tt,
                                    grad_dtype=tt, scale=s["scale"], padding=0)
        s["out"] = (torch.empty(n, d, device="cuda", dtype=t) if op == "lookup"
                    else torch.empty(v, d, device="cuda", dtype=tt))
    else:
        tensors, grads = [], []
        for bits in (8, 32):
            if bits not in s:
                continue
            p, n = s[bits], case["n%d" % bits]
            p["out"] = {"param": torch.zeros(p["master"].shape, device="cuda",
                                             dtype=torch.bfloat16)}
            for name in ("master", "m", "v", "m_scale", "v_scale"):
                if name in p:
                    p["out"][name] = torch.zeros_like(p[name])
            for i, decay in enumerate(p["decay"].tolist()):
                def of(a):
                    return a[i].reshape(-1)[:n]

                def scales(a):
                    return a[i]

                more = {} if bits == 32 else {
                    "m_scale": scales(p["m_scale"]), "v_scale": scales(p["v_scale"]),
                    "m_scale_out": scales(p["out"]["m_scale"]),
                    "v_scale_out": scales(p["out"]["v_scale"])}
                tensors.append(Z.adamw_tensor(
                    of(p["master"]), of(p["m"]), of(p["v"]), param_out=of(p["out"]["param"]),
                    master_out=of(p["out"]["master"]), m_out=of(p["out"]["m"]),
                    v_out=of(p["out"]["v"]), grad_dtype=TYPES[case["grad"]],
                    weight_decay=decay, **more))
                grads.append(of(p["grad"]))
        s["plan"] = Z.ZeroAdamW(tensors, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS,
                                max_norm=MAX_NORM if case["clip"] else 0.0)
        s["table"] = Z.contrib_table(grads)
        s["sumsq"] = torch.zeros(1, device="cuda", dtype=torch.float64)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _OWN[op](case, state)
    return _PLAIN[op](case, state)


# ------------------------------------------------------------ the framework

def _own_seam(case, s):
    plan = s["plan"]
    plan.forward(s["x"], s["block"], s["sum"], s["y"], gate=s["gate"],
                 gamma_post=s["gamma_post"], beta_post=s["beta_post"], gamma=s["gamma"],
                 beta=s["beta"])
    return {"sum": s["sum"], "y": s["y"], "stats": plan.stats}


def _own_seam_grad(case, s):
    s["plan"].backward(s["dy"], s["x"], s["block"], s["dx"], s["dblock"], dsum=s["dsum"],
                       gate=s["gate"], gamma_post=s["gamma_post"], beta_post=s["beta_post"],
                       gamma=s["gamma"], stats=s["stats"], **s["grads"])
    return {"dx": s["dx"], "dblock": s["dblock"], **s["grads"]}


def _own_lookup(case, s):
    s["plan"].forward(s["ids"], s["table"], s["out"])
    return {"y": s["out"]}


def _own_lookup_grad(case, s):
    s["plan"].backward(s["ids"], s["dy"], s["out"])
    return {"dtable": s["out"]}


def _own_adamw(case, s):
    plan, sumsq = s["plan"], None
    if case["clip"]:
        sumsq = s["sumsq"]
        plan.gnorm(s["table"], sumsq)
    plan.step(s["table"], LR, T, sumsq, key=s["key"])
    return {bits: s[bits]["out"] for bits in (8, 32) if bits in s}


_OWN = {"seam": _own_seam, "seam_grad": _own_seam_grad, "lookup": _own_lookup,
        "lookup_grad": _own_lookup_grad, "adamw": _own_adamw}


# ------------------------------------------------------------ the plain form

def _norm(a, layer):
    """Rows normalised, and their rstd and mean."""
    mean = a.mean(1, keepdim=True) if layer else None
    c = a - mean if layer else a
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * rstd, rstd, mean


def _plain_seam(case, s):
    t, layer = TYPES[case["type"]], case["norm"] == "layer"
    h, r0, m0 = _norm(s["block"].float(), layer)
    n = h * s["gamma_post"].float() + s["beta_post"].float()
    if case["gate"] == "column":
        n = s["gate"].float() * n
    elif case["gate"] == "sigmoid":
        n = n / (1.0 + torch.exp(-s["gate"].float()))
    total = (s["residual_scale"] * s["x"].float() + n).to(t)
    h, r1, m1 = _norm(total.float(), layer)
    y = (h * s["gamma"].float() + s["beta"].float()).to(t)
    stats = [r0, r1, m0, m1] if layer else [r0, r1]
    return {"sum": total, "y": y, "stats": torch.cat(stats, 1).t().contiguous()}


def _norm_grad(g, h, rstd, layer):
    """Through the rows' normalisation h."""
    out = g - h * (g * h).mean(1, keepdim=True)
    if layer:
        out = out - g.mean(1, keepdim=True)
    return rstd * out


def _plain_seam_grad(case, s):
    t, layer = TYPES[case["type"]], case["norm"] == "layer"
    p = TYPES[case["params"]]
    stats = s["stats"][..., None]
    b, total, dy = s["block"].float(), s["x"].float(), s["dy"].float()
    h0 = ((b - stats[2]) if layer else b) * stats[0]
    h1 = ((total - stats[3]) if layer else total) * stats[1]
    d = _norm_grad(dy * s["gamma"].float(), h1, stats[1], layer) + s["dsum"].float()
    n = h0 * s["gamma_post"].float() + s["beta_post"].float()
    out = {"dx": (s["residual_scale"] * d).to(t), "dgamma": (dy * h1).sum(0).to(p),
           "dbeta": dy.sum(0).to(p)}
    dn = d
    if case["gate"] == "column":
        out["dgate"] = (d * n).sum(0).to(p)
        dn = d * s["gate"].float()
    elif case["gate"] == "sigmoid":
        z = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
        out["dgate"] = (d * n * z * (1.0 - z)).to(t)
        dn = d * z
    out["dgamma_post"] = (dn * h0).sum(0).to(p)
    out["dbeta_post"] = dn.sum(0).to(p)
    out["dblock"] = _norm_grad(dn * s["gamma_post"].float(), h0, stats[0], layer).to(t)
    return out


def _plain_lookup(case, s):
    return {"y": (s["table"][s["ids"]].float() * s["scale"]).to(TYPES[case["type"]])}


def _plain_lookup_grad(case, s):
    out = torch.zeros(case["vocab"], case["cols"], device="cuda")
    # token 0 is padding: its row gets no gradient
    live = (s["ids"] != 0).float()[:, None]
    out.index_add_(0, s["ids"], s["dy"].float() * live)
    return {"dtable": (out * s["scale"]).to(TYPES[case["table"]])}


def _mix(x):
    """32 bits, each of which depends on all of x's."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & WORD
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & WORD
    return x ^ (x >> 16)


def _random(shape, key, first):
    """The 32 random bits of every element: of the key, the tensor's number and the element's."""
    many, blocks, _ = shape
    tensor = torch.arange(first, first + many, device="cuda").view(-1, 1, 1)
    element = torch.arange(blocks * BLOCK, device="cuda").view(1, blocks, BLOCK)
    base = _mix((key + 0x9E3779B9 * (tensor + 1)) & WORD)
    return _mix((base + element) & WORD)


def _to_8_bits(a, dither, least):
    """Values of [0, scale * 256] as e4m3 numbers: down, or up as the dither says, in
    proportion to how near each of the two is."""
    top = a.amax(2, keepdim=True)
    inv = torch.where(top >= 2.0 ** -126, 1.0 / top, 0.0)
    q = torch.clamp(a * inv, max=1.0) * 2.0 ** -112
    code = (q.view(torch.int32).long() + dither) >> 20
    code = torch.maximum(code, least & (top >= 2.0 ** -126)).to(torch.uint8)
    return code, torch.where(top >= 2.0 ** -126, top / 256, 0.0)[..., 0]


def _plain_adamw(case, s):
    coef, out, first = 1.0, {}, 0
    if case["clip"]:
        total = sum((s[bits]["grad"].double() ** 2).sum() for bits in (8, 32) if bits in s)
        coef = torch.clamp(MAX_NORM / (torch.sqrt(total) + 1e-6), max=1.0)
    if 8 in s:
        out[8] = _plain_adamw_8(s[8], s["key"], coef)
        first = case["many8"]
    if 32 in s:
        p = s[32]
        g = p["grad"].float() * coef
        m = BETA1 * p["m"] + (1 - BETA1) * g
        v = BETA2 * p["v"] + (1 - BETA2) * (g * g)
        out[32] = {"m": m, "v": v, **_plain_weights(p, m, torch.sqrt(v))}
    return out


def _plain_weights(p, m, root):
    bc1, bc2 = 1 - BETA1 ** T, 1 - BETA2 ** T
    decay = (LR * p["decay"]).to("cuda")[:, None, None]
    w = p["master"]
    w = w - decay * w - (LR / bc1) * m / (root / math.sqrt(bc2) + ADAM_EPS)
    return {"master": w.float(), "param": w.to(torch.bfloat16)}


def _f32(v):
    return float(torch.tensor(v))


def _plain_adamw_8(p, key, coef):
    g = p["grad"].double() * coef
    m = (p["m"].float() * p["m_scale"][..., None]).double()
    r = (p["v"].float() * p["v_scale"][..., None]).double()
    b1, b2 = _f32(BETA1), _f32(BETA2)
    m = b1 * m + (1 - b1) * g
    r = torch.sqrt(b2 * (r * r) + (1 - b2) * (g * g))
    m32, r32 = m.float(), r.float()
    out = _plain_weights(p, m32, r32)
    bits = _random(g.shape, key, 0)
    code, out["m_scale"] = _to_8_bits(m32.abs(), ((bits & 0xFFFF) << 4) + 8, 0)
    out["m"] = torch.where(m32 < 0, code | 0x80, code).view(F8)
    code, out["v_scale"] = _to_8_bits(r32, ((bits >> 16) << 4) + 8, (r32 > 0).long())
    out["v"] = code.view(F8)
    return out


_PLAIN = {"seam": _plain_seam, "seam_grad": _plain_seam_grad, "lookup": _plain_lookup,
          "lookup_grad": _plain_lookup_grad, "adamw": _plain_adamw}


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False  # inputs only
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](case, s)


def _exact_seam(case, s):
    n, layer = case["cols"], case["norm"] == "layer"

    def normed(a, gamma, beta):
        var, mean = torch.var_mean(a, dim=1, correction=0)
        if not layer:
            var = torch.einsum("rd,rd->r", a, a) / n
        rstd = torch.rsqrt(var + EPS)
        c = a - mean[:, None] if layer else a
        y = torch.addcmul(beta.double(), c * rstd[:, None], gamma.double())
        return y, rstd, mean

    y0, r0, m0 = normed(s["block"].double(), s["gamma_post"], s["beta_post"])
    gate = {"none": lambda: 1.0, "column": lambda: s["gate"].double(),
            "sigmoid": lambda: torch.sigmoid(s["gate"].double())}[case["gate"]]()
    total = torch.addcmul(s["residual_scale"] * s["x"].double(),
                          y0, gate * torch.ones_like(y0)).to(TYPES[case["type"]]).double()
    y1, r1, m1 = normed(total, s["gamma"], s["beta"])
    return {"sum": total, "y": y1, "stats": torch.stack([r0, r1, m0, m1] if layer else [r0, r1])}


def _exact_seam_grad(case, s):
    n, layer = case["cols"], case["norm"] == "layer"
    stats = s["stats"].double()

    def back(g, a, rstd, mean):
        """The projection of g off the span of h (and 1), as inner products; h too."""
        h = (a - mean[:, None] if layer else a) * rstd[:, None]
        along = torch.einsum("rd,rd->r", g, h)[:, None] / n
        rest = g.sum(1, keepdim=True) / n if layer else 0.0
        return (g - rest - along * h) * rstd[:, None], h

    m0, m1 = (stats[2], stats[3]) if layer else (None, None)
    dy = s["dy"].double()
    d, h1 = back(dy * s["gamma"].double(), s["x"].double(), stats[1], m1)
    d = d + s["dsum"].double()
    gate = {"none": lambda: torch.ones(n, device="cuda", dtype=torch.float64),
            "column": lambda: s["gate"].double(),
            "sigmoid": lambda: torch.sigmoid(s["gate"].double())}[case["gate"]]()
    dn = d * gate
    db, h0 = back(dn * s["gamma_post"].double(), s["block"].double(), stats[0], m0)
    out = {"dx": s["residual_scale"] * d, "dblock": db,
           "dgamma": torch.einsum("rd,rd->d", dy, h1), "dbeta": dy.sum(0),
           "dgamma_post": torch.einsum("rd,rd->d", dn, h0), "dbeta_post": dn.sum(0)}
    n0 = torch.addcmul(s["beta_post"].double(), h0, s["gamma_post"].double())
    if case["gate"] == "column":
        out["dgate"] = torch.einsum("rd,rd->d", d, n0)
    elif case["gate"] == "sigmoid":
        out["dgate"] = d * n0 * gate * torch.sigmoid(-s["gate"].double())
    return out


def _exact_lookup(case, s):
    return {"y": torch.nn.functional.embedding(s["ids"], s["table"].double()) * s["scale"]}


def _exact_lookup_grad(case, s):
    # token by token of each row: the sums over the runs of equal ids of the sorted tokens
    live = s["ids"] != 0
    ids, order = torch.sort(s["ids"][live], stable=True)
    out = torch.zeros(case["vocab"], case["cols"], device="cuda", dtype=torch.float64)
    lengths = torch.bincount(ids, minlength=case["vocab"])
    ends = torch.cumsum(lengths, 0)
    dy = s["dy"][live]
    for at in range(0, case["cols"], 1024):
        part = dy[:, at:at + 1024].double()[order]
        sums = torch.nn.functional.pad(torch.cumsum(part, 0), (0, 0, 1, 0))
        out[:, at:at + 1024] = s["scale"] * (sums[ends] - sums[ends - lengths])
    return {"dtable": out}


def _exact_adamw(case, s):
    """The weights and the state in 32 bits.  A state in 8 bits is a random choice between
    neighbours: its numbers have no value of their own, their scales do."""
    coef, out = 1.0, {}
    b1, b2, lr = (float(torch.tensor(v)) for v in (BETA1, BETA2, LR))
    if case["clip"]:
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(s[b]["grad"].double()) ** 2)
                             for b in (8, 32) if b in s))
        coef = min(1.0, MAX_NORM / (norm + 1e-6))
    for bits in (8, 32):
        if bits not in s:
            continue
        p = s[bits]
        g = p["grad"].double().mul_(coef)
        m, v = p["m"].double(), p["v"].double()
        if bits == 8:
            m = m * p["m_scale"].double()[..., None]
            v = (v * p["v_scale"].double()[..., None]).square_()
        m = torch.lerp(g, m, b1)
        v = torch.lerp(g.square(), v, b2)
        w = p["master"].double()
        w = w * (1 - lr * p["decay"].double().to("cuda"))[:, None, None] - torch.div(
            m * (lr / (1 - b1 ** T)), torch.sqrt(v / (1 - b2 ** T)) + float(torch.tensor(ADAM_EPS)))
        out[bits] = {"master": w, "param": w, "m": m if bits == 32 else None,
                     "v": v if bits == 32 else None}
        if bits == 8:
            out[8]["m_scale"] = m.abs().amax(2) / 256
            out[8]["v_scale"] = torch.sqrt(v.amax(2)) / 256
    return out


_EXACT = {"seam": _exact_seam, "seam_grad": _exact_seam_grad, "lookup": _exact_lookup,
          "lookup_grad": _exact_lookup_grad, "adamw": _exact_adamw}
