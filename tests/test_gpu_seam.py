"""The seam between two blocks, forward and backward, on the GPU against the
formulas in 64 bits: every type, norm, gate and register shape, odd widths,
padded and unaligned rows, absent parameters and blocks, infinities and NaN,
buffers used in place, another stream, a captured graph, differences."""

from __future__ import annotations

import itertools

import pytest
import torch

import sharded_mixed_precision_zero_amd as Z
from tests import _operators as R
from tests import _seam as S

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# (rows, cols): every register shape and its edges, one row, one column, odd
# widths, more rows than workgroups
SIZES = [(1, 1), (3, 2), (5, 8), (1, 5120), (7, 511), (6, 512), (9, 1601), (3, 2056), (5, 5120),
         (3, 8192), (2, 8200), (2, 16383), (3, 16384), (2100, 64), (1030, 2064), (600, 4099),
         (4, 7), (3, 9), (1100, 15), (1030, 515), (40, 1030), (1500, 2562)]
TYPES = [(F32, F32), (BF, BF), (BF, F32), (F16, F16), (F16, F32)]
WAYS = list(itertools.product(("rms", "layer"), ("none", "column", "sigmoid")))
EPS, SCALE = 1e-5, 0.7


def _rows(rows, cols, dtype, pad, seed, spread=True):
    a = R.randn(rows, cols, pad=pad, seed=seed)
    if spread:
        a = a * (1.0 + torch.arange(rows, device="cuda", dtype=F32)[:, None] % 7) + 0.5
    full = torch.empty(rows, cols + pad, device="cuda", dtype=dtype)
    full[:, :cols] = a.to(dtype)
    return full[:, :cols]


def _inputs(rows, cols, dtype, ptype, gate, pad, affine=True):
    p = {"x": _rows(rows, cols, dtype, pad, 1), "block": _rows(rows, cols, dtype, pad, 2)}
    for i, (name, mid) in enumerate((("gamma_post", 1.0), ("beta_post", 0.0), ("gamma", 1.0),
                                     ("beta", 0.0))):
        p[name] = (mid + R.randn(cols, seed=10 + i, scale=0.2)).to(ptype) if affine else None
    p["gate"] = {"none": lambda: None,
                 "column": lambda: (0.5 + R.randn(cols, seed=20, scale=0.2)).to(ptype),
                 "sigmoid": lambda: _rows(rows, cols, dtype, pad, 21, spread=False)}[gate]()
    return p


def _serial(rows):
    """A thread's rows, the row groups of a workgroup, a group's partials, the groups."""
    return rows // 256 + 2 + 16 + 4 + 64


def _within(name, got, ref, tol):
    R.within(name, got, ref, tol + R.half_step(got.dtype, ref.abs() + tol))


def _check_forward(plan, p, kind, gate, post, total, y, scale=SCALE):
    if post:
        (n, dn), (r, dr), (m, dm) = S.norm_ref(p["block"], kind, p["gamma_post"], p["beta_post"],
                                               EPS)
        R.within("rstd 0", plan.stats[0], r, dr + 2 * R.U * r)
        if kind == "layer":
            R.within("mean 0", plan.stats[2], m, dm + R.U * abs(m))
    else:
        n, dn = p["block"].double(), 0.0
    s, ds = S.sum_ref(p["x"], n, dn, S.gate_ref(p["gate"], gate), scale)
    _within("sum", total, s, ds)
    _check_second(plan, p, kind, total, y)


def _check_second(plan, p, kind, total, y):
    (v, dv), (r, dr), (m, dm) = S.norm_ref(total, kind, p["gamma"], p["beta"], EPS)
    _within("y", y, v, dv)
    R.within("rstd 1", plan.stats[1], r, dr + 2 * R.U * r)
    if kind == "layer":
        R.within("mean 1", plan.stats[3], m, dm + R.U * abs(m))


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype, ptype):
    for i, (kind, gate) in enumerate(WAYS):
        pad, affine, post = (0, 8, 3)[i % 3], i % 4 != 1, i != 4
        p = _inputs(rows, cols, dtype, ptype, gate, pad, affine)
        if not post:
            p["gamma_post"] = p["beta_post"] = None
        plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, kind=kind,
                               gate=gate, post=post, eps=EPS, residual_scale=SCALE)
        total, y = _rows(rows, cols, dtype, pad, 5), _rows(rows, cols, dtype, 0, 6)
        plan.forward(p["x"], p["block"], total, y,
                     **{k: v for k, v in p.items() if k not in ("x", "block")})
        _check_forward(plan, p, kind, gate, post, total, y, float(torch.tensor(SCALE)))


def _backward(rows, cols, dtype, ptype, kind, gate, pad, affine, post, dsum=True, which=None):
    p = _inputs(rows, cols, dtype, ptype, gate, pad, affine)
    if not post:
        p["gamma_post"] = p["beta_post"] = None
    total, block = p["x"], p["block"]
    stats = []
    for a in (block.double(), total.double()):
        m = a.mean(1) if kind == "layer" else torch.zeros(rows, device="cuda", dtype=torch.float64)
        stats.append((1.0 / torch.sqrt(((a - m[:, None]) ** 2).mean(1) + EPS), m))
    stats = [s[0] for s in stats] + ([s[1] for s in stats] if kind == "layer" else [])
    stats = torch.stack(stats).float()
    dy = _rows(rows, cols, dtype, pad, 30)
    ds = _rows(rows, cols, dtype, pad, 31) if dsum else None
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, kind=kind,
                           gate=gate, post=post, eps=EPS, residual_scale=SCALE)
    grads = {"dgamma": torch.full((cols,), 7.0, device="cuda", dtype=ptype)}
    grads["dbeta"] = grads["dgamma"].clone()
    if post:
        grads["dgamma_post"], grads["dbeta_post"] = grads["dbeta"].clone(), grads["dbeta"].clone()
    if gate == "column":
        grads["dgate"] = grads["dbeta"].clone()
    elif gate == "sigmoid":
        grads["dgate"] = _rows(rows, cols, dtype, pad, 40)
    if which is not None:
        grads = {k: v for k, v in grads.items() if k in which}
    dx, dblock = _rows(rows, cols, dtype, pad, 41), _rows(rows, cols, dtype, 0, 42)
    plan.backward(dy, total, block, dx, dblock, dsum=ds, gate=p["gate"],
                  gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"],
                  stats=stats, **grads)
    ref = S.backward_ref(dy, ds, total, block, p["gate"], kind, gate, post,
                         float(torch.tensor(SCALE)), p["gamma_post"], p["beta_post"], p["gamma"],
                         stats, _serial(rows))
    for name, got in {"dx": dx, "dblock": dblock, **grads}.items():
        _within(f"{kind} {gate} {name}", got, *ref[name])


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, dtype, ptype):
    for i, (kind, gate) in enumerate(WAYS):
        _backward(rows, cols, dtype, ptype, kind, gate, (0, 8, 3)[i % 3], i % 4 != 1, i != 4,
                  dsum=i % 5 != 3)


@pytest.mark.parametrize("which", [(), ("dgamma",), ("dbeta_post",), ("dgate",),
                                   ("dgate", "dbeta")])
@pytest.mark.parametrize("gate", ["column", "sigmoid"])
def test_gradients_that_are_not_asked_for(which, gate):
    for rows in (5, 700):
        _backward(rows, 1000, BF, F32, "layer", gate, 0, True, True, which=which)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,ptype", TYPES)
def test_without_a_block_it_is_one_norm(kind, dtype, ptype):
    for rows, cols, pad in ((4, 5120, 0), (300, 777, 3), (2, 9000, 8)):
        x = _rows(rows, cols, dtype, pad, 1)
        p = _inputs(rows, cols, dtype, ptype, "none", pad)
        plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=dtype, param_dtype=ptype, kind=kind,
                               post=False, eps=EPS)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        plan.forward(x, None, None, y, gamma=p["gamma"], beta=p["beta"])
        _check_second(plan, p, kind, x, y)
        assert (plan.stats[0] == 0).all()  # of a norm that is not there
        dy = _rows(rows, cols, dtype, pad, 30)
        grads = {n: torch.empty(cols, device="cuda", dtype=ptype) for n in ("dgamma", "dbeta")}
        plan.backward(dy, x, None, dx, None, gamma=p["gamma"], **grads)
        ref = S.backward_ref(dy, None, x, None, None, kind, "none", False, 1.0, None, None,
                             p["gamma"], plan.stats, _serial(rows))
        for name, got in {"dx": dx, **grads}.items():
            _within(name, got, *ref[name])


@pytest.mark.parametrize("kind,gate", WAYS)
@pytest.mark.parametrize("cols", [96, 1601, 9000])
def test_backward_is_the_forward_differentiated(kind, gate, cols):
    """Every gradient against central differences of the formula in 64 bits
    along random directions."""
    rows, eps, scale = 6, 1e-5, 0.5
    p = _inputs(rows, cols, F32, F32, gate, 0)
    dy, dsum = R.randn(rows, cols, seed=30), R.randn(rows, cols, seed=31)
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=F32, kind=kind, gate=gate, eps=eps,
                           residual_scale=scale)
    total, y = torch.empty_like(p["x"]), torch.empty_like(p["x"])
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan.forward(p["x"], p["block"], total, y, **args)
    names = ["gamma_post", "beta_post", "gamma", "beta"] + (["gate"] if gate != "none" else [])
    grads = {"d" + n: torch.empty_like(p[n]) for n in names}
    dx, db = torch.empty_like(y), torch.empty_like(y)
    plan.backward(dy, total, p["block"], dx, db, dsum=dsum, gate=p["gate"],
                  gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"], **grads)

    def norm(a):
        c = a - a.mean(1, keepdim=True) if kind == "layer" else a
        return c / torch.sqrt((c * c).mean(1, keepdim=True) + eps)

    def loss(q):
        n = norm(q["block"]) * q["gamma_post"] + q["beta_post"]
        s = scale * q["x"] + S.gate_ref(q["gate"], gate) * n
        return float(((norm(s) * q["gamma"] + q["beta"]) * dy.double()).sum()
                     + (s * dsum.double()).sum())

    at = {k: None if v is None else v.double() for k, v in p.items()}
    for name, grad in {"x": dx, "block": db, **{n: grads["d" + n] for n in names}}.items():
        for seed in range(3):
            v = R.randn(*at[name].shape, seed=50 + seed).double()
            step = 1e-4
            want = (loss({**at, name: at[name] + step * v})
                    - loss({**at, name: at[name] - step * v})) / (2 * step)
            got = float((grad.double() * v).sum())
            size = float(torch.linalg.norm(grad.double()) * torch.linalg.norm(v)) + 1e-3
            # the difference's own error: step^2 of the third derivative, and
            # 2^-52 of the loss over the step
            assert abs(got - want) <= 2e-5 * size, (name, got, want, size)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["column", "sigmoid"])
@pytest.mark.parametrize("cols", [1000, 515, 1029])
def test_buffers_used_in_place(kind, gate, cols):
    """sum over x or block, y over the other; dx and dblock over what they are
    the gradients from, dz over z: the same bits as into new buffers."""
    rows = 777
    p = _inputs(rows, cols, BF, F32, gate, 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, kind=kind, gate=gate,
                           residual_scale=SCALE)
    total, y = torch.empty_like(p["x"]), torch.empty_like(p["x"])
    plan.forward(p["x"], p["block"], total, y, **args)
    for swap in (False, True):
        x, b = p["x"].clone(), p["block"].clone()
        s2, y2 = (b, x) if swap else (x, b)
        plan.forward(x, b, s2, y2, **args)
        assert torch.equal(s2, total) and torch.equal(y2, y)
    dy, ds = _rows(rows, cols, BF, 0, 30), _rows(rows, cols, BF, 0, 31)
    new = lambda: torch.empty_like(dy)
    pars = dict(gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"])
    wide = gate == "sigmoid"
    dx, db, dz = new(), new(), new() if wide else None
    plan.backward(dy, total, p["block"], dx, db, dsum=ds, gate=p["gate"], dgate=dz, **pars)
    for use in (("dy", "block"), ("dsum", "sum"), ("sum", "dy"), ("block", "dsum")):
        t = {"dy": dy.clone(), "dsum": ds.clone(), "sum": total.clone(),
             "block": p["block"].clone()}
        z = p["gate"].clone() if wide else p["gate"]
        plan.backward(t["dy"], t["sum"], t["block"], t[use[0]], t[use[1]], dsum=t["dsum"], gate=z,
                      dgate=z if wide else None, **pars)
        assert torch.equal(t[use[0]], dx) and torch.equal(t[use[1]], db), use
        assert not wide or torch.equal(z, dz)


def test_rows_behind_the_last_are_left_alone():
    rows, cols = 5, 1601
    p = _inputs(rows, cols, BF, BF, "sigmoid", 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, gate="sigmoid")
    bufs = [torch.full((rows + 2, cols + 5), 3.0, device="cuda", dtype=BF) for _ in range(5)]
    total, y, dx, db, dz = (b[1:rows + 1, :cols] for b in bufs)
    plan.forward(p["x"], p["block"], total, y, **args)
    plan.backward(p["x"], total, p["block"], dx, db, gate=p["gate"], dgate=dz,
                  gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"])
    for b in bufs:
        assert (b[0] == 3.0).all() and (b[rows + 1:] == 3.0).all() and (b[:, cols:] == 3.0).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [512, 515, 9000])
def test_infinities_and_nan_stay_in_their_rows(kind, cols):
    rows = 40
    p = _inputs(rows, cols, BF, F32, "column", 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, kind=kind,
                           gate="column")
    clean = [torch.empty_like(p["x"]) for _ in range(2)]
    plan.forward(p["x"], p["block"], *clean, **args)
    x, b = p["x"].clone(), p["block"].clone()
    x[3, 7], b[11, cols - 1], b[20, 0] = float("inf"), float("nan"), float("-inf")
    total, y = torch.empty_like(x), torch.empty_like(x)
    plan.forward(x, b, total, y, **args)
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    ok[[3, 11, 20]] = False
    assert torch.equal(y[ok], clean[1][ok]) and torch.equal(total[ok], clean[0][ok])
    # an RMS norm of a row with an infinity is 0 but for that element's own NaN
    bad = torch.isnan(y)
    assert bad[3, 7] and bad[11].all() and bad[20, 0]
    if kind == "layer":
        assert bad[3].all() and bad[20].all()


def test_extreme_gates():
    """The sigmoid's ends: 0 and 1 with no NaN, the slope 0."""
    rows, cols = 4, 64
    p = _inputs(rows, cols, F32, F32, "sigmoid", 0)
    inf = float("inf")
    p["gate"][:] = torch.tensor([-inf, -200.0, 200.0, inf], device="cuda")[:, None]
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=F32, gate="sigmoid", eps=EPS)
    total, y, dx, db, dz = (torch.empty_like(p["x"]) for _ in range(5))
    plan.forward(p["x"], p["block"], total, y, **args)
    assert torch.equal(total[:2], p["x"][:2])
    n, dn = S.norm_ref(p["block"], "rms", p["gamma_post"], p["beta_post"], EPS)[0]
    _within("sum", total[2:], (p["x"].double() + n)[2:],
            (dn + 4 * R.U * (abs(n) + abs(p["x"].double())))[2:])
    plan.backward(y, total, p["block"], dx, db, gate=p["gate"], dgate=dz,
                  gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"])
    assert (db[:2] == 0).all() and torch.isfinite(db).all() and (dz == 0).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_zero_rows_give_beta(kind):
    rows, cols = 3, 1601
    p = _inputs(rows, cols, F32, F32, "none", 0)
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=F32, kind=kind, eps=EPS)
    z, total, y = (torch.zeros(rows, cols, device="cuda") for _ in range(3))
    plan.forward(z, z.clone(), total, y, gamma_post=p["gamma_post"], gamma=p["gamma"],
                 beta=p["beta"])
    assert (total == 0).all() and torch.equal(y, p["beta"].expand(rows, cols))


def test_no_rows():
    plan = Z.ZeroBlockNorm(rows=0, cols=300, dtype=BF, gate="column")
    e = torch.empty(0, 300, device="cuda", dtype=BF)
    p = torch.ones(300, device="cuda", dtype=BF)
    plan.forward(e, e, e.clone(), e.clone(), gate=p, gamma=p)
    grads = {n: torch.full((300,), 5.0, device="cuda", dtype=BF)
             for n in ("dgate", "dgamma", "dbeta", "dgamma_post", "dbeta_post")}
    plan.backward(e, e, e, e, e, gate=p, gamma=p, **grads)
    for n, g in grads.items():
        assert (g == 0).all(), n


def test_the_same_bits_every_time_and_on_another_stream():
    rows, cols = 1500, 2048
    p = _inputs(rows, cols, BF, F32, "column", 0)
    dy = _rows(rows, cols, BF, 0, 30)

    def once(stream):
        with torch.cuda.stream(stream):
            plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, kind="layer",
                                   gate="column", residual_scale=SCALE)
            out = [torch.empty_like(p["x"]) for _ in range(4)]
            grads = {n: torch.empty(cols, device="cuda")
                     for n in ("dgate", "dgamma", "dbeta", "dgamma_post", "dbeta_post")}
            args = {k: v for k, v in p.items() if k not in ("x", "block")}
            plan.forward(p["x"], p["block"], out[0], out[1], **args)
            plan.backward(dy, out[0], p["block"], out[2], out[3], gate=p["gate"],
                          gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"],
                          **grads)
        stream.synchronize()
        return out + list(grads.values())

    torch.cuda.synchronize()
    want = once(torch.cuda.current_stream())
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        assert all(torch.equal(a, b) for a, b in zip(once(stream), want))


def test_in_a_captured_graph():
    rows, cols = 64, 1601
    p = _inputs(rows, cols, BF, F32, "column", 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, gate="column")
        eager = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, param_dtype=F32, gate="column")
        outs = [torch.empty_like(p["x"]) for _ in range(4)]
        grads = {n: torch.empty(cols, device="cuda")
                 for n in ("dgate", "dgamma", "dbeta", "dgamma_post", "dbeta_post")}

    def call(pl, out, grads):
        pl.forward(p["x"], p["block"], out[0], out[1], **args)
        pl.backward(out[1], out[0], p["block"], out[2], out[3], gate=p["gate"],
                    gamma_post=p["gamma_post"], beta_post=p["beta_post"], gamma=p["gamma"],
                    **grads)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(plan, outs, grads)
    for k in range(3):
        with torch.cuda.stream(side):
            p["x"].copy_(_rows(rows, cols, BF, 0, 60 + k))
            graph.replay()
            want = [torch.empty_like(o) for o in outs]
            wg = {n: torch.empty_like(g) for n, g in grads.items()}
            call(eager, want, wg)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(grads[n], wg[n]) for n in grads)


def test_rows_past_32_bit_offsets():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements."""
    rows, cols, ld = 3, 512, (1 << 30) + 8
    buf = torch.empty(2 * ld + cols, device="cuda", dtype=BF)
    x = buf.as_strided((rows, cols), (ld, 1))
    x.copy_(_rows(rows, cols, BF, 0, 1))
    p = _inputs(rows, cols, BF, BF, "column", 0)
    args = {k: v for k, v in p.items() if k not in ("x", "block")}
    plan = Z.ZeroBlockNorm(rows=rows, cols=cols, dtype=BF, gate="column")
    total, y = torch.empty_like(p["x"]), torch.empty_like(p["x"])
    plan.forward(p["x"], p["block"], total, y, **args)
    plan.forward(x, p["block"], x, p["x"], **args)
    assert torch.equal(x, total) and torch.equal(p["x"], y)
