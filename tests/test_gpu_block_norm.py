"""zero_block_norm_forward and zero_block_norm_backward against fp64 forms.

Bounds, with u = 2^-24.  A row sum of positive terms is an fp32 sum of at most
32 terms per thread and a tree of 10 levels, so the row statistics are right to
48 u relative (the mean to 48 u mean|v| absolute), and an elementwise formula of
fewer than 16 operations adds 16 u of the sum of its terms' magnitudes: C = 64
bounds one norm, and twice that the two that follow one another, each weighed
by the magnitudes of all terms that enter.  Sums over R rows add R u.  A result
that is rounded to bf16 adds half an ulp of it.
"""
import numpy as np
import pytest
import torch

from fsdp_sharded_optimizer_gb300 import _binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_ulp(x):
    """Half a unit in the last of bf16's 8 significant bits at |x|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def norm64(v, w, b, layer, eps):
    mu = v.mean(1, keepdims=True) if layer else 0.0
    r = 1 / np.sqrt(((v - mu) ** 2).mean(1, keepdims=True) + eps)
    xh = (v - mu) * r
    # magnitude that the rounding of xh is measured by
    mag = np.abs(xh) + (r * np.abs(v).mean(1, keepdims=True) if layer else 0.0)
    return xh * w + b, xh, r, mag


def back64(d, w, xh, r, mag, layer):
    dw = d * w
    m0 = dw.mean(1, keepdims=True) if layer else 0.0
    out = r * (dw - m0 - xh * (dw * xh).mean(1, keepdims=True))
    a = np.abs(dw)
    bound = r * (a + (a.mean(1, keepdims=True) if layer else 0.0)
                 + mag * (a * mag).mean(1, keepdims=True))
    return out, bound


def place(shape, dtype, offset, values):
    n = int(np.prod(shape))
    buf = torch.full((offset + n + 64,), 7.0, dtype=dtype, device="cuda")
    t = buf[offset:offset + n].view(*shape)
    if values is not None:
        t.copy_(torch.from_numpy(np.asarray(values, dtype=np.float32)))
    return buf, t


class Case:
    def __init__(self, rows, dim, kind="rms", act="bf16", res="bf16", span=None, gate=True,
                 post=True, pre=True, bias=False, weights=True, branch=True, offset=0,
                 param="bf16", mean=0.3):
        rng = np.random.default_rng(rows * 31 + dim)
        self.rows, self.dim, self.kind, self.layer = rows, dim, kind, kind == "layer"
        self.span = span or max(1, rows)
        self.post, self.pre, self.offset = post and branch, pre, offset
        self.act, self.res, self.param = TYPES[act], TYPES[res], TYPES[param]
        self.eps, self.a, self.b = 1e-5, 0.9, 0.5
        R, D = rows, dim

        def tensor(shape, dtype, sigma, mu=0.0):
            return place(shape, dtype, offset, mu + sigma * rng.standard_normal(shape))[1]

        self.x = tensor((R, D), self.res, 2.0, mean)
        self.h = tensor((R, D), self.act, 0.7, mean) if branch else None
        groups = max(1, -(-R // self.span))
        self.gate = tensor((groups, D), torch.bfloat16, 0.3, 0.8) if gate and branch else None
        one = lambda on, mu: tensor((D,), self.param, 0.1, mu) if on else None
        self.pw, self.pb = one(self.post and weights, 1.0), one(self.post and bias, 0.0)
        self.qw, self.qb = one(pre and weights, 1.0), one(pre and bias, 0.0)
        self.dy = tensor((R, D), self.res, 1.0)
        self.du = tensor((R, D), self.act, 1.0) if pre else None

    def common(self):
        return dict(branch=self.h, gate=self.gate, post_weight=self.pw, post_bias=self.pb,
                    pre_weight=self.qw, kind=self.kind, rows_per_gate=self.span,
                    post_norm=self.post, pre_norm=self.pre, eps=self.eps, residual_scale=self.a,
                    branch_scale=self.b)

    def f64(self, t, absent):
        return absent if t is None else t.detach().cpu().double().numpy()

    def gate64(self):
        g = self.f64(self.gate, None)
        return 1.0 if g is None else g[np.arange(self.rows) // self.span]

    def f32(self, x):
        return float(np.float32(x))


def close(got, want, bound, dtype, what):
    tol = bound * U
    if dtype == torch.bfloat16:
        tol = tol + half_ulp(np.abs(want) + tol)
    got = got.detach().cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol * (1 + 1e-6) + 1e-37)
    assert not bad.any(), "%s: %d off, worst %g of the bound" % (
        what, bad.sum(), np.nanmax(np.abs(got - want) / (tol + 1e-300)))


CASES = [
    dict(rows=1, dim=4096), dict(rows=1, dim=1), dict(rows=3, dim=7, kind="layer", bias=True),
    dict(rows=5, dim=768, kind="layer", bias=True), dict(rows=1000, dim=768, act="bf16", res="f32"),
    dict(rows=2500, dim=64), dict(rows=700, dim=33, kind="layer", bias=True),
    dict(rows=3001, dim=100, act="f32", res="f32"), dict(rows=400, dim=1001),
    dict(rows=400, dim=1002, span=1), dict(rows=333, dim=520, span=100),
    dict(rows=333, dim=515, span=100), dict(rows=2048, dim=256, span=7),
    dict(rows=1300, dim=256, span=1), dict(rows=90, dim=4096, span=2, kind="layer", bias=True),
    dict(rows=2500, dim=256), dict(rows=2500, dim=256, kind="layer", bias=True),
    dict(rows=400, dim=4096), dict(rows=61, dim=2048, gate=False), dict(rows=61, dim=2048, post=False),
    dict(rows=61, dim=2048, pre=False), dict(rows=61, dim=264, branch=False),
    dict(rows=40, dim=5000), dict(rows=9, dim=16384, kind="layer", bias=True),
    dict(rows=9, dim=16383), dict(rows=40, dim=256, offset=1), dict(rows=40, dim=131, offset=3),
    dict(rows=40, dim=256, weights=False, param="f32"),
    dict(rows=70, dim=256, param="f32", kind="layer", bias=True, act="f32", res="f32"),
    dict(rows=50, dim=512, kind="layer", mean=50.0, act="f32", res="f32", bias=True),
]
IDS = ["-".join("%s%s" % (k[:4], v) for k, v in c.items()) for c in CASES]


def forward64(c):
    """y, u and their error magnitudes in units of u."""
    a, b = c.f32(c.a), c.f32(c.b)
    x = c.f64(c.x, None)
    if c.h is not None:
        h = c.f64(c.h, None)
        w, cb = c.f64(c.pw, 1.0), c.f64(c.pb, 0.0)
        if c.post:
            n, _, _, mag = norm64(h, w, cb, c.layer, c.f32(c.eps))
            nb = np.abs(w) * mag + np.abs(cb)
        else:
            n, nb = h, np.abs(h)
        y = a * x + b * c.gate64() * n
        yb = 64 * (np.abs(a * x) + np.abs(b * c.gate64()) * nb)
    else:
        y, yb = x, np.zeros_like(x)
    if not c.pre:
        return y, yb, None, None
    w, cb = c.f64(c.qw, 1.0), c.f64(c.qb, 0.0)
    u, xh, r, mag = norm64(y, w, cb, c.layer, c.f32(c.eps))
    moved = r * (yb + yb.mean(1, keepdims=True)
                 + np.abs(xh) * (np.abs(xh) * yb).mean(1, keepdims=True))
    return y, yb, u, np.abs(w) * (64 * mag + moved) + 64 * np.abs(cb)


@pytest.mark.parametrize("spec", CASES, ids=IDS)
def test_forward(spec):
    c = Case(**spec)
    shape = (c.rows, c.dim)
    ybuf, y = place(shape, c.res, c.offset, None) if c.h is not None else (None, None)
    ubuf, u = place(shape, c.act, c.offset, None) if c.pre else (None, None)
    B.zero_block_norm_forward(c.x, pre_bias=c.qb, y=y, u=u, **c.common())
    wy, by, wu, bu = forward64(c)
    for t, want, bound, dtype, buf, name in ((y, wy, by, c.res, ybuf, "y"),
                                             (u, wu, bu, c.act, ubuf, "u")):
        if t is not None:
            close(t, want, bound, dtype, name)
            n = c.rows * c.dim
            assert bool((buf[:c.offset] == 7).all()) and bool((buf[c.offset + n:] == 7).all())
    if y is not None:  # in place
        x = c.x.clone()
        keep = c.x
        c.x = x
        u2 = torch.empty_like(u) if u is not None else None
        B.zero_block_norm_forward(x, pre_bias=c.qb, y=x, u=u2, **c.common())
        if c.offset == 0:
            assert torch.equal(x, y) and (u is None or torch.equal(u, u2))
        c.x = keep


def backward64(c):
    """name -> (gradient, error magnitude in units of u)."""
    a, b, eps = c.f32(c.a), c.f32(c.b), c.f32(c.eps)
    out = {}
    g = c.f64(c.dy, None)
    gb = 4 * np.abs(g)
    if c.pre:
        y, du = c.f64(c.x, None), c.f64(c.du, None)
        w = c.f64(c.qw, 1.0)
        _, xh, r, mag = norm64(y, w, 0.0, c.layer, eps)
        p, pb = back64(du, w, xh, r, mag, c.layer)
        g, gb = g + p, gb + 64 * pb
        out["dpre_weight"] = ((du * xh).sum(0), ((64 + c.rows) * np.abs(du) * mag).sum(0))
        out["dpre_bias"] = (du.sum(0), ((4 + c.rows) * np.abs(du)).sum(0))
    out["dx"] = (a * g, abs(a) * gb + 4 * np.abs(a * g))
    if c.h is None:
        return out
    h, gate = c.f64(c.h, None), c.gate64()
    d, db = b * gate * g, np.abs(b * gate) * (gb + 4 * np.abs(g))
    if c.post:
        w, cb = c.f64(c.pw, 1.0), c.f64(c.pb, 0.0)
        n, xh, r, mag = norm64(h, w, cb, c.layer, eps)
        v, vb = back64(d, w, xh, r, mag, c.layer)
        _, moved = back64(db, np.abs(w), xh, r, mag, c.layer)
        out["dbranch"] = (v, 64 * vb + moved)
        out["dpost_weight"] = ((d * xh).sum(0),
                               (np.abs(d) * mag * (64 + c.rows) + db * np.abs(xh)).sum(0))
        out["dpost_bias"] = (d.sum(0), (np.abs(d) * (4 + c.rows) + db).sum(0))
        nb = np.abs(w) * mag + np.abs(cb)
    else:
        n, nb = h, np.abs(h)
        out["dbranch"] = (d, db + 4 * np.abs(d))
    if c.gate is not None:
        groups = c.gate.shape[0]
        which = np.arange(c.rows) // c.span
        total, bound = np.zeros((groups, c.dim)), np.zeros((groups, c.dim))
        np.add.at(total, which, b * g * n)
        np.add.at(bound, which, abs(b) * (np.abs(g) * nb * (64 + c.span) + gb * np.abs(n)))
        out["dgate"] = (total, bound)
    return out


def run_backward(c, grad_type, names):
    shape = (c.rows, c.dim)
    bufs = {"dx": place(shape, c.res, c.offset, None)}
    if c.h is not None:
        bufs["dbranch"] = place(shape, c.act, c.offset, None)
        if c.gate is not None:
            bufs["dgate"] = place(tuple(c.gate.shape), grad_type, c.offset, None)
    for n in ("dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"):
        if n in names:
            bufs[n] = place((c.dim,), grad_type, c.offset, None)
    scratch = torch.full((B.zero_block_norm_scratch_bytes(c.rows, c.dim, c.span),), 255,
                         dtype=torch.uint8, device="cuda")
    B.zero_block_norm_backward(c.x, scratch, dy=c.dy, du=c.du, **c.common(),
                               **{k: t for k, (_, t) in bufs.items()})
    return bufs


@pytest.mark.parametrize("grad_type", ["bf16", "f32"])
@pytest.mark.parametrize("spec", CASES, ids=IDS)
def test_backward(spec, grad_type):
    c = Case(**spec)
    want = backward64(c)
    bufs = run_backward(c, TYPES[grad_type], want)
    again = run_backward(c, TYPES[grad_type], want)
    for name, (buf, t) in bufs.items():
        g, bound = want[name]
        close(t, g, bound, t.dtype, name)
        n = t.numel()
        assert bool((buf[:c.offset] == 7).all()) and bool((buf[c.offset + n:] == 7).all()), name
        assert torch.equal(t, again[name][1]), name  # the same bits again


def test_gradient_agrees_with_differences():
    """Directional differences of the fp64 form at the kernel's inputs: the step
    2^-12 leaves a truncation of about 2^-24 of third derivatives of order one,
    so 1e-5 of the gradient's magnitude along the direction covers both."""
    for kind in ("rms", "layer"):
        c = Case(6, 40, kind=kind, act="f32", res="f32", param="f32", bias=True, span=2)
        rng = np.random.default_rng(3)
        dy, du = c.f64(c.dy, None), c.f64(c.du, None)
        names = {"dx": "x", "dbranch": "h", "dgate": "gate", "dpost_weight": "pw",
                 "dpost_bias": "pb", "dpre_weight": "qw", "dpre_bias": "qb"}
        y = torch.empty(c.rows, c.dim, device="cuda")
        u = torch.empty_like(y)
        B.zero_block_norm_forward(c.x, pre_bias=c.qb, y=y, u=u, **c.common())

        def loss(values):
            a, b, eps = c.f32(c.a), c.f32(c.b), c.f32(c.eps)
            n = norm64(values["h"], values["pw"], values["pb"], c.layer, eps)[0]
            yy = a * values["x"] + b * values["gate"][np.arange(c.rows) // c.span] * n
            uu = norm64(yy, values["qw"], values["qb"], c.layer, eps)[0]
            return (yy * dy).sum() + (uu * du).sum()

        base = {v: c.f64(getattr(c, v), None) for v in names.values()}
        stream, c.x = c.x, y
        got = run_backward(c, torch.float32, names)
        c.x = stream
        for g, v in names.items():
            step = rng.standard_normal(base[v].shape)
            e = 2.0 ** -12
            up, down = dict(base), dict(base)
            up[v], down[v] = base[v] + e * step, base[v] - e * step
            numeric = (loss(up) - loss(down)) / (2 * e)
            gv = got[g][1].cpu().double().numpy()
            mine = (gv * step).sum()
            assert abs(mine - numeric) <= 1e-5 * np.abs(gv * step).sum() + 1e-6, (kind, g)


def test_no_rows():
    """No rows: nothing to normalise, and every sum over rows is +0."""
    D = 64
    x = torch.empty(0, D, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    B.zero_block_norm_forward(x, branch=x, pre_weight=w, post_weight=w, y=x, u=x)
    dw = torch.full((D,), 7.0, device="cuda")
    dg = torch.full((1, D), 7.0, device="cuda")
    scratch = torch.empty(B.zero_block_norm_scratch_bytes(0, D), dtype=torch.uint8, device="cuda")
    B.zero_block_norm_backward(x, scratch, dy=x, du=x, branch=x, gate=w.view(1, D), pre_weight=w,
                               post_weight=w, dx=x, dbranch=x, dpre_weight=dw, dgate=dg)
    assert not dw.any() and not dg.any()


def test_rows_stay_apart():
    """A row of NaN or infinities spoils its own outputs only, and a row of
    zeros has the norm 0 and a finite gradient."""
    c = Case(12, 264)
    c.h[3].fill_(float("nan"))
    c.x[5].fill_(float("inf"))
    c.x[7].zero_()
    c.h[7].zero_()
    y, u = torch.empty_like(c.x), torch.empty_like(c.h)
    B.zero_block_norm_forward(c.x, y=y, u=u, **c.common())
    fine = [i for i in range(12) if i not in (3, 5)]
    assert torch.isfinite(u[fine].float()).all() and torch.isnan(u[3].float()).all()
    assert not y[7].any() and not u[7].any()
    bufs = run_backward(c, torch.float32, ())
    for n in ("dx", "dbranch"):
        assert torch.isfinite(bufs[n][1][fine].float()).all()
