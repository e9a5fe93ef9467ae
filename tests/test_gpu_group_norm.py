"""zero_group_norm_forward and zero_group_norm_backward against fp64 forms.

Bounds, with u = 2^-24, D the largest |x - mean| of a group and m its |mean|.

Mean: a value passes a difference, at most 64 sums of a thread, 64 + 5 of a block's
join and (runs / 32 + 6) of the runs' join, a product and three sums more: less
than 160 + runs / 32 roundings, each of a value of at most m + 2 D:
em = (160 + runs / 32) u (m + 2 D); runs are less than 8192 in every case here, so
em = 416 u (m + 2 D).

Variance: a thread's squares are about its own first value, which lies within 5 standard
deviations of the mean here, so they add to at most 26 times those about the mean.  Their
sum passes up to 64 roundings of partial sums, of either sign: three standard deviations
are 3 * sqrt(64 / 3) * 26 u = 360 u; the joins' 143 roundings and the terms' own 3 add
150 u: 600 u covers it, and em^2, as the squares are about the rounded mean.  So
1/sqrt(var + eps) is right to er = 300 u + em^2 * rstd^2 / 2 + 4 u relative.

z = (x - mean) * (rstd * w) + b: ez = em rstd |w| + |z - b| (er + 4 u) + 2 u (|z| + |b|).
Activations have slopes below 1.13; silu's exponential is right to (2 + 1.2 |z|) ulp and
its quotient to 2 ulp: ey = 1.13 ez + (14 + 3 |z|) u (|y| + |z| 2^-10).  gelu's probability is
a polynomial of absolute error 7.5e-8 = 1.3 u (Abramowitz and Stegun 26.2.17) with
coefficients that add to 5.7, times a density of at most 0.4: 16 roundings of that and the
method's error are 16 * 5.7 * 0.4 u + 1.3 u < 40 u, so 40 u |z| more for y.

The gradient takes its statistics as they are given: h has 3 roundings; the slope's error
is es = (24 + 6 |z|) u + 0.8 * (2 u (|h w| + |b|) + 3 u |h w|), and (41 + 41 |z|) u more with
gelu.  A sum over rows passes at
most K = 64 (a thread) + 256 (row groups) + runs + samples / 8 + 16 roundings, each
of at most the sum of magnitudes.
"""
import math

import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_ulp(x):
    """Half a unit in the last of bf16's 8 significant bits at |x|."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126))) - 8)


def act64(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def place(shape, dtype, pad, offset, values, fill=7.0):
    """[N, P, C] with rows pad elements further apart, offset elements into a buffer."""
    N, P, C = shape
    buf = torch.full((offset + N * P * (C + pad) + 16,), fill, dtype=dtype, device="cuda")
    t = buf[offset:offset + N * P * (C + pad)].view(N, P, C + pad)[..., :C]
    if values is not None:
        t.copy_(values)
    return buf, t


def close(got, want, tol, what):
    if got.dtype == torch.bfloat16:
        tol = tol + half_ulp(want.abs() + tol)
    off = (got.double() - want).abs()
    bad = ~(off <= tol + 1e-37)
    assert not bad.any(), "%s: %d off, worst %g of the bound" % (
        what, int(bad.sum()), float((off / (tol + 1e-300)).nan_to_num(nan=math.inf).max()))


class Case:
    def __init__(self, N=2, P=64, C=64, G=8, type="bf16", param="bf16", act="silu", weight=True,
                 bias=True, ragged=False, mean=0.5, pad=0, offset=0, eps=1e-5):
        self.__dict__.update(N=N, P=P, C=C, G=G, type=TYPES[type], param=TYPES[param], act=act,
                             pad=pad, offset=offset, eps=eps)
        gen = torch.Generator(device="cuda").manual_seed(N * 31 + P * 7 + C)
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
        x = randn(N, P, C) * (0.5 + torch.rand(C, generator=gen, device="cuda")) + mean
        self.xbuf, self.x = place((N, P, C), self.type, pad, offset, x)
        _, self.dy = place((N, P, C), self.type, pad, offset, randn(N, P, C))
        vec = lambda on, mu: ((mu + 0.3 * randn(C + 1)).to(self.param)[1:] if on else None)
        self.w, self.b = vec(weight, 1.0), vec(bias, 0.0)
        self.lengths, self.len = None, [P] * N
        if ragged:
            want = [(P, 0, max(1, P // 3), P + 4, -2, 1)[n % 6] for n in range(N)]
            self.lengths = torch.tensor(want, dtype=torch.int32, device="cuda")
            self.len = [min(P, max(0, n)) for n in want]
            for n in range(N):  # what does not count may hold anything
                self.x[n, self.len[n]:] = math.nan
                self.dy[n, self.len[n]:] = math.nan
        need = Z.zero_group_norm_scratch_bytes(N, P, C, G)
        self.scratch = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        self.need = need
        self.per = C // G

    def scr(self):
        return self.scratch[:self.need]

    def wide(self, t, absent):
        if t is None:
            return torch.full((self.C,), absent, dtype=torch.float64, device="cuda")
        return t.double()

    def spread(self, v):
        return v.repeat_interleave(self.per)


CASES = [
    dict(N=1, P=64, C=1280, G=32), dict(N=1, P=1, C=8, G=1), dict(N=3, P=1, C=2, G=2),
    dict(N=2, P=1, C=4096, G=32, act="none"), dict(N=500, P=1, C=256, G=4, act="gelu"),
    dict(N=2, P=4096, C=320, G=32), dict(N=5, P=300, C=81, G=3, act="gelu", ragged=True),
    dict(N=7, P=100, C=96, G=6, ragged=True, type="f32"), dict(N=1, P=20000, C=16, G=2),
    dict(N=1, P=50000, C=3, G=1, type="f32"), dict(N=2, P=9, C=2052 * 2, G=2, act="gelu"),
    dict(N=2, P=37, C=16384, G=1), dict(N=2, P=5, C=16383, G=1, type="f32"),
    dict(N=2, P=33, C=3000, G=3, type="f32"), dict(N=1, P=40, C=2600, G=2),
    dict(N=2, P=70, C=512, G=512, act="none"), dict(N=2, P=70, C=2560, G=2560, type="f32"),
    dict(N=3, P=65, C=40, G=4, pad=8), dict(N=3, P=65, C=40, G=4, pad=3),
    dict(N=3, P=65, C=40, G=4, offset=1), dict(N=2, P=65, C=24, G=1, offset=2, type="f32"),
    dict(N=2, P=500, C=64, G=8, weight=False, bias=False), dict(N=2, P=500, C=64, G=8, weight=False,
                                                             act="none", param="f32"),
    dict(N=2, P=500, C=64, G=8, bias=False, act="gelu"), dict(N=40, P=200, C=1000, G=8, type="f32"),
    dict(N=2, P=3000, C=64, G=8, mean=1000.0, type="f32", act="none"),
    dict(N=2, P=300, C=64, G=8, mean=-30.0, eps=1e-3), dict(N=30, P=1000, C=640, G=32, ragged=True),
    dict(N=1200, P=4, C=64, G=8, type="f32"), dict(N=4, P=2500, C=17, G=17, act="gelu"),
    dict(N=64, P=256, C=128, G=32, param="f32"), dict(N=9, P=1024, C=72, G=9),
]
IDS = ["-".join("%s%s" % kv for kv in c.items()) for c in CASES]


def statistics(c, n):
    v = c.x[n, :c.len[n]].double().view(c.len[n], c.G, c.per)
    if c.len[n] == 0:
        zero = torch.zeros(c.G, dtype=torch.float64, device="cuda")
        # eps, its root and the quotient are rounded here too: er of the docstring with em = 0
        return zero, zero + c.eps ** -0.5, zero, zero + 304 * U
    mean = v.mean((0, 2))
    var = ((v - mean[:, None]) ** 2).mean((0, 2))
    rstd = 1 / torch.sqrt(var + c.eps)
    em = 416 * U * (mean.abs() + 2 * (v - mean[:, None]).abs().amax((0, 2)))
    er = 304 * U + em ** 2 * rstd ** 2 / 2
    return mean, rstd, em, er


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, in_place):
    c = Case(**case)
    x = c.x.clone()
    if in_place:
        buf, y = c.xbuf, c.x
    else:
        buf, y = place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    before = y.clone()
    stats = torch.full((c.N, c.G, 2), -7.0, device="cuda")
    want = [statistics(c, n) for n in range(c.N)]
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), weight=c.w, bias=c.b, lengths=c.lengths,
                              act=c.act, eps=c.eps)
    w, b = c.wide(c.w, 1.0), c.wide(c.b, 0.0)
    for n in range(c.N):
        mean, rstd, em, er = want[n]
        close(stats[n, :, 0], mean, em, "mean")
        close(stats[n, :, 1], rstd, er * rstd, "rstd")
        L = c.len[n]
        z0 = (x[n, :L].double() - c.spread(mean)) * c.spread(rstd) * w
        z = z0 + b
        ez = (c.spread(em * rstd) * w.abs() + z0.abs() * (c.spread(er) + 4 * U)
              + 2 * U * (z.abs() + b.abs()))
        out = act64(z, c.act)[0]
        ey = 1.13 * ez + (14 + 3 * z.abs()) * U * (out.abs() + z.abs() * 2.0 ** -10)
        if c.act == "gelu":
            ey = ey + 40 * U * z.abs()
        close(y[n, :L], out, ey, "y of sample %d" % n)
        assert torch.equal(y[n, L:].nan_to_num(), before[n, L:].nan_to_num())
    rows = buf[c.offset:c.offset + c.N * c.P * (c.C + c.pad)].view(c.N * c.P, -1)
    assert torch.all(rows[:, c.C:] == 7) and torch.all(buf[-16:] == 7)
    assert torch.all(c.scratch[c.need:] == 255)
    if not in_place:
        again, only = torch.full_like(stats, 3.0), place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)[1]
        Z.zero_group_norm_forward(c.x, only, again, c.scr(), weight=c.w, bias=c.b,
                                  lengths=c.lengths, act=c.act, eps=c.eps)
        assert torch.equal(stats, again) and torch.equal(only, y)
        only.fill_(7.0)
        Z.zero_group_norm_forward(c.x, only, None, c.scr(), weight=c.w, bias=c.b, groups=c.G,
                                  lengths=c.lengths, act=c.act, eps=c.eps)
        assert torch.equal(only, y)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    c = Case(**case)
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    for n in range(c.N):
        mean, rstd, _, _ = statistics(c, n)
        stats[n, :, 0], stats[n, :, 1] = mean, rstd
    buf, dx = place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    grad_type = torch.float32 if c.type == torch.float32 else torch.bfloat16
    dw, db = (torch.full((c.C + 1,), 9.0, dtype=grad_type, device="cuda")[1:] for _ in range(2))
    common = dict(weight=c.w, bias=c.b, lengths=c.lengths, act=c.act)
    Z.zero_group_norm_backward(c.x, c.dy, stats, dx, c.scr(), dweight=dw, dbias=db, **common)
    w, b = c.wide(c.w, 1.0), c.wide(c.b, 0.0)
    sums = {k: torch.zeros(c.C, dtype=torch.float64, device="cuda") for k in ("w", "b", "ew", "eb")}
    K = 64 + 256 + 5120 + c.N / 8 + 16  # runs are less than 5120 in every case here
    for n in range(c.N):
        L = c.len[n]
        mean, rstd = c.spread(stats[n, :, 0].double()), c.spread(stats[n, :, 1].double())
        h = (c.x[n, :L].double() - mean) * rstd
        dy = c.dy[n, :L].double()
        z = h * w + b
        slope = act64(z, c.act)[1]
        es = 0.0
        if c.act != "none":
            es = (24 + 6 * z.abs()) * U + 0.8 * U * (5 * (h * w).abs() + 2 * b.abs())
            if c.act == "gelu":
                es = es + (41 + 41 * z.abs()) * U
        d = dy * slope
        ed = dy.abs() * es + 2 * U * d.abs()
        eh = 3 * U * h.abs()
        sums["w"] += (d * h).sum(0)
        sums["b"] += d.sum(0)
        sums["ew"] += (ed * h.abs() + d.abs() * eh + K * U * (d * h).abs()).sum(0)
        sums["eb"] += (ed + K * U * d.abs()).sum(0)
        if L == 0:
            assert torch.all(dx[n] == 7)
            continue
        over = lambda v: c.spread(v.sum(0).view(c.G, c.per).sum(1) / (L * c.per))
        dw_, M = d * w, K + c.per / 32 + 16
        s1, s2 = over(dw_), over(dw_ * h)
        e1 = over(ed * w.abs() + M * U * dw_.abs())
        e2 = over((ed * h.abs() + d.abs() * eh) * w.abs() + M * U * (dw_ * h).abs())
        want = rstd * (dw_ - s1 - h * s2)
        tol = rstd * (ed * w.abs() + e1 + h.abs() * e2 + eh * s2.abs()
                      + 4 * U * (dw_.abs() + s1.abs() + (h * s2).abs()))
        close(dx[n, :L], want, tol, "dx of sample %d" % n)
        assert torch.all(dx[n, L:] == 7)
    close(dw, sums["w"], sums["ew"], "dweight")
    close(db, sums["b"], sums["eb"], "dbias")
    rows = buf[c.offset:c.offset + c.N * c.P * (c.C + c.pad)].view(c.N * c.P, -1)
    assert torch.all(rows[:, c.C:] == 7) and torch.all(buf[-16:] == 7)
    assert torch.all(c.scratch[c.need:] == 255)
    # each gradient alone, and dx in dy's place: the same bits
    only = place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)[1]
    Z.zero_group_norm_backward(c.x, c.dy, stats, only, c.scr(), **common)
    assert torch.equal(only, dx)
    one = torch.empty_like(dw)
    Z.zero_group_norm_backward(c.x, c.dy, stats, None, c.scr(), dweight=one, **common)
    assert torch.equal(one, dw)
    Z.zero_group_norm_backward(c.x, c.dy, stats, None, c.scr(), dbias=one, **common)
    assert torch.equal(one, db)
    dy = c.dy.clone(memory_format=torch.preserve_format) if c.pad == 0 else c.dy
    if c.pad == 0 and c.offset:
        dy = c.dy
    Z.zero_group_norm_backward(c.x, dy, stats, dy, c.scr(), **common)
    for n in range(c.N):
        assert torch.equal(dy[n, :c.len[n]], dx[n, :c.len[n]])


def test_outliers_keep_the_variance():
    """A first value far from the others: the shift that the sums start from."""
    x = torch.randn((2, 1000, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x[:, 0] = 1e4
    x[:, 100] = -1e4
    c = Case(N=2, P=1000, C=64, G=8, type="f32", act="none")
    c.x.copy_(x)
    y, stats = torch.empty_like(c.x), torch.empty((2, 8, 2), device="cuda")
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="none", eps=c.eps)
    for n in range(2):
        mean, rstd, em, er = statistics(c, n)
        close(stats[n, :, 0], mean, em, "mean")
        close(stats[n, :, 1], rstd, er * rstd, "rstd")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_not_finite_values_stay_in_their_group(bad):
    c = Case(N=2, P=100, C=64, G=8, act="silu")
    y, clean = torch.empty_like(c.x), torch.empty_like(c.x)
    stats = torch.empty((2, 8, 2), device="cuda")
    Z.zero_group_norm_forward(c.x, clean, stats, c.scr(), weight=c.w, bias=c.b)
    c.x[1, 17, 9] = bad
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), weight=c.w, bias=c.b)
    assert torch.isnan(y[1, :, 8:16]).all()
    y[1, :, 8:16] = clean[1, :, 8:16]
    assert torch.equal(y, clean)


def test_gradient_against_differences():
    """fp32: the derivative of sum(dy * y) along a direction, by central differences of
    the definition in fp64 around the same x (an error of step^2), against dx."""
    c = Case(N=2, P=30, C=24, G=3, type="f32", param="f32", act="silu")
    stats = torch.empty((2, 3, 2), device="cuda")
    y, dx = torch.empty_like(c.x), torch.empty_like(c.x)
    dw, db = torch.empty(24, device="cuda"), torch.empty(24, device="cuda")
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), weight=c.w, bias=c.b, eps=c.eps)
    Z.zero_group_norm_backward(c.x, c.dy, stats, dx, c.scr(), weight=c.w, bias=c.b, dweight=dw,
                               dbias=db)
    gen = torch.Generator("cuda").manual_seed(1)

    def value(x, w, b):
        v = x.view(2, 30, 3, 8)
        mean = v.mean((1, 3), keepdim=True)
        h = ((v - mean) / torch.sqrt(((v - mean) ** 2).mean((1, 3), keepdim=True) + c.eps)).view(x.shape)
        return (act64(h * w + b, "silu")[0] * c.dy.double()).sum()

    at = [t.double() for t in (c.x, c.w, c.b)]
    for k, grad in enumerate((dx, dw, db)):
        way = torch.randn(at[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        step = 1e-4
        ends = [[v + (s * step * way if i == k else 0.0) for i, v in enumerate(at)] for s in (1, -1)]
        slope = float((value(*ends[0]) - value(*ends[1])) / (2 * step))
        # fp32 sums of 1440 terms and the statistics' rounding: 1e-4 of the magnitudes at most
        size = float((grad.double().abs() * way.abs()).sum())
        assert abs(float((grad.double() * way).sum()) - slope) <= 1e-4 * size + 1e-6


def test_empty_sizes():
    scratch = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for shape in ((0, 5, 8), (2, 0, 8)):
        x = torch.empty(shape, device="cuda")
        stats = torch.full((shape[0], 2, 2), 5.0, device="cuda")
        Z.zero_group_norm_forward(x, torch.empty_like(x), stats, scratch, eps=0.25)
        assert torch.all(stats[..., 0] == 0) and torch.all(stats[..., 1] == 2)
        dw, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
        Z.zero_group_norm_backward(x, x, stats, torch.empty_like(x), scratch, dweight=dw, dbias=db)
        assert torch.all(dw == 0) and torch.all(db == 0)


def test_pictures_and_slices():
    """[samples, height, width, channels], and half of the channels of a wider tensor."""
    gen = torch.Generator("cuda").manual_seed(5)
    both = torch.randn((2, 6, 7, 64), generator=gen, device="cuda")
    x = both[..., 32:]
    y, stats = torch.empty((2, 6, 7, 32), device="cuda"), torch.empty((2, 4, 2), device="cuda")
    scratch = torch.empty(Z.zero_group_norm_scratch_bytes(2, 42, 32, 4), dtype=torch.uint8,
                          device="cuda")
    Z.zero_group_norm_forward(x, y, stats, scratch, act="none")
    flat = torch.empty((2, 42, 32), device="cuda")
    Z.zero_group_norm_forward(x.reshape(2, 42, 32), flat, stats, scratch, act="none")
    assert torch.equal(y.view(2, 42, 32), flat)


def test_captured_and_on_another_stream():
    c = Case(N=3, P=200, C=64, G=8)
    y, dx = torch.empty_like(c.x), torch.empty_like(c.x)
    stats = torch.empty((3, 8, 2), device="cuda")
    dw, db = torch.empty_like(c.w), torch.empty_like(c.b)

    def call():
        Z.zero_group_norm_forward(c.x, y, stats, c.scr(), weight=c.w, bias=c.b)
        Z.zero_group_norm_backward(c.x, c.dy, stats, dx, c.scr(), weight=c.w, bias=c.b,
                                   dweight=dw, dbias=db)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    outs = (y, stats, dx, dw, db)
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_past_2_31_elements():
    N, P, C, G = 3, 1 << 16, 1 << 14, 32
    x = torch.zeros((N, P, C), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    x[2, :, -512:] = 1.0
    x[2, ::2, -512:] = -1.0
    x[2, 1, -1] = 1.0
    stats = torch.empty((N, G, 2), device="cuda")
    scratch = torch.empty(Z.zero_group_norm_scratch_bytes(N, P, C, G), dtype=torch.uint8,
                          device="cuda")
    Z.zero_group_norm_forward(x, x, stats, scratch, act="none", eps=1e-5)
    assert float(stats[2, 31, 0]) == 0.0
    assert abs(float(stats[2, 31, 1]) - 1 / math.sqrt(1 + 1e-5)) < 1e-6
    assert float(x[2, 1, -1]) == 1.0 and float(x[2, 0, -1]) == -1.0 and float(x[1, 5, 5]) == 0.0
