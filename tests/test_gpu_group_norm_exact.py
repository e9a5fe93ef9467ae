"""The group norm's sums where one lost or doubled value shows, on every way it runs.

Gradient: with statistics of mean 0 and deviation 1 and no activation, whole x, dy and weights of
-2 .. 2 have sums below 2^24, which fp32 holds: dweight and dbias are exact.  dx = d w - s1 - h s2
has sums that are whole, times an fp32 1 / size of an fp32 size: s1 and s2 are right to 3 u, the
result's three operations round u each of at most |d w| + |s1| + |h s2|: 6 u of that.

Statistics: N samples of which each holds ones in every N-th row, another one's in each.  The mean
of a group is m = (ones) / (values), its deviations add to 2 m (1 - m) of the values.  A thread's
sums are whole, its means right to 2 u; a join of k parts rounds k times by u of a partial sum of
differences, and those are at most 2 m (1 - m) (1 + 2^-10) of the values: with the docstring of
test_gpu_group_norm_sums.py em = 12 u + (352 + P / 32 + per / 32) u 4 m.  A vector of eight values
is 8 / (P per) of the mean, three times em and more in every case here.
"""
import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z
import test_gpu_group_norm as T

pytestmark = pytest.mark.gpu
U = T.U

GRADIENT = {
    "held": dict(N=700, P=33, C=72, G=3), "held-many": dict(N=2, P=300, C=64, G=8),
    "held-ragged": dict(N=400, P=100, C=128, G=8, ragged=True), "held-f32": dict(N=9, P=64, C=256, G=32, type="f32"),
    "held-along": dict(N=650, P=64, C=45, G=9, ragged=True), "held-along-small": dict(N=400, P=11, C=7, G=7),
    "one position": dict(N=5000, P=1, C=1024, G=32),
    "passes": dict(N=7, P=6000, C=64, G=8, ragged=True), "passes-wide": dict(N=2, P=3000, C=640, G=32, pad=16),
    "passes-f32": dict(N=3, P=7000, C=64, G=2, type="f32", ragged=True), "passes-long": dict(N=2, P=9000, C=24, G=6),
    "passes-split": dict(N=2, P=300, C=4096, G=1), "passes-groups": dict(N=2, P=3000, C=2048, G=2048),
    "along": dict(N=7, P=5001, C=81, G=3, ragged=True), "along-one": dict(N=3, P=9001, C=19, G=1, type="f32", ragged=True),
    "along-offset": dict(N=2, P=8191, C=64, G=8, offset=3), "along-long": dict(N=1, P=70001, C=2, G=1),
    "along-channels": dict(N=3, P=20001, C=5, G=5), "along-24": dict(N=24, P=3001, C=81, G=3, ragged=True),
    "along-wide": dict(N=16, P=2000, C=201, G=3),
    "single": dict(N=3, P=900, C=33, G=3, pad=1, ragged=True), "single-wide": dict(N=2, P=2000, C=1017, G=3),
    "single-f32": dict(N=2, P=3000, C=300, G=100, pad=2, type="f32"), "single-odd": dict(N=2, P=50, C=2052, G=1, ragged=True),
}


@pytest.mark.parametrize("weighted", [False, True], ids=["plain", "weighted"])
@pytest.mark.parametrize("case", GRADIENT.values(), ids=GRADIENT.keys())
def test_gradient_of_whole_numbers(case, weighted):
    c = T.Case(act="none", weight=False, bias=False, param="f32", **case)
    gen = torch.Generator("cuda").manual_seed(c.N + c.P)
    whole = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda")
    nan = torch.isnan(c.x)
    c.x.copy_(whole(c.N, c.P, c.C))
    c.dy.copy_(whole(c.N, c.P, c.C))
    x, dy = (torch.where(nan, 0.0, t.double()) for t in (c.x, c.dy))
    c.x[nan] = c.dy[nan] = float("nan")  # behind the lengths
    w = whole(c.C).float() if weighted else None
    stats = torch.zeros((c.N, c.G, 2), device="cuda")
    stats[..., 1] = 1.0
    dw, db = torch.empty(c.C, device="cuda"), torch.empty(c.C, device="cuda")
    _, dx = T.place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    Z.zero_group_norm_backward(c.x, c.dy, stats, dx, c.scr(), weight=w, lengths=c.lengths, dweight=dw, dbias=db,
                               act="none")
    assert torch.equal(db.double(), dy.sum((0, 1))), "dbias"
    assert torch.equal(dw.double(), (dy * x).sum((0, 1))), "dweight"
    d = dy if w is None else dy * w.double()
    size = torch.tensor(c.len, dtype=torch.float64, device="cuda").clamp(min=1)[:, None] * c.per
    s1, s2 = ((v.sum(1).view(c.N, c.G, c.per).sum(2) / size).repeat_interleave(c.per, 1)[:, None]
              for v in (d, d * x))
    want, tol = d - s1 - x * s2, 6 * U * (d.abs() + s1.abs() + (x * s2).abs())
    for n in range(0, c.N, max(1, c.N // 40)):
        L = c.len[n]
        T.close(dx[n, :L], want[n, :L], tol[n, :L], "dx of sample %d" % n)
        assert torch.all(dx[n, L:] == 7)


STATISTICS = {
    "held": dict(N=50, P=300, C=64, G=8), "held-few": dict(N=20, P=33, C=72, G=3), "held-wide": dict(N=16, P=64, C=1280, G=32),
    "held-along": dict(N=30, P=400, C=33, G=3), "passes": dict(N=60, P=6000, C=64, G=8),
    "passes-wide": dict(N=32, P=3000, C=320, G=32), "passes-split": dict(N=100, P=200, C=4096, G=1),
    "along": dict(N=60, P=5001, C=81, G=3), "along-one": dict(N=60, P=9001, C=19, G=1),
    "along-offset": dict(N=40, P=4001, C=64, G=8, offset=3),
    "single": dict(N=40, P=900, C=33, G=3, pad=1), "single-wide": dict(N=40, P=1000, C=321, G=3),
}


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("case", STATISTICS.values(), ids=STATISTICS.keys())
def test_statistics_see_every_row(case, type):
    c = T.Case(type=type, act="none", weight=False, bias=False, **case)
    rows = torch.arange(c.P, device="cuda")
    ones = (rows[None] % c.N == torch.arange(c.N, device="cuda")[:, None])[:, :, None]
    c.x.copy_(ones.expand(c.N, c.P, c.C))
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    _, y = T.place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="none", eps=c.eps)
    m = ones.double().mean(1)  # [N, 1]: the same for every group
    em = 12 * U + (352 + c.P / 32 + c.per / 32) * U * 4 * m
    assert float((em * c.P * c.per).max()) < 8 / 3
    T.close(stats[..., 0], m.expand(c.N, c.G), em.expand(c.N, c.G), "mean")
    rstd = 1 / torch.sqrt(m - m * m + c.eps)
    # as in test_gpu_group_norm_sums.py
    er = 304 * U + em * rstd + em ** 2 * rstd ** 2 / 2
    T.close(stats[..., 1], rstd.expand(c.N, c.G), (er * rstd).expand(c.N, c.G), "rstd")
    mean, rstd = (stats[..., i].double().repeat_interleave(c.per, 1)[:, None] for i in (0, 1))
    z = (c.x.double() - mean) * rstd
    T.close(y, z, 3 * U * z.abs(), "y")
