"""The group norm's sums where they are hardest: means that are large beside the deviations.

Bounds, with u = 2^-24, D the largest |x - mean| of a group and m its |mean|.  Sums are of
differences from a value of the group, so a rounding is of at most 2 D: a thread has at most 64
rows and 3 more roundings, its block's row groups and lanes 256 + 5, the runs (of 4 rows at
least) P / 32 + 13 and the channels or parts of a group per / 32 + 10.  Each of those four
steps rounds its mean once: em = 4 u m + (352 + P / 32 + per / 32) u 2 D.  The variance adds the squares of
parts' means about the common one; means that are off by em move those by 2 d em each, and em^2: em
rstd + em^2 rstd^2 / 2 relative in 1/sqrt(variance + eps), besides the 304 u of test_gpu_group_norm.py.
"""
import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z
import test_gpu_group_norm as T

pytestmark = pytest.mark.gpu
U = T.U

SINGLE = [  # a channel at a time
    dict(N=1, P=16384, C=1279, G=1), dict(N=2, P=9001, C=33, G=3, pad=1), dict(N=6, P=700, C=1017, G=3, ragged=True),
    dict(N=3, P=5, C=2052, G=1, offset=1), dict(N=2, P=2500, C=300, G=100, pad=2), dict(N=1, P=40000, C=3, G=1, pad=1),
]


def ids(cases):
    return ["-".join("%s%s" % kv for kv in c.items()) for c in cases]


def check_statistics(c, stats):
    for n in range(c.N):
        if c.len[n] == 0:
            continue
        v = c.x[n, :c.len[n]].double().view(c.len[n], c.G, c.per)
        mean = v.mean((0, 2))
        d = v - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).mean((0, 2)) + c.eps)
        em = 4 * U * mean.abs() + (352 + c.P / 32 + c.per / 32) * U * 2 * d.abs().amax((0, 2))
        T.close(stats[n, :, 0], mean, em, "mean")
        T.close(stats[n, :, 1], rstd, (304 * U + em * rstd + em ** 2 * rstd ** 2 / 2) * rstd, "rstd")


@pytest.mark.parametrize("mean", [1000.3, -500.1])
@pytest.mark.parametrize("case", SINGLE, ids=ids(SINGLE))
def test_large_mean_a_channel_at_a_time(case, mean):
    c = T.Case(type="f32", act="none", mean=mean, weight=False, bias=False, **case)
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    _, y = T.place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="none", groups=c.G, eps=c.eps, lengths=c.lengths)
    check_statistics(c, stats)


HELD = [dict(N=2, P=300, C=64, G=8), dict(N=3, P=700, C=45, G=3, ragged=True), dict(N=1, P=200, C=96, G=24),
        dict(N=5, P=1, C=4096, G=32), dict(N=400, P=9, C=12, G=6), dict(N=1, P=40, C=2048, G=1)]
PASSES = [dict(N=1, P=300000, C=64, G=1), dict(N=2, P=9000, C=640, G=32), dict(N=7, P=6000, C=72, G=9, ragged=True),
          dict(N=2, P=6000, C=24, G=6), dict(N=2, P=300, C=4096, G=1)]
ALONG = [dict(N=1, P=200000, C=33, G=1), dict(N=7, P=5001, C=81, G=3, ragged=True), dict(N=3, P=20001, C=5, G=5),
         dict(N=2, P=8191, C=64, G=8, offset=3)]


@pytest.mark.parametrize("mean", [1000.3, -500.1])
@pytest.mark.parametrize("case", HELD + PASSES + ALONG, ids=ids(HELD + PASSES + ALONG))
def test_large_mean(case, mean):
    test_large_mean_a_channel_at_a_time(case, mean)


@pytest.mark.parametrize("value", [1000.3, -0.1, 7e-5])
@pytest.mark.parametrize("case", SINGLE + HELD + PASSES + ALONG, ids=ids(SINGLE + HELD + PASSES + ALONG))
def test_groups_of_one_value(case, value):
    """A mean of parts that all are v is v again: a sum of them comes to v (1 + k u) for a few k,
    all differences from that are -v k u exactly, their mean the same up to its own rounding, and v
    is the number next to the corrected one.  Then every x - mean is 0, and y is the bias."""
    c = T.Case(type="f32", act="none", **case)
    c.x.fill_(value)
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    _, y = T.place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="none", bias=c.b, eps=c.eps, lengths=c.lengths)
    for n in range(c.N):
        if c.len[n]:
            assert torch.all(stats[n, :, 0] == c.x[n, 0, 0]), "mean"
            assert torch.all(y[n, :c.len[n]] == c.b.float()), "y"
