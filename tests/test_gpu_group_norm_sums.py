"""The group norm's sums where they are hardest: means that are large beside the deviations.

Bounds, with u = 2^-24, D the largest |x - mean| of a group and m its |mean|.  Sums are of
differences from a value of the group, so a rounding is of at most 2 D: a thread has at most 64
rows and 3 more roundings, its block's row groups and lanes 256 + 5, the runs (of 4 rows at
least) P / 32 + 13 and the channels or parts of a group per / 32 + 10.  Each of those four
steps rounds its mean once: em = 4 u m + (352 + P / 32 + per / 32) u 2 D.  1/sqrt(variance + eps) is
right to 304 u + em^2 rstd^2 / 2, as in test_gpu_group_norm.py.
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
        T.close(stats[n, :, 1], rstd, (304 * U + em ** 2 * rstd ** 2 / 2) * rstd, "rstd")


@pytest.mark.parametrize("mean", [1000.3, -500.1])
@pytest.mark.parametrize("case", SINGLE, ids=ids(SINGLE))
def test_large_mean_a_channel_at_a_time(case, mean):
    c = T.Case(type="f32", act="none", mean=mean, weight=False, bias=False, **case)
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    _, y = T.place((c.N, c.P, c.C), c.type, c.pad, c.offset, None)
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="none", groups=c.G, eps=c.eps, lengths=c.lengths)
    check_statistics(c, stats)
