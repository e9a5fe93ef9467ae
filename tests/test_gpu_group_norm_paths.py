"""Sizes that reach every way the group norm runs: slabs held in one block, two passes by
vectors (whole rows, or along a sample, or groups wider than a slab in parts), and a channel
at a time; with the bounds of test_gpu_group_norm.py."""
import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z
import test_gpu_group_norm as T

pytestmark = pytest.mark.gpu

CASES = [
    # two passes: whole rows, ragged and padded
    dict(N=7, P=6000, C=64, G=8, ragged=True), dict(N=5, P=5000, C=72, G=9, ragged=True, act="gelu"),
    dict(N=2, P=3000, C=640, G=32, pad=16), dict(N=3, P=7000, C=64, G=2, type="f32", ragged=True),
    dict(N=2, P=6000, C=32, G=8, act="none", type="f32"), dict(N=2, P=9000, C=24, G=6, act="gelu"),
    # as many groups as a slab has channels: the most shared memory
    dict(N=2, P=3000, C=2048, G=2048), dict(N=1, P=2500, C=2048, G=1024, type="f32", act="none"),
    # along a sample
    dict(N=7, P=5001, C=81, G=3, ragged=True, act="gelu"), dict(N=3, P=9001, C=19, G=1, type="f32", ragged=True),
    dict(N=2, P=8191, C=64, G=8, offset=3), dict(N=3, P=20001, C=5, G=5), dict(N=2, P=7001, C=21, G=3, act="none"),
    dict(N=2, P=6001, C=30, G=3, offset=1, type="f32"), dict(N=1, P=70001, C=2, G=1),
    # groups wider than a slab
    dict(N=2, P=300, C=4096, G=1), dict(N=2, P=70, C=8192, G=2, ragged=True, act="gelu"),
    dict(N=3, P=40, C=6144, G=2, type="f32"),
    # a channel at a time
    dict(N=3, P=900, C=33, G=3, pad=1, ragged=True), dict(N=2, P=2000, C=1017, G=3, act="gelu"),
    dict(N=2, P=3000, C=300, G=100, pad=2, type="f32"), dict(N=2, P=50, C=2052, G=1, type="f32", ragged=True),
    # held, several samples and slabs to a block
    dict(N=400, P=100, C=128, G=8, ragged=True), dict(N=700, P=33, C=72, G=3, act="gelu"),
    dict(N=650, P=64, C=45, G=9, ragged=True), dict(N=330, P=20, C=1024, G=32, type="f32", param="f32"),
    dict(N=40, P=10, C=16384, G=512, act="none"), dict(N=400, P=9, C=12, G=6), dict(N=400, P=11, C=7, G=7),
    # fp32 through the activations
    dict(N=4, P=500, C=64, G=8, type="f32", act="silu", mean=-2.0, param="f32"),
]
IDS = ["-".join("%s%s" % kv for kv in c.items()) for c in CASES]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, in_place):
    T.test_forward(case, in_place)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    T.test_backward(case)


@pytest.mark.parametrize("shape", [(2, 300, 64, 8), (1, 9000, 64, 8), (2, 400, 33, 3)],
                         ids=["held", "passes", "along"])
def test_gelu_in_fp32(shape):
    """GELU's cumulative probability is a polynomial of absolute error 7.5e-8 (Abramowitz and
    Stegun 26.2.17) with coefficients of magnitudes that add to 5.7, times a density of at most
    0.4: 16 roundings of that, 16 * 5.7 * 0.4 u = 37 u, and 1.3 u of the method: 40 u absolute.
    So y is right to 1.13 ez + 40 u |z| + 4 u |y| and the slope to (41 + 41 |z|) u + 0.8 ez."""
    n, p, c, g = shape
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((n, p, c), generator=gen, device="cuda") * 2
    dy = torch.randn((n, p, c), generator=gen, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty((n, g, 2), device="cuda")
    dw, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    s = torch.empty(Z.zero_group_norm_scratch_bytes(n, p, c, g), dtype=torch.uint8, device="cuda")
    Z.zero_group_norm_forward(x, y, stats, s, act="gelu")
    Z.zero_group_norm_backward(x, dy, stats, dx, s, dweight=dw, dbias=db, act="gelu")
    per = c // g
    mean, rstd = (stats[..., i].double().repeat_interleave(per, 1)[:, None] for i in (0, 1))
    z = (x.double() - mean) * rstd  # from the statistics as they were written
    out, slope = T.act64(z, "gelu")
    ez = 5 * T.U * (z.abs() + mean.abs() * rstd)
    T.close(y, out, 1.13 * ez + 40 * T.U * z.abs() + 4 * T.U * out.abs(), "y")
    d = dy.double() * slope
    ed = dy.abs().double() * ((41 + 41 * z.abs()) * T.U + 0.8 * ez) + 2 * T.U * d.abs()
    K = 64 + 256 + 600 + 16  # roundings of a term in its sums, at most
    for got, value, bound in ((db, d, ed), (dw, d * z, ed * z.abs() + d.abs() * ez)):
        T.close(got, value.sum((0, 1)), (bound + K * T.U * value.abs()).sum((0, 1)), "sums")


def test_tiny_eps_and_constant_groups():
    """A group of one value has a variance of 0: rstd is 1/sqrt(eps), nothing overflows."""
    for shape in ((2, 64, 32, 4), (1, 9000, 64, 8), (2, 64, 33, 3)):
        n, p, c, g = shape
        x = torch.full((n, p, c), 3.0, device="cuda")
        y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty((n, g, 2), device="cuda")
        b = torch.full((c,), 0.5, device="cuda")
        s = torch.empty(Z.zero_group_norm_scratch_bytes(n, p, c, g), dtype=torch.uint8, device="cuda")
        Z.zero_group_norm_forward(x, y, stats, s, bias=b, act="none", eps=1e-37)
        assert torch.all(y == 0.5) and torch.all(stats[..., 0] == 3.0)
        Z.zero_group_norm_backward(x, torch.ones_like(x), stats, dx, s, bias=b, act="none")
        # d w - s1 is 0 but for the rounding of the mean of ones
        assert torch.isfinite(dx).all() and float(dx.abs().max()) <= 4 * T.U * float(stats[..., 1].max())
