"""GELU of fp32 tensors to fp32's own precision, on every way the group norm runs.

With u = 2^-24, phi the density and Phi the probability at z < 0: Phi = exp(-z^2 / 2) t Q(t).  Q is
fitted to 3.0e-8 = 0.51 u; with its fp32 roundings t Q(t) is right to 5.1 u (every step emulated at
400,000 values of z in 0 .. 13, t rounded correctly).  t is a unit of the last place off, 2 u, and t Q(t)
changes by at most 1.2 times that: 7.5 u.  The exponent has one rounding, u z^2 / 2, the exponential 2
units of the last place (4 u), the product u: Phi is right to (13 + z^2 / 2) u, and 1 - Phi for z > 0 to that
of Phi and u more.  phi is right to (6 + z^2 / 2) u, with its constant and product.  y = z Phi has another
u, and the slope Phi + z phi its own.  Results below 2^-126 may be 0.
"""
import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z
import test_gpu_group_norm as T

pytestmark = pytest.mark.gpu
U = T.U
WAYS = [dict(N=2, P=300, C=64, G=8), dict(N=2, P=200, C=33, G=3), dict(N=1, P=9000, C=64, G=8),
        dict(N=3, P=9001, C=33, G=3), dict(N=3, P=400, C=33, G=3, pad=1)]
IDS = ["held", "held_along", "passes", "along", "single"]


def parts(z):
    """phi, Phi and how far off each may be."""
    phi = torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    half = z * z / 2
    tail = 0.5 * torch.special.erfc(z.abs() * 0.5 ** 0.5)
    off = tail * (13 + half) * U + torch.where(z > 0, U, 0.0)
    return phi, 0.5 * torch.special.erfc(-z * 0.5 ** 0.5), off, phi * (6 + half) * U


@pytest.mark.parametrize("way", WAYS, ids=IDS)
def test_forward(way):
    c = T.Case(type="f32", act="gelu", weight=False, bias=False, mean=0.0, **way)
    c.x.mul_(1 + c.x.abs())  # long tails: up to some ten deviations
    stats = torch.empty((c.N, c.G, 2), device="cuda")
    _, y = T.place((c.N, c.P, c.C), c.type, c.pad, 0, None)
    Z.zero_group_norm_forward(c.x, y, stats, c.scr(), act="gelu")
    mean, rstd = (stats[..., i].double().repeat_interleave(c.per, 1)[:, None] for i in (0, 1))
    z = (c.x.double() - mean) * rstd  # from the statistics as they were written
    assert float(z.min()) < -4
    phi, cdf, off, _ = parts(z)
    slope = (cdf + z * phi).abs() + 3 * U * (z.abs() + 1)
    ez = 3 * U * z.abs()  # the difference and the product; the bias is 0
    tol = slope * ez + z.abs() * off + U * (z * cdf).abs()
    T.close(y, z * cdf, tol, "y")


@pytest.mark.parametrize("way", WAYS, ids=IDS)
def test_slope(way):
    """Statistics of mean 0 and deviation 1, and one row that counts: dbias is its dy * slope(x)."""
    c = T.Case(type="f32", act="gelu", weight=False, bias=False, mean=0.0, **way)
    c.x.mul_(1 + c.x.abs())
    stats = torch.zeros((c.N, c.G, 2), device="cuda")
    stats[..., 1] = 1.0
    db = torch.empty(c.C, device="cuda")
    for n, row in ((0, 0), (c.N - 1, c.P - 1), (c.N - 1, c.P // 2)):
        c.dy.zero_()
        c.dy[n, row] = 1.0
        Z.zero_group_norm_backward(c.x, c.dy, stats, None, c.scr(), dbias=db, act="gelu")
        z = c.x[n, row].double()
        phi, cdf, off, off_phi = parts(z)
        want = cdf + z * phi
        T.close(db, want, off + z.abs() * off_phi + U * want.abs(), "slope")
