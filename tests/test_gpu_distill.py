"""zero_distill_forward and zero_distill_forward_backward against fp64 forms.

Bounds, with u = 2^-24.  An exponential is taken of a difference d <= 0 from the
row's maximum: rounding the argument costs 4u|d|, the exponential itself 8u.
A sum of V of them is at most V/128 additions deep in a thread and 20 levels
above, so log Z is right to (V/128 + 64) u plus what |d| e^d <= 1 allows, which
the 64 holds too.  ce adds 4u (|s - m| + log Z); kl has the two sums and the
cross term, 16u sum p (|t - tm| + |s - m|) / tau, all times tau^2.  The
gradient's parts carry the relative error of q and p; a result in bf16 adds half
an ulp of it.
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


def reference(s, t, ids, labels, weight, tau, cw, kw):
    """ce, kl, dlogits and their error bounds (before rounding to bf16), fp64."""
    R, V = s.shape
    ce, kl, g = np.zeros(R), np.zeros(R), np.zeros((R, V))
    ce_tol, kl_tol, g_tol = np.zeros(R), np.zeros(R), np.zeros((R, V))
    deep = (V / 128 + 64) * U
    for r in range(R):
        w = 1.0 if weight is None else weight[r]
        if w == 0 or (s[r] == -np.inf).all():
            continue
        m = s[r].max()
        d = s[r] - m
        with np.errstate(invalid="ignore"):
            slack = np.where(np.isfinite(d), np.abs(d), 0.0)
        ok = (ids[r] >= 0) & (ids[r] < V)
        tt = np.where(ok, t[r], -np.inf)
        if (tt > -np.inf).any():
            z = np.exp(d / tau).sum()
            q = np.exp(d / tau) / z
            td = tt - tt.max()
            p = np.exp(td / tau)
            p /= p.sum()
            on = p > 0
            at = ids[r][on]
            with np.errstate(divide="ignore"):
                kl[r] = tau ** 2 * (p[on] * (np.log(p[on]) - np.log(q[at]))).sum()
            cross = (p[on] * (np.abs(td[on]) + slack[at]) / tau).sum()
            kl_tol[r] = tau ** 2 * (2 * deep + 16 * U * (cross + np.log(z) + np.log(len(p) + 1)))
            f = abs(w * kw * tau)
            g[r] += w * kw * tau * q
            g_tol[r] += f * q * (deep + 8 * U * slack / tau)
            np.add.at(g[r], at, -w * kw * tau * p[on])
            np.add.at(g_tol[r], at, f * p[on] * (deep + 8 * U * np.abs(td[on]) / tau))
        if labels is not None and 0 <= labels[r] < V:
            z = np.exp(d).sum()
            q = np.exp(d) / z
            ce[r] = np.log(z) - d[labels[r]]
            ce_tol[r] = deep + 4 * U * (slack[labels[r]] + np.log(z))
            g[r] += w * cw * q
            g[r, labels[r]] -= w * cw
            g_tol[r] += abs(w * cw) * q * (deep + 8 * U * slack)
            g_tol[r, labels[r]] += abs(w * cw) * 4 * U
    return ce, kl, g, ce_tol, kl_tol, g_tol


def make(R, V, K, logits="bf16", teacher="f32", wide=False, labels=True, stride=None, offset=0,
         seed=0, spread=3.0):
    rng = np.random.default_rng(R * 7 + V + K + seed)
    stride = stride or V
    buf = torch.full((offset + R * stride + 64,), 7.0, dtype=TYPES[logits], device="cuda")
    s = torch.as_strided(buf, (R, V), (stride, 1), offset)
    s.copy_(torch.from_numpy((spread * rng.standard_normal((R, V))).astype(np.float32)))
    t = torch.from_numpy(np.sort(rng.standard_normal((R, K)) * spread)[:, ::-1].astype(np.float32))
    ids = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K)
                    for _ in range(R)])
    short = rng.random(R) < 0.3
    ids[short, K // 2:] = -1
    lab = rng.integers(-1, V, R)
    lab[rng.random(R) < 0.4] = ids[rng.random(R) < 2, 0][0]  # some labels that the teacher holds
    weight = rng.random(R).astype(np.float32) + 0.5
    if R > 2:
        weight[R // 2] = 0.0
    idt = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    return dict(buf=buf, s=s, t=t.to(TYPES[teacher]).cuda(), ids=idt,
                labels=torch.from_numpy(lab).to(torch.int64 if wide else torch.int32).cuda()
                if labels else None, weight=torch.from_numpy(weight).cuda(), offset=offset,
                stride=stride)


def n64(t):
    return None if t is None else t.cpu().double().numpy()


def check(c, tau=1.0, cw=0.4, kw=0.6, weight=True, out_stride=None, in_place=False):
    R, V = c["s"].shape
    w = c["weight"] if weight else None
    lab = None if c["labels"] is None else c["labels"].cpu().numpy()
    ce0, kl0, g0, ct, kt, gt = reference(n64(c["s"]), n64(c["t"]), c["ids"].cpu().numpy(), lab,
                                         n64(w), float(np.float32(tau)), float(np.float32(cw)),
                                         float(np.float32(kw)))
    ce, kl = (torch.full((R,), float("nan"), device="cuda") for _ in range(2))
    B.zero_distill_forward(c["s"], c["t"], c["ids"], ce, kl, labels=c["labels"], row_weight=w,
                           temperature=tau)
    one, two = ce.clone(), kl.clone()
    assert np.all(np.abs(n64(ce) - ce0) <= ct), np.abs(n64(ce) - ce0).max()
    inf = np.isinf(kl0)
    assert np.all(n64(kl)[inf] == kl0[inf])
    assert np.all(np.abs(n64(kl) - kl0)[~inf] <= kt[~inf])
    if in_place:
        g, buf, ostride = c["s"], c["buf"], c["stride"]
    else:
        ostride = out_stride or V
        buf = torch.full((c["offset"] + R * ostride + 64,), 7.0, dtype=c["s"].dtype, device="cuda")
        g = torch.as_strided(buf, (R, V), (ostride, 1), c["offset"])
    B.zero_distill_forward_backward(c["s"], c["t"], c["ids"], ce, kl, g, labels=c["labels"],
                                    row_weight=w, temperature=tau, ce_weight=cw, kl_weight=kw)
    assert np.all(np.abs(n64(ce) - ce0) <= ct)
    assert np.all(np.abs(n64(kl) - kl0)[~inf] <= kt[~inf])
    tol = gt + (half_ulp(np.abs(g0) + gt) if g.dtype == torch.bfloat16 else 2 * U * np.abs(g0))
    off = np.abs(n64(g) - g0) - tol
    assert np.all(off <= 1e-36), off.max()
    # nothing outside the rows was written
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, (R, V), (ostride, 1), c["offset"]).fill_(False)
    assert bool((buf[mask] == 7).all())
    return one, two


@pytest.mark.parametrize("R,V,K,kw", [
    (1, 50257, 16, dict(logits="f32")), (5, 50257, 64, dict()),
    (3, 50257, 64, dict(logits="f32", stride=50304)), (17, 4000, 1, dict(labels=False)),
    (300, 1000, 33, dict(wide=True, teacher="bf16")), (4, 7, 5, dict()), (4, 1, 1, dict()),
    (2, 3, 1024, dict()), (9, 513, 1024, dict(logits="f32")), (40, 32000, 128, dict(teacher="bf16")),
    (6, 4097, 20, dict(offset=1)), (6, 4097, 20, dict(offset=3, logits="f32", stride=4111)),
    (3, 131072, 64, dict()), (2, 200003, 8, dict(logits="f32")), (2, 400001, 8, dict()),
    (160, 8200, 7, dict(stride=8208))])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
def test_losses_and_gradient(R, V, K, kw, tau):
    check(make(R, V, K, **kw), tau)


def test_in_place_equals_apart():
    for kw in (dict(), dict(offset=1), dict(logits="f32", stride=5011)):
        c = make(20, 5003, 12, **kw)
        apart = torch.empty((20, 5003), dtype=c["s"].dtype, device="cuda")
        ce, kl = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
        B.zero_distill_forward_backward(c["s"], c["t"], c["ids"], ce, kl, apart,
                                        labels=c["labels"], row_weight=c["weight"],
                                        temperature=2.0, ce_weight=0.4, kl_weight=0.6)
        check(c, 2.0, in_place=True)
        assert torch.equal(c["s"], apart)


def test_out_stride_and_no_weights():
    check(make(12, 3001, 9), 3.0, weight=False, out_stride=3016)
    check(make(12, 3001, 9, logits="f32"), 0.5, weight=False, out_stride=3003)


def test_masked_places():
    """-inf logits of the student, also at a teacher's entry (kl is +inf, the
    gradient finite), -inf teacher entries, rows with nothing left, a repeated
    id, an id in the last place, and NaN in a row of weight 0."""
    c = make(12, 2051, 6)
    s, t, ids, lab = c["s"], c["t"], c["ids"], c["labels"]
    for r in range(12):
        ids[r] = torch.arange(100 * r, 100 * r + 6)
        lab[r] = 3
    c["weight"].fill_(1.0)
    s[0].fill_(-float("inf"))           # no distribution
    s[1, 1000:] = -float("inf")
    s[2, 202] = -float("inf")           # where the teacher has mass
    t[3, 2:] = -float("inf")
    t[4].fill_(-float("inf"))           # a teacher without any
    ids[5].fill_(-1)
    ids[6] = torch.tensor([9, 9, 3, 9, 3, 8])  # repeated, and the label among them
    ids[7] = torch.tensor([2050, 5000000, -7, 0, 1, 2])
    lab[8] = -100
    lab[9] = 2050
    s[10].fill_(-3e38)                  # equal logits, lowest value of the type
    s[11, :] = torch.finfo(s.dtype).min
    s[11, 5] = 0.0
    check(c, 2.0)
    c["weight"][1] = 0.0
    s[1].fill_(float("nan"))
    check_masked = torch.empty_like(s)
    ce, kl = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
    B.zero_distill_forward_backward(s, t, ids, ce, kl, check_masked, labels=lab,
                                    row_weight=c["weight"], ce_weight=1.0)
    assert not check_masked[1].any() and ce[1] == 0 and kl[1] == 0
    assert torch.isinf(kl[2]) and torch.isfinite(check_masked.float()).all()


def test_nan_and_inf_are_not_hidden():
    c = make(4, 3000, 6)
    c["s"][0, 17] = float("nan")
    c["s"][1, 2999] = float("inf")
    c["s"][2].fill_(float("nan"))
    c["t"][3].fill_(float("nan"))
    c["ids"][:] = torch.arange(6)
    c["labels"].fill_(2)
    c["weight"].fill_(1.0)
    ce, kl = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    g = torch.empty_like(c["s"])
    B.zero_distill_forward_backward(c["s"], c["t"], c["ids"], ce, kl, g, labels=c["labels"],
                                    row_weight=c["weight"], ce_weight=0.5, kl_weight=0.5)
    assert torch.isnan(ce[:3]).all() and torch.isnan(kl).all() and torch.isfinite(ce[3])
    assert torch.isnan(g[2].float()).all()


def test_gradient_agrees_with_differences():
    """Central differences of the fp64 losses along random directions; the step
    2^-10 leaves 2^-20 / 6 of third derivatives of order one."""
    R, V, K, tau = 5, 200, 9, 2.0
    c = make(R, V, K, logits="f32")
    s, t, ids = n64(c["s"]), n64(c["t"]), c["ids"].cpu().numpy()
    lab, w = c["labels"].cpu().numpy(), n64(c["weight"])
    g = torch.empty_like(c["s"])
    ce, kl = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    B.zero_distill_forward_backward(c["s"], c["t"], c["ids"], ce, kl, g, labels=c["labels"],
                                    row_weight=c["weight"], temperature=tau, ce_weight=0.4,
                                    kl_weight=0.6)

    def loss(x):
        a, b = reference(x, t, ids, lab, w, tau, 0.4, 0.6)[:2]
        return (w * (0.4 * a + 0.6 * b)).sum()

    rng = np.random.default_rng(1)
    for _ in range(5):
        d = rng.standard_normal((R, V))
        e = 2.0 ** -10
        numeric = (loss(s + e * d) - loss(s - e * d)) / (2 * e)
        mine = (n64(g) * d).sum()
        assert abs(mine - numeric) <= 1e-5 * np.abs(n64(g) * d).sum() + 1e-6


def test_no_rows_is_nothing():
    e = torch.empty((0, 100), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, device="cuda")
    ids = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    B.zero_distill_forward(e, torch.empty((0, 4), device="cuda"), ids, z, z)
