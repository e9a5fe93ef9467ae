"""Distillation where finite mask values stand in the logits: whole parts of a
row that is split over 2, 4 or 8 blocks, stretches that a thread meets first, and
whole rows.  References and bounds are those of test_gpu_distill: the loss of a
row does not depend on how far below the row's maximum a masked logit without a
teacher's entry lies."""
import numpy as np
import pytest
import torch

import test_gpu_distill
from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu
ROWS = {2: 40, 4: 20, 8: 12}  # rows of which each is split over so many blocks


@pytest.fixture
def log_q(monkeypatch):
    """The reference's kl with log q as a difference: over 700 below the maximum,
    or at a small temperature, the exponential itself is subnormal or 0 in 64 bits."""
    plain = test_gpu_distill.reference

    def reference(s, t, ids, labels, weight, tau, cw, kw):
        with np.errstate(divide="ignore"):
            ce, kl, *rest = plain(s, t, ids, labels, weight, tau, cw, kw)
        for r in np.nonzero(kl)[0]:
            d = (s[r] - s[r].max()) / tau
            on = (ids[r] >= 0) & (ids[r] < s.shape[1]) & (t[r] > -np.inf)
            a = (t[r][on] - t[r][on].max()) / tau
            p = np.exp(a) / np.exp(a).sum()
            terms = a - np.log(np.exp(a).sum()) - d[ids[r][on]] + np.log(np.exp(d).sum())
            with np.errstate(over="ignore"):  # infinite where fp32, the output's type, cannot hold it
                kl[r] = np.float32(tau ** 2 * (p[p > 0] * terms[p > 0]).sum())
        return (ce, kl, *rest)

    monkeypatch.setattr(test_gpu_distill, "reference", reference)


def masked(R, V, K, logits, value, lo, hi):
    """Columns [lo, hi) hold the mask; the teacher's entries and the labels lie outside."""
    c = make(R, V, K, logits=logits)
    gen = torch.Generator(device="cuda").manual_seed(V + lo)
    live = torch.cat([torch.arange(0, max(lo, 0), device="cuda"),
                      torch.arange(min(hi, V), V, device="cuda")])
    c["s"][:, max(lo, 0):hi] = torch.finfo(c["s"].dtype).min if value is None else value
    for r in range(R):
        at = live[torch.randperm(live.numel(), generator=gen, device="cuda")[:K]]
        c["ids"][r] = torch.where(c["ids"][r] < 0, -1, at)
        if c["labels"][r] >= 0:
            c["labels"][r] = at[r % K]  # one that the teacher holds
    return c


@pytest.mark.parametrize("value", [-1e4, -1e9, None], ids=["1e4", "1e9", "lowest"])
@pytest.mark.parametrize("ranks,logits,V", [(2, "bf16", 5003), (2, "f32", 27001), (4, "bf16", 8192),
                                            (4, "f32", 5003), (8, "f32", 50257), (8, "bf16", 9001)])
@pytest.mark.parametrize("where", ["first", "middle", "last", "all but the last"])
def test_masked_parts(ranks, logits, V, where, value):
    part = -(-V // ranks)
    r = {"first": 0, "middle": ranks // 2, "last": ranks - 1}.get(where, 0)
    lo, hi = r * part - 50, (r + 1) * part + 50
    if where == "all but the last":
        hi = V - part // 2
    c = masked(ROWS[ranks], V, 16, logits, value, lo, hi)
    check(c, 1.0)
    check(c, 2.0)


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0, 0.25, 1e-3])
@pytest.mark.parametrize("logits", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-3e9, -1e10, -1e30, -1e36, -1e38])
def test_large_masks(log_q, value, logits, tau):
    """Whole rows, the start of a row, every thread's first pieces, and all but one
    column at a mask of any size; in one block and over several."""
    for R, V in ((12, 5003), (100, 4097)):
        c = make(R, V, 8, logits=logits)
        c["weight"].fill_(1.0)
        c["s"][0].fill_(value)
        c["s"][1, :V // 2] = value
        c["s"][2, :-1] = value
        c["s"][3, 1:] = value
        c["s"][4, ::2] = value
        c["s"][5].fill_(-value)
        for r in range(1, 5):  # the teacher's entries and the label where the row lives
            c["ids"][r] = -1
            c["ids"][r, 0] = c["labels"][r] = [V - 3, V - 1, 0, 1][r - 1]
        check(c, tau)


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("exponent", [22, 23, 24, 25, 26, 28])
def test_differences_of_large_logits(log_q, exponent, tau):
    """Logits near 2^exponent whose differences are a few units of their last place."""
    for R, V in ((12, 1003), (100, 4097)):
        c = make(R, V, 8, logits="f32")
        step = 2.0 ** max(exponent - 23, 0)
        gen = torch.Generator(device="cuda").manual_seed(exponent)
        k = torch.randint(0, 24, (R, V), generator=gen, device="cuda").double()
        sign = 1.0 if exponent % 2 else -1.0
        c["s"].copy_((sign * (2.0 ** exponent + step * 32) + k * step).float())
        check(c, tau)


@pytest.mark.parametrize("value", [-1e9, 1e9, None], ids=["-1e9", "1e9", "lowest"])
@pytest.mark.parametrize("ranks,logits,V", [(2, "f32", 5003), (4, "bf16", 8192), (8, "f32", 9001)])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
def test_parts_without_live_entries(log_q, ranks, logits, V, value, tau):
    """The teacher's entries all in the masked part, or none; one live column in the
    part whose other columns are masked; a part far above the others."""
    part = -(-V // ranks)
    for r in {0, ranks // 2, ranks - 1}:
        lo, hi = max(0, r * part - 50), min(V, (r + 1) * part + 50)
        c = masked(ROWS[ranks], V, 4, logits, value, lo, hi)
        c["ids"][::3] = -1
        c["ids"][1::3] = torch.arange(lo, lo + 4, device="cuda")
        c["labels"][2::3] = lo + 1
        c["s"][2, (lo + hi) // 2] = 1.0
        check(c, tau)


@pytest.mark.parametrize("tau", [0.9, 0.5, 0.1, 1e-3])
@pytest.mark.parametrize("R,V,logits", [(12, 5003, "f32"), (100, 4097, "bf16"), (2, 400003, "f32")])
def test_lowest_value_at_the_teachers_entries(log_q, R, V, logits, tau):
    """A loss near the end of fp32's range: the lowest value at all of the teacher's
    entries, at one, and at an entry without a probability to speak of."""
    c = make(R, V, 8, logits=logits)
    c["weight"].fill_(1.0)
    low = torch.finfo(c["s"].dtype).min
    for r in range(R):
        c["ids"][r] = torch.arange(V - 8, V)
        at = {0: slice(V - 8, V), 1: slice(V - 8, V - 7)}.get(r % 3, slice(V - 1, V))
        c["s"][r, at] = low
        c["t"][r] = torch.linspace(0.0, -0.7 * tau, 8, device="cuda")
        if r % 3 == 2:
            c["t"][r, 7] = -1e4 * tau
        if c["labels"][r] >= V - 8:
            c["labels"][r] = 0
    check(c, tau)
