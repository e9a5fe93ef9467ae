"""Paths of the distillation that depend on a row's size and on the number of
rows: every kernel that the dispatch can choose, with a cluster, or a block,
that takes several rows one after the other.  References and bounds are those
of test_gpu_distill; of many rows a sample is compared, and the others with
the same rows on their own."""
import numpy as np
import pytest
import torch

from fsdp_sharded_optimizer_gb300 import _binding as B
from test_gpu_distill import U, check, half_ulp, make, n64, reference

pytestmark = pytest.mark.gpu


def lively(R, V, K, **kw):
    """make()'s case with repeated ids, labels among the teacher's entries (the
    first, the middle and the repeated one) and scattered rows of weight 0."""
    c = make(R, V, K, **kw)
    row = torch.arange(R, device="cuda")
    if K > 2:
        twice = row % 3 == 0
        c["ids"][twice, K // 2 - 1] = c["ids"][twice, 0]
    if c["labels"] is not None:
        for k, rest in ((0, 1), (K // 2 - 1, 2), (K // 4, 3)):
            on = (row % 5 == rest) & (c["ids"][:, k] >= 0)
            c["labels"][on] = c["ids"][on, k].to(c["labels"].dtype)
    c["weight"][(row * 7) % 11 == 3] = 0.0
    return c


def run(c, tau, cw=0.4, kw=0.6, rows=slice(None), out=None):
    s = c["s"][rows]
    R = s.shape[0]
    ce, kl = (torch.full((R,), float("nan"), device="cuda") for _ in range(2))
    g = torch.full_like(s, 7.0) if out is None else out
    lab = None if c["labels"] is None else c["labels"][rows]
    B.zero_distill_forward_backward(s, c["t"][rows], c["ids"][rows], ce, kl, g, labels=lab,
                                    row_weight=c["weight"][rows], temperature=tau, ce_weight=cw,
                                    kl_weight=kw)
    return ce, kl, g


def compare(c, got, tau, rows, cw=0.4, kw=0.6):
    ce, kl, g = (x[rows] for x in got)
    at = c["s"][rows], c["t"][rows], c["ids"][rows], c["weight"][rows]
    lab = None if c["labels"] is None else c["labels"][rows].cpu().numpy()
    ce0, kl0, g0, ct, kt, gt = reference(n64(at[0]), n64(at[1]), at[2].cpu().numpy(), lab, n64(at[3]),
                                         float(np.float32(tau)), float(np.float32(cw)),
                                         float(np.float32(kw)))
    assert np.all(np.abs(n64(ce) - ce0) <= ct)
    assert np.all(np.abs(n64(kl) - kl0) <= kt)
    tol = gt + (half_ulp(np.abs(g0) + gt) if g.dtype == torch.bfloat16 else 2 * U * np.abs(g0))
    off = np.abs(n64(g) - g0) - tol
    assert np.all(off <= 1e-36), off.max()


@pytest.mark.parametrize("R,V,logits", [(80, 32000, "bf16"), (80, 23001, "bf16"), (80, 36001, "bf16"),
                                        (80, 15000, "f32"), (80, 18001, "f32")])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0, 4.0])
def test_rows_of_43_to_72_kb(R, V, logits, tau):
    c = lively(R, V, 16, logits=logits)
    got = run(c, tau)
    compare(c, got, tau, torch.arange(0, R, 5, device="cuda"))


@pytest.mark.parametrize("R,V,K,kw", [
    (3000, 2049, 9, dict()), (3000, 2049, 9, dict(labels=False, logits="f32")),
    (2500, 4001, 300, dict(wide=True)),       # a block takes several rows
    (700, 32001, 24, dict(logits="f32")),     # 2 blocks to a row
    (700, 54001, 24, dict(teacher="bf16")),   # 2
    (500, 60002, 24, dict(logits="f32")),     # 4
    (400, 128256, 16, dict()), (400, 131075, 16, dict(offset=3)),  # 4
    (300, 256000, 16, dict()), (160, 120001, 16, dict(logits="f32"))])  # 8
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
def test_many_rows(R, V, K, kw, tau):
    c = lively(R, V, K, **kw)
    got = run(c, tau)
    n = max(8, min(R, 4000000 // V))
    rows = torch.unique(torch.cat([torch.arange(0, R, max(1, R // n), device="cuda"),
                                   torch.tensor([R - 1], device="cuda")]))
    compare(c, got, tau, rows)
    one, two = run(c, tau)[:2]
    assert torch.equal(one, got[0]) and torch.equal(two, got[1])
    again = c["s"].clone() if c["offset"] == 0 else c["s"]
    ce, kl, _ = run(dict(c, s=again), tau, out=again)  # in place
    assert torch.equal(again, got[2]) or c["offset"] % 8 != 0
    assert torch.equal(ce, got[0]) and torch.equal(kl, got[1])


@pytest.mark.parametrize("V,logits", [(800003, "bf16"), (400003, "f32")])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
def test_rows_that_no_cluster_holds(V, logits, tau):
    """Read twice, by one block; masked stretches, a repeated id, in place."""
    for offset in (0, 1):
        c = lively(4, V, 16, logits=logits, offset=offset)
        c["weight"].fill_(1.0)
        c["weight"][2] = 0.0
        c["s"][1, :V // 2] = -1e30
        c["ids"][1] = -1
        c["ids"][1, :2] = c["labels"][1] = V - 1
        c["s"][3].fill_(-1e9)
        check(c, tau)
    keep = c["s"].clone()
    first = run(c, tau)
    inside = run(c, tau, out=c["s"])
    assert torch.equal(inside[2], first[2]) and torch.equal(inside[1], first[1])
    c["s"].copy_(keep)


@pytest.mark.parametrize("V,logits", [(785001, "bf16"), (392001, "f32")])
def test_the_largest_rows_of_a_cluster(V, logits):
    """Parts of almost 192 KB on 8 blocks, with as many entries as there may be."""
    check(lively(2, V, 1024, logits=logits), 1.5)
