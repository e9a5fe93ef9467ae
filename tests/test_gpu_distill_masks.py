"""Distillation where finite mask values stand in the logits: whole parts of a
row that is split over 2, 4 or 8 blocks.  References and bounds are those of
test_gpu_distill: the loss of a row does not depend on how far below the row's
maximum a masked logit without a teacher's entry lies."""
import pytest
import torch

from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu
ROWS = {2: 40, 4: 20, 8: 12}  # rows of which each is split over so many blocks


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
