"""Lists as training has them: large and tiny tensors of both types at any alignment, above and
below the 1216 * 2048 elements where the passes go from chunks of 2,048 elements to 16,384.

Elements are whole numbers of -3 .. 3, whose squares have sums that fp32 (a thread's 64) and fp64 hold
exactly: the norm is the root of a whole number, so that one element that is lost or counted twice
shows; a scaled element is one fp32 product, rounded once.
"""
import math

import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
CHUNK, SMALL = 16384, 1216 * 2048


def whole(n, dtype, offset, gen):
    t = torch.empty(n + offset, dtype=dtype, device="cuda")[offset:]
    return t.copy_(torch.randint(-3, 4, (n,), generator=gen, device="cuda"))


def scratch():
    return torch.full((Z.zero_clip_scratch_bytes(),), 255, dtype=torch.uint8, device="cuda")


def squares(tensors):
    return sum(int((t.long() ** 2).sum()) for t in tensors)


def root(total):
    return float(torch.tensor(math.sqrt(total), dtype=torch.float64).float())


LISTS = {
    "ends at chunks": [CHUNK * 50 - 1, 3, CHUNK * 60, 1, CHUNK * 50 + 1, 7, CHUNK, CHUNK - 1, CHUNK + 1, 0, 2],
    "tiny between": [n for k in range(130) for n in (CHUNK + (k % 3) - 1, 1 + k % 9, CHUNK // 2 + k)],
    "one large": [5, SMALL + 11, 768, 768, 1],
    "just below": [SMALL - 1000, 999], "at the border": [SMALL - 1000, 1000], "just above": [SMALL - 1000, 1001],
    "many": [2500 + 13 * (k % 41) for k in range(1300)],
}


@pytest.mark.parametrize("src,dst", [((F,), (B,)), ((B,), (B,)), ((F,), (F,)), ((B, F), (B,)), ((F, B, B), (F, B))],
                         ids=["f32-bf16", "bf16-bf16", "f32-f32", "mixed-bf16", "mixed-mixed"])
@pytest.mark.parametrize("offsets", [(0, 0), (1, 0), (3, 5), (4, 4)])
@pytest.mark.parametrize("sizes", LISTS.values(), ids=LISTS.keys())
def test_clip(sizes, offsets, src, dst):
    gen = torch.Generator("cuda").manual_seed(len(sizes))
    a = [whole(n, src[i % len(src)], offsets[0], gen) for i, n in enumerate(sizes)]
    if len(dst) == 1:  # one flat gradient, places one after another
        flat = torch.full((offsets[1] + sum(sizes) + 8,), 7.0, dtype=dst[0], device="cuda")
        places = list(flat[offsets[1]:offsets[1] + sum(sizes)].split(sizes))
    else:
        places = [torch.full((n + offsets[1] + 8,), 7.0, dtype=dst[i % len(dst)], device="cuda")
                  [offsets[1]:offsets[1] + n] for i, n in enumerate(sizes)]
    norm = math.sqrt(squares(a))
    nc = torch.zeros(2, device="cuda")
    Z.zero_tensors_clip(Z.zero_tensor_list(a, places), 0.3 * norm, nc, scratch())
    coef = torch.tensor(0.3 * norm / (norm + 1e-6), dtype=torch.float64).float()
    assert float(nc[0]) == root(squares(a))
    assert abs(float(nc[1]) / float(coef) - 1) <= 2.0 ** -23  # one quotient in fp64, rounded to fp32
    for i, (x, y) in enumerate(zip(a, places)):
        assert torch.equal(y, (x.float() * nc[1]).to(y.dtype)), i
        ends = y.as_strided((8,), (1,), y.storage_offset() + y.numel())
        assert len(dst) == 1 or torch.all(ends == 7)
    if len(dst) == 1:
        assert torch.all(flat[:offsets[1]] == 7) and torch.all(flat[-8:] == 7)


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("sizes", LISTS.values(), ids=LISTS.keys())
def test_in_place(sizes, offset):
    gen = torch.Generator("cuda").manual_seed(len(sizes))
    a = [whole(n, (F, B)[i % 2], offset, gen) for i, n in enumerate(sizes)]
    before, nc = [t.clone() for t in a], torch.zeros(2, device="cuda")
    Z.zero_tensors_clip(a, 4.0, nc, scratch())
    assert float(nc[0]) == root(squares(before))
    for i, (x, y) in enumerate(zip(a, before)):
        assert torch.equal(x, (y.float() * nc[1]).to(x.dtype)), i


def test_norm_of_tensors_that_overlap():
    """A tensor that is listed twice counts twice; nothing is written."""
    a = whole(30000, F, 1, torch.Generator("cuda").manual_seed(1))
    b = whole(SMALL, B, 3, torch.Generator("cuda").manual_seed(2))
    lists = ([a, a], [a, a[100:20000], a[7:]], [b, a, b, b[1:]])
    for tensors in lists:
        s, nc = scratch(), torch.zeros(2, device="cuda")
        before = [t.clone() for t in tensors]
        Z.zero_tensors_sqnorm(tensors, s)
        Z.zero_clip_coef(s, 1.0, nc)
        assert float(nc[0]) == root(squares(tensors))
        assert all(torch.equal(x, y) for x, y in zip(tensors, before))
