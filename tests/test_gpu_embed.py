"""zero_embed_forward and zero_embed_backward against plain fp64 forms.

The lookup is one fp32 product and one rounding per element, so it has to be
equal bit for bit.  A row's gradient is an fp32 sum of n rows of dout in some
order, times the scale: each addition rounds once, so with u = 2^-24 its error
is at most (n + 2) u scale sum|dout|, plus half an ulp of bf16 where the
result is rounded to it.
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


def place(rows, cols, dtype, offset, fill=None):
    """A rows x cols tensor that starts `offset` elements into its buffer, with
    guard elements on both sides."""
    buf = torch.full((offset + rows * cols + 64,), 7.0, dtype=dtype, device="cuda")
    t = buf[offset:offset + rows * cols].view(rows, cols)
    if fill is not None:
        t.copy_(fill)
    return buf, t


def guards_intact(buf, offset, n):
    return bool((buf[:offset] == 7).all()) and bool((buf[offset + n:] == 7).all())


def make_ids(rng, n, vocab, how):
    if how == "one":
        ids = np.full(n, vocab // 2)
    elif how == "zipf":
        ids = np.minimum((1.0 / np.maximum(rng.random(n), 1e-6)).astype(np.int64) - 1, vocab - 1)
    elif how == "outside":
        ids = rng.integers(-3, vocab + 3, n)
        ids[rng.random(n) < 0.1] = -(2 ** 31)
    elif how == "none":
        ids = np.full(n, -1)
    else:
        ids = rng.integers(0, vocab, n)
    return ids


@pytest.mark.parametrize("n,vocab,dim,table,out,offset,how,wide", [
    (1, 50257, 768, "bf16", "bf16", 0, "uniform", True),
    (0, 10, 8, "bf16", "bf16", 0, "uniform", True),
    (1000, 777, 64, "bf16", "f32", 0, "outside", False),
    (333, 101, 771, "bf16", "bf16", 0, "zipf", True),
    (257, 1, 8, "f32", "bf16", 0, "outside", True),
    (65, 4000, 128, "f32", "f32", 3, "uniform", False),
    (65, 4000, 136, "bf16", "bf16", 1, "zipf", False),
    (513, 32000, 4096, "bf16", "bf16", 8, "zipf", True),
    (3, 5, 1, "f32", "f32", 0, "uniform", True)])
def test_lookup_is_exact(n, vocab, dim, table, out, offset, how, wide):
    rng = np.random.default_rng(n + dim)
    ids = make_ids(rng, n, vocab, how)
    w = torch.from_numpy(rng.standard_normal((vocab, dim)).astype(np.float32))
    _, t = place(vocab, dim, TYPES[table], offset, w)
    buf, o = place(n, dim, TYPES[out], offset)
    idt = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    B.zero_embed_forward(t, idt, o, scale=0.3)
    want = torch.zeros((n, dim), dtype=torch.float32)
    ok = (ids >= 0) & (ids < vocab)
    rows = t.cpu().float().numpy()[np.where(ok, ids, 0)] * np.float32(0.3)
    want = torch.from_numpy(np.where(ok[:, None], rows, np.float32(0)))
    assert torch.equal(o.cpu(), want.to(TYPES[out]))
    assert guards_intact(buf, offset, n * dim)


@pytest.mark.parametrize("n,vocab,dim,dout,grad,offset,how,wide", [
    (1, 50257, 768, "bf16", "bf16", 0, "uniform", True),
    (0, 300, 24, "bf16", "bf16", 0, "uniform", True),
    (31, 200, 40, "f32", "f32", 0, "uniform", False),
    (33, 3, 8, "bf16", "f32", 0, "uniform", True),
    (5000, 1000, 64, "bf16", "bf16", 0, "one", True),
    (4097, 4001, 96, "bf16", "f32", 0, "zipf", False),
    (4096, 50257, 768, "bf16", "bf16", 0, "zipf", True),
    (1500, 170, 771, "bf16", "bf16", 0, "zipf", True),
    (1500, 170, 72, "f32", "bf16", 1, "outside", True),
    (700, 33, 5, "bf16", "f32", 3, "outside", False),
    (64, 100, 16, "bf16", "bf16", 0, "none", True),
    (2048, 200000, 16, "bf16", "bf16", 0, "uniform", True),
    (20000, 160, 264, "f32", "f32", 0, "zipf", True)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_by_sorted_tokens(n, vocab, dim, dout, grad, offset, how, wide, accumulate):
    rng = np.random.default_rng(n + dim + vocab)
    ids = make_ids(rng, n, vocab, how)
    scale = 0.7
    _, d = place(n, dim, TYPES[dout], offset,
                 torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)))
    d_in = d.cpu().double().numpy()
    if n and ((ids < 0) | (ids >= vocab)).any():  # rows that must not be read
        d[torch.from_numpy((ids < 0) | (ids >= vocab)).cuda()] = float("nan")
    start = torch.from_numpy(rng.standard_normal((vocab, dim)).astype(np.float32)).to(TYPES[grad])
    buf, g = place(vocab, dim, TYPES[grad], offset, start)
    if not accumulate:
        g.fill_(float("nan"))
    idt = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    scratch = torch.full((B.zero_embed_scratch_bytes(n, vocab, dim),), 255, dtype=torch.uint8,
                         device="cuda")
    B.zero_embed_backward(d, idt, g, scratch, scale=scale, accumulate=accumulate)
    first = g.clone()
    ok = (ids >= 0) & (ids < vocab)
    want, mass = np.zeros((vocab, dim)), np.zeros((vocab, dim))
    np.add.at(want, ids[ok], d_in[ok])
    np.add.at(mass, ids[ok], np.abs(d_in[ok]))
    count = np.bincount(ids[ok], minlength=vocab)[:, None]
    s = float(np.float32(scale))
    want, mass = want * s, mass * s
    if accumulate:
        want = want + start.double().numpy()
        mass = mass + np.abs(start.double().numpy())
    tol = (count + 3) * U * mass
    if grad == "bf16":
        tol = tol + half_ulp(np.abs(want) + tol)
    got = g.cpu().double().numpy()
    assert np.all(np.abs(got - want) <= tol * (1 + 1e-6))
    if accumulate:  # rows without tokens are not touched
        assert torch.equal(g.cpu()[count[:, 0] == 0], start[count[:, 0] == 0])
    assert guards_intact(buf, offset, vocab * dim)
    # the same bits again
    g.copy_(start)
    B.zero_embed_backward(d, idt, g, scratch, scale=scale, accumulate=accumulate)
    assert torch.equal(first.view(torch.int16 if grad == "bf16" else torch.int32),
                       g.view(torch.int16 if grad == "bf16" else torch.int32))


def test_gradient_agrees_with_differences():
    """The table's gradient of sum(out * c) along a random direction against the
    difference of the lookup, which is linear: equal up to fp32 rounding."""
    rng = np.random.default_rng(5)
    n, V, D = 200, 37, 48
    ids = torch.from_numpy(rng.integers(0, V, n)).cuda()
    c = torch.randn(n, D, device="cuda")
    w = torch.randn(V, D, device="cuda")
    direction = torch.randn(V, D, device="cuda")
    out = [torch.empty(n, D, device="cuda") for _ in range(2)]
    B.zero_embed_forward(w + direction, ids, out[0], scale=2.0)
    B.zero_embed_forward(w - direction, ids, out[1], scale=2.0)
    difference = float(((out[0].double() - out[1].double()) * c.double()).sum() / 2)
    g = torch.empty(V, D, device="cuda")
    scratch = torch.empty(B.zero_embed_scratch_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    B.zero_embed_backward(c, ids, g, scratch, scale=2.0)
    along = float((g.double() * direction.double()).sum())
    mass = float((c.double().abs() * 2 * 4).sum())  # |w +- direction| rarely above 4
    assert abs(along - difference) <= 40 * U * mass


def test_other_stream():
    """Inputs made on one stream, the call on another that waits for it."""
    V, D, n = 1000, 256, 4096
    side = torch.cuda.Stream()
    ids = torch.randint(0, V, (n,), device="cuda")
    d = torch.randn(n, D, device="cuda").bfloat16()
    g = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(B.zero_embed_scratch_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    B.zero_embed_backward(d, ids, g, scratch, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    again = torch.empty_like(g)
    B.zero_embed_backward(d, ids, again, scratch)
    assert torch.equal(g, again)
