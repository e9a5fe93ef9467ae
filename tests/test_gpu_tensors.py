"""zero_tensors_sqnorm, zero_tensors_scale and zero_tensors_clip against fp64.

Bounds, with u = 2^-24: a square passes 11 roundings at most on its way into the
fp64 sum (its own or the fused product's, two of the pairwise sum, eight of the
thread's sum), so the squared norm is right to 11 u relative, the norm to 5.5 u, and
norm and coef, rounded to fp32, to 6.5 u.  dst adds the product's rounding (and
half an ulp of bf16): 8 u covers it.
"""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_ulp(x):
    """Half a unit in the last of bf16's 8 significant bits at |x|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def scratch():
    return torch.full((Z.zero_clip_scratch_bytes(),), 255, dtype=torch.uint8, device="cuda")


def tensors(sizes, dtype, seed=0, offset=0, sigma=1e-2):
    """Tensors of the sizes, each `offset` elements behind a 16-byte boundary."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.empty(n + offset, dtype=dtype, device="cuda")[offset:]
        t.copy_(torch.randn(n, generator=gen, device="cuda") * (sigma * (1 + i % 5)))
        out.append(t)
    return out


def norm64(src):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in src))


def close(got, want, dtype, what):
    tol = 8 * U * np.abs(want) + 2.0 ** -149
    if dtype == torch.bfloat16:
        tol = tol + half_ulp(np.abs(want) + tol)
    got = got.detach().cpu().double().numpy()
    assert np.all(np.abs(got - want) <= tol), what


SIZES = [
    [1], [3], [8], [2047], [16384], [16385], [5, 0, 7], [0], [],
    [768] * 40 + [100003, 1, 65536, 9], [1 << 20, 77], [16384 * 1300 + 5],
]


@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("offsets", [(0, 0), (1, 0), (0, 3), (5, 2), (4, 4)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), sum(s)))
def test_clip(sizes, offsets, src, dst):
    if sum(sizes) > 1 << 22 and offsets[0] != offsets[1]:
        pytest.skip("the large list once aligned and once not")
    a = tensors(sizes, TYPES[src], 1, offsets[0])
    total = sum(sizes)
    flat = torch.full((total + offsets[1] + 9,), 7.0, dtype=TYPES[dst], device="cuda")
    places = list(flat[offsets[1]:offsets[1] + total].split(sizes)) if sizes else []
    before = [t.clone() for t in a]
    norm = norm64(a)
    for max_norm in (0.25 * norm + 1e-3, 4 * norm + 1.0):
        nc = torch.full((4,), -1.0, device="cuda")
        Z.zero_tensors_clip(Z.zero_tensor_list(a, places), max_norm, nc, scratch())
        coef = min(1.0, max_norm / (norm + 1e-6))
        got = nc.cpu().double().numpy()
        assert abs(got[0] - norm) <= 6.5 * U * norm and abs(got[1] - coef) <= 6.5 * U * coef
        assert got[2] == -1.0
        if coef == 1.0:
            assert got[1] == 1.0
        for x, y in zip(a, places):
            close(y, x.double().cpu().numpy() * coef, TYPES[dst], "dst")
        assert torch.all(flat[:offsets[1]] == 7) and torch.all(flat[offsets[1] + total:] == 7)
    for x, y in zip(a, before):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_three_calls_give_the_same_bits(dtype):
    sizes = [1000, 1, 33333, 16384 * 3, 12]
    a = tensors(sizes, TYPES[dtype], 2, 1)
    out = [torch.empty_like(t) for t in a]
    nc, s = torch.empty(2, device="cuda"), scratch()
    Z.zero_tensors_clip(Z.zero_tensor_list(a, out), 0.5, nc, s)
    nc3, s3 = torch.empty(2, device="cuda"), scratch()
    half = len(a) // 2
    Z.zero_tensors_sqnorm(a, s3)
    Z.zero_clip_coef(s3, 0.5, nc3)
    assert torch.equal(nc, nc3)
    # in two parts: the same partials added up in another order, so the same to fp64
    Z.zero_tensors_sqnorm(a[:half], s3)
    Z.zero_tensors_sqnorm(a[half:], s3, accumulate=True)
    Z.zero_clip_coef(s3, 0.5, nc3)
    assert torch.allclose(nc, nc3, rtol=1e-6, atol=0)
    again = [t.clone() for t in a]
    Z.zero_tensors_scale(again, norm_coef=nc)
    in_place = [t.clone() for t in a]
    Z.zero_tensors_clip(in_place, 0.5, nc3, s3)
    for w, x, y in zip(out, again, in_place):
        assert torch.equal(w, x) and torch.equal(w, y)
    # nothing to clip: nothing changes, NaN payloads and all
    quiet = [t.clone() for t in a]
    Z.zero_tensors_clip(quiet, 1e9, nc3, s3)
    for x, y in zip(quiet, a):
        assert torch.equal(x, y)
    assert float(nc3[1]) == 1.0


def test_adds_to_the_flat_buffers_norm():
    """The partials are zero_grad_sqnorm's: a flat buffer and loose tensors under one norm."""
    flat = tensors([4096], torch.bfloat16, 3)[0].view(1, 4096)
    loose = tensors([100, 7], torch.float32, 4)
    s, nc = scratch(), torch.empty(2, device="cuda")
    Z.zero_grad_sqnorm(flat, s)
    Z.zero_tensors_sqnorm(loose, s, accumulate=True)
    Z.zero_clip_coef(s, 1.0, nc)
    assert abs(float(nc[0]) / norm64([flat, *loose]) - 1) <= 8 * U


def test_more_tensors_than_a_launch_takes():
    sizes = [(i * 37) % 200 for i in range(2345)]
    a = tensors(sizes, torch.float32, 5)
    flat = torch.zeros(sum(sizes), dtype=torch.bfloat16, device="cuda")
    nc = torch.empty(2, device="cuda")
    Z.zero_tensors_clip(Z.zero_tensor_list(a, list(flat.split(sizes))), 0.1, nc, scratch())
    norm = norm64(a)
    assert abs(float(nc[0]) - norm) <= 6.5 * U * norm
    close(flat, torch.cat(a).double().cpu().numpy() * 0.1 / (norm + 1e-6), torch.bfloat16, "flat")
    # the same tensor twice counts twice in the norm
    s = scratch()
    Z.zero_tensors_sqnorm(Z.zero_tensor_list([a[1], a[1]], [torch.empty_like(a[1]) for _ in "ab"]), s)
    Z.zero_clip_coef(s, 1.0, nc)
    assert abs(float(nc[0]) / (math.sqrt(2) * norm64([a[1]])) - 1) <= 6.5 * U


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e15, 3e25, 1e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norms_beyond_the_squares_range(dtype, scale):
    """Squares that fp32 cannot hold: the norm is right all the same."""
    a = tensors([3000, 16384 * 2 + 3, 5], TYPES[dtype], 6, 1, sigma=1.0)
    for t in a:
        t.copy_((t.double() * (scale / 64)).to(t.dtype))
    nc = torch.empty(2, device="cuda")
    out = [torch.empty_like(t) for t in a]
    Z.zero_tensors_clip(Z.zero_tensor_list(a, out), 1.0, nc, scratch())
    norm = norm64(a)
    if norm > 3.4e38:
        assert math.isinf(float(nc[0]))
    else:
        # below fp32's normal numbers its last place is 2^-149
        assert abs(float(nc[0]) - norm) <= 6.5 * U * norm + 2.0 ** -149
    coef = min(1.0, 1.0 / (norm + 1e-6))
    for x, y in zip(a, out):
        # coef below fp32's normal numbers is off by half its last place
        want = x.double().cpu().numpy() * coef
        tol = 8 * U * np.abs(want) + 2.0 ** -149 + np.abs(x.double().cpu().numpy()) * 2.0 ** -149
        tol = tol + (half_ulp(np.abs(want) + tol) if y.dtype == torch.bfloat16 else 0)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


def test_mixed_magnitudes_and_zeros():
    """Rows of zeros beside gradients of every size (an embedding table's gradient)."""
    t = torch.zeros(64 * 4096, device="cuda")
    t[::4096] = torch.logspace(-30, 15, 64, device="cuda")
    t[7::1024] = 1e-24
    nc, s = torch.empty(2, device="cuda"), scratch()
    for part in (t, t[:4096 * 20]):
        Z.zero_tensors_clip([part.clone()], 1.0, nc, s)
        norm = norm64([part])
        assert abs(float(nc[0]) - norm) <= 6.5 * U * norm


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(bad):
    a = tensors([1000, 50000], torch.float32, 7)
    a[1][777] = bad
    out = [torch.empty_like(t) for t in a]
    nc = torch.empty(2, device="cuda")
    Z.zero_tensors_clip(Z.zero_tensor_list(a, out), 1.0, nc, scratch())
    if math.isnan(bad):
        assert torch.isnan(nc).all() and all(torch.isnan(t).all() for t in out)
    else:
        assert math.isinf(float(nc[0])) and float(nc[1]) == 0.0
        assert torch.isnan(out[1][777]) and int(torch.count_nonzero(out[0])) == 0


def test_scale_without_a_norm():
    a = tensors([1000, 77], torch.float32, 8)
    flat = torch.empty(1077, dtype=torch.bfloat16, device="cuda")
    Z.zero_tensors_scale(Z.zero_tensor_list(a, list(flat.split([1000, 77]))), scale=0.25)
    assert torch.equal(flat, (torch.cat(a) * 0.25).bfloat16())
    Z.zero_tensors_scale([], scale=2.0)
    Z.zero_tensors_scale(a, scale=2.0)
    assert torch.equal(flat, (torch.cat(a) * 0.125).bfloat16())


def test_captured_and_on_another_stream():
    a = tensors([1000, 70000], torch.bfloat16, 9)
    out = [torch.empty_like(t) for t in a]
    nc, s = torch.zeros(2, device="cuda"), scratch()
    tl = Z.zero_tensor_list(a, out)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        Z.zero_tensors_clip(tl, 0.5, nc, s)
    stream.synchronize()
    want, coef = [t.clone() for t in out], nc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_tensors_clip(tl, 0.5, nc, s)
    for k in range(3):
        for t in out:
            t.zero_()
        nc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(nc, coef) and all(torch.equal(x, y) for x, y in zip(out, want))
    a[0].mul_(2)  # a replay reads what the tensors hold now
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(nc[0]) - norm64(a)) <= 6.5 * U * norm64(a)


def test_past_2_31_elements():
    n = (1 << 31) + 12345
    t = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    t.fill_(0.0)
    t[:1000] = 3.0
    t[-1000:] = 4.0
    t[1 << 31] = 5.0
    nc = torch.empty(2, device="cuda")
    Z.zero_tensors_clip([t], 1.0, nc, scratch())
    norm = math.sqrt(9e3 + 16e3 + 25.0)
    assert abs(float(nc[0]) - norm) <= 6.5 * U * norm
    for at, v in ((0, 3.0), (n - 1, 4.0), (1 << 31, 5.0), (5000, 0.0)):
        want = v / (norm + 1e-6)
        assert abs(float(t[at]) - want) <= 8 * U * want + half_ulp(want)
