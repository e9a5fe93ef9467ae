"""The block norms' gradient with an eps far below the rows' squares: rows of
zeros have a gradient of finite size, and spoil no sum over the rows."""
import pytest
import torch

from test_gpu_block_norm import Case, backward64, close, run_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 131, 4096, 5000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows", [1, 5, 12])
def test_small_eps(rows, kind, dim):
    c = Case(rows, dim, kind=kind, bias=kind == "layer", act="f32", res="f32")
    c.eps = 1e-30
    want = backward64(c)
    for name, (_, t) in run_backward(c, torch.float32, want).items():
        close(t, *want[name], t.dtype, name)
    if rows == 12:  # the same with a row of zeros, whose own gradient is its du * w / sqrt(eps)
        c.x[7].zero_()
        c.h[3].zero_()
        c.du[7].mul_(1e-15)
        c.dy[3].mul_(1e-15)
        c.du[3].mul_(1e-15)
        want = backward64(c)
        for name, (_, t) in run_backward(c, torch.float32, want).items():
            close(t, *want[name], t.dtype, name)
