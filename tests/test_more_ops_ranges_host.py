"""Numbers that a field of the C structures cannot hold are refused: ctypes would keep their lowest
bits and the call would answer for another start, distance or number of groups."""
import pytest
import torch

from test_more_ops_host import B, P  # noqa: F401  (B is a fixture)


class Device:
    """A contiguous tensor of a shape in device memory."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.nbytes = shape, dtype, 1 << 30

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


class NoStream:
    cuda_stream = 0


@pytest.fixture
def calls(B, monkeypatch):  # noqa: F811
    made = []
    for name in ("zero_relpos_forward", "zero_relpos_backward", "zero_group_norm_forward",
                 "zero_group_norm_scratch_bytes", "zero_relpos_scratch_bytes"):
        monkeypatch.setattr(B.lib, name, lambda *args, name=name: made.append(name) or 0)
    return made


def relpos(B, buckets=32, **kw):  # noqa: F811
    B.zero_relpos_forward(Device(buckets, 4), Device(2, 4, 5, 6), stream=NoStream(), **kw)


def relpos_grad(B, buckets=32, **kw):  # noqa: F811
    B.zero_relpos_backward(Device(2, 4, 5, 6), Device(buckets, 4), Device(1), stream=NoStream(), **kw)


def norm(B, **kw):  # noqa: F811
    B.zero_group_norm_forward(Device(2, 3, 64), Device(2, 3, 64), None, Device(1), stream=NoStream(), **kw)


def test_fits(B, calls):  # noqa: F811
    relpos(B, start=-(1 << 40), max_distance=8192)
    relpos_grad(B, start=1 << 40)
    norm(B, groups=8)
    B.zero_group_norm_scratch_bytes(1 << 30, 1 << 10, 64, 8)
    B.zero_relpos_scratch_bytes(1, 1, 8, 8, 32)
    assert len(calls) == 5


@pytest.mark.parametrize("call,kw", [
    (relpos, dict(start=(1 << 64) + 5)), (relpos, dict(start=-(1 << 63) - 1)),
    (relpos, dict(max_distance=(1 << 64) + 128)), (relpos, dict(buckets=(1 << 32) + 32)),
    (relpos_grad, dict(start=1 << 63)), (relpos_grad, dict(buckets=(1 << 32) + 32)),
    (norm, dict(groups=(1 << 32) + 8)), (norm, dict(groups=-(1 << 32) + 8)),
    (lambda B: B.zero_group_norm_scratch_bytes(2, 3, 64, (1 << 32) + 8), {}),
    (lambda B: B.zero_group_norm_scratch_bytes((1 << 64) + 2, 3, 64, 8), {}),
    (lambda B: B.zero_relpos_scratch_bytes(1, 1, 8, 8, (1 << 32) + 32), {}),
    (lambda B: B.zero_relpos_scratch_bytes(1, 1, (1 << 64) + 8, 8, 32), {})])
def test_refuses(B, calls, call, kw):  # noqa: F811
    with pytest.raises(ValueError):
        call(B, **kw)
    assert not calls


def test_stats_of_too_few_dimensions(B):  # noqa: F811
    with pytest.raises(ValueError):
        B.zero_group_norm_forward(Device(2, 3, 64), Device(2, 3, 64), Device(2), Device(1), stream=NoStream())
