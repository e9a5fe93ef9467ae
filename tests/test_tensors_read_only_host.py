"""zero_tensors_sqnorm only reads: its list may hold a tensor twice, or views that overlap."""
import pytest
import torch

from test_more_ops_host import B, P, Fake  # noqa: F401  (B is a fixture)


class NoStream:
    cuda_stream = 0


def test_norm_of_tensors_that_overlap(B, monkeypatch):  # noqa: F811
    a, b, empty = Fake(P, 100), Fake(P + 40, 30, torch.bfloat16), Fake(P, 0)
    calls = []
    monkeypatch.setattr(B.lib, "zero_tensors_sqnorm", lambda *args: calls.append(args) or 0)
    scratch = Fake(2 * P, B.lib.zero_clip_scratch_bytes(), torch.uint8)
    B.zero_tensors_sqnorm((t for t in (a, a, b, empty)), scratch, stream=NoStream())
    (array, n, accumulate, *_), = calls
    assert n == 4 and accumulate == 0
    assert [(e.src, e.dst, e.n, e.src_type) for e in array] == [
        (P, None, 100, B.ZERO_TYPE_F32), (P, None, 100, B.ZERO_TYPE_F32),
        (P + 40, None, 30, B.ZERO_TYPE_BF16), (P, None, 0, B.ZERO_TYPE_F32)]
    kept = B.zero_tensor_list([a], [Fake(3 * P, 100)])
    B.zero_tensors_sqnorm(kept, scratch, accumulate=True, stream=NoStream())
    assert calls[1][0] is kept.array and calls[1][2] == 1


def test_refusals_stay(B):  # noqa: F811
    scratch = Fake(2 * P, 9728, torch.uint8)
    for bad in ([torch.zeros(4)], [Fake(P, 4, torch.float64)]):
        with pytest.raises(ValueError):
            B.zero_tensors_sqnorm(bad, scratch, stream=NoStream())
    with pytest.raises(ValueError):  # a call that writes takes no tensor twice
        B.zero_tensors_scale([Fake(P, 4), Fake(P, 4)], stream=NoStream())
