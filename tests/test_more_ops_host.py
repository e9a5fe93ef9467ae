"""Refusals of the calls on tensor lists, group norm and relative position bias, on the
CPU: every bad argument is answered by an error code (or the binding's ValueError)
before anything is launched."""
import ctypes as C

import pytest
import torch

P = 1 << 20  # stands for an aligned device address; no call below gets to use it
EINVAL, EALIGN = -1, -2


@pytest.fixture(scope="module")
def B():
    from fsdp_sharded_optimizer_gb300 import build
    build.build()
    from fsdp_sharded_optimizer_gb300 import _binding
    return _binding


def entry(B, **kw):
    a = dict(src=P, dst=2 * P, n=100, src_type=2, dst_type=1)
    a.update(kw)
    return B.zero_tensor_t(**a)


BAD_TENSORS = [dict(src=None), dict(n=-1), dict(n=(1 << 40) + 1), dict(src_type=0), dict(src_type=3)]
BAD_PLACES = [dict(dst=None), dict(dst_type=0), dict(dst_type=4), dict(dst=P)]


def test_tensors_refuse(B):
    need = B.lib.zero_clip_scratch_bytes()

    def sqnorm(e=None, n=1, acc=0, scratch=P, bytes=need, null=False):
        arr = (B.zero_tensor_t * 1)(e if e is not None else entry(B))
        return B.lib.zero_tensors_sqnorm(None if null else arr, n, acc, scratch, bytes, None)

    def scale(e=None, n=1, by=1.0, nc=P, null=False):
        arr = (B.zero_tensor_t * 1)(e if e is not None else entry(B))
        return B.lib.zero_tensors_scale(None if null else arr, n, by, nc, None)

    def clip(e=None, n=1, max_norm=1.0, nc=P, scratch=P, bytes=need, null=False):
        arr = (B.zero_tensor_t * 1)(e if e is not None else entry(B))
        return B.lib.zero_tensors_clip(None if null else arr, n, max_norm, nc, scratch, bytes, None)

    for call in (sqnorm, scale, clip):
        for kw in BAD_TENSORS + (BAD_PLACES if call is not sqnorm else []):
            assert call(entry(B, **kw)) == EINVAL, kw
        assert call(n=-1) == EINVAL and call(n=(1 << 30) + 1) == EINVAL and call(null=True) == EINVAL
        assert call(entry(B, src=P + 2)) == EALIGN
        if call is not sqnorm:
            assert call(entry(B, dst=2 * P + 1)) == EALIGN
    assert sqnorm(acc=2) == EINVAL and sqnorm(scratch=None) == EINVAL
    assert sqnorm(bytes=need - 1) == EINVAL and sqnorm(scratch=P + 8) == EALIGN
    for by in (float("nan"), float("inf"), 1e39):
        assert scale(by=by) == EINVAL
    assert scale(nc=P + 8) == EALIGN
    assert B.lib.zero_tensors_scale(None, 0, 1.0, None, None) == 0  # nothing to do
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert clip(max_norm=bad) == EINVAL
    assert clip(nc=None) == EINVAL and clip(scratch=None) == EINVAL and clip(bytes=8) == EINVAL
    assert clip(nc=P + 4) == EALIGN and clip(scratch=P + 8) == EALIGN


def norm(B, **kw):
    a = dict(samples=2, positions=10, channels=64, x_stride=64, y_stride=64, groups=8, type=1,
             param_type=1, grad_type=1, act=1, eps=1e-5)
    a.update(kw)
    return B.zero_group_norm_t(**a)


BAD_NORMS = [dict(samples=-1), dict(positions=-1), dict(channels=0), dict(groups=0), dict(groups=7),
             dict(channels=16392, x_stride=1 << 15, y_stride=1 << 15), dict(x_stride=63),
             dict(y_stride=63), dict(type=0), dict(type=3), dict(param_type=4), dict(act=3),
             dict(act=-1), dict(samples=(1 << 30) + 1), dict(samples=1 << 25, positions=1 << 20),
             dict(samples=1 << 29)]


def test_group_norm_refuses(B):
    need = B.lib.zero_group_norm_scratch_bytes(2, 10, 64, 8)
    assert need > 0
    for bad in ((-1, 10, 64, 8), (2, -1, 64, 8), (2, 10, 0, 8), (2, 10, 64, 0), (2, 10, 64, 5)):
        assert B.lib.zero_group_norm_scratch_bytes(*bad) == EINVAL
    big = 1 << 60

    def forward(x=P, w=P, b=P, lengths=P, y=2 * P, stats=P, scratch=P, bytes=big, **kw):
        return B.lib.zero_group_norm_forward(C.byref(norm(B, **kw)), x, w, b, lengths, y, stats,
                                             scratch, bytes, None)

    def backward(x=P, dy=P, w=P, b=P, lengths=P, stats=P, dx=2 * P, dw=P, db=P, scratch=P,
                 bytes=big, **kw):
        return B.lib.zero_group_norm_backward(C.byref(norm(B, **kw)), x, dy, w, b, lengths, stats,
                                              dx, dw, db, scratch, bytes, None)

    for call in (forward, backward):
        for kw in BAD_NORMS:
            assert call(**kw) == EINVAL, kw
        for kw in (dict(x=None), dict(scratch=None), dict(bytes=need - 1)):
            assert call(**kw) == EINVAL, kw
        for kw in (dict(x=P + 1), dict(w=P + 1), dict(b=P + 1), dict(lengths=P + 2),
                   dict(stats=P + 4), dict(scratch=P + 8)):
            assert call(**kw) == EALIGN, kw
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-60),
               dict(y=None), dict(y=P, y_stride=72)):
        assert forward(**kw) == EINVAL, kw
    assert forward(y=P + 1) == EALIGN
    assert forward(samples=0, x=None, y=None) == 0
    for kw in (dict(dy=None), dict(stats=None), dict(grad_type=0), dict(dy=2 * P, y_stride=72)):
        assert backward(**kw) == EINVAL, kw
    for kw in (dict(dy=P + 1), dict(dx=P + 1), dict(dw=P + 1), dict(db=P + 1)):
        assert backward(**kw) == EALIGN, kw
    assert B.lib.zero_group_norm_forward(None, P, P, P, P, P, P, P, big, None) == EINVAL
    assert B.lib.zero_group_norm_backward(None, P, P, P, P, P, P, P, P, P, P, big, None) == EINVAL


def relpos(B, **kw):
    a = dict(batch=2, heads=4, q_len=10, k_len=12, start=2, max_distance=128, buckets=32,
             bidirectional=1, causal=0, table_type=1, type=1)
    a.update(kw)
    return B.zero_relpos_t(**a)


BAD_RELPOS = [dict(batch=-1), dict(heads=0), dict(heads=65536), dict(q_len=-1), dict(k_len=-1),
              dict(q_len=(1 << 24) + 1), dict(k_len=(1 << 24) + 1), dict(start=(1 << 40) + 1),
              dict(start=-(1 << 40) - 1), dict(max_distance=8), dict(max_distance=8193),
              dict(max_distance=16, bidirectional=0), dict(buckets=1, bidirectional=0),
              dict(buckets=2), dict(buckets=33), dict(buckets=514), dict(bidirectional=2),
              dict(causal=-1), dict(table_type=0), dict(type=4), dict(batch=1 << 30)]


def test_relpos_refuses(B):
    need = B.lib.zero_relpos_scratch_bytes(2, 4, 10, 12, 32)
    assert need > 0
    for bad in ((-1, 4, 10, 12, 32), (2, 0, 10, 12, 32), (2, 4, -1, 12, 32), (2, 4, 10, 12, 513)):
        assert B.lib.zero_relpos_scratch_bytes(*bad) == EINVAL

    def forward(table=P, starts=P, ql=P, kl=P, s=P, ss=12, out=2 * P, os=12, **kw):
        return B.lib.zero_relpos_forward(C.byref(relpos(B, **kw)), table, starts, ql, kl, s, ss,
                                         out, os, None)

    def backward(starts=P, ql=P, kl=P, dout=P, ds=12, dtable=P, acc=0, scratch=P, bytes=1 << 60,
                 **kw):
        return B.lib.zero_relpos_backward(C.byref(relpos(B, **kw)), starts, ql, kl, dout, ds,
                                          dtable, acc, scratch, bytes, None)

    for call in (forward, backward):
        for kw in BAD_RELPOS:
            assert call(**kw) == EINVAL, kw
        for kw in (dict(starts=P + 2), dict(ql=P + 1), dict(kl=P + 2)):
            assert call(**kw) == EALIGN, kw
    for kw in (dict(table=None), dict(out=None), dict(os=11), dict(ss=11), dict(os=(1 << 30) + 1),
               dict(out=P, os=13)):
        assert forward(**kw) == EINVAL, kw
    for kw in (dict(table=P + 1), dict(s=P + 1), dict(out=P + 1)):
        assert forward(**kw) == EALIGN, kw
    assert forward(batch=0, table=None, out=None) == 0
    for kw in (dict(dout=None), dict(ds=11), dict(dtable=None), dict(scratch=None),
               dict(bytes=need - 1), dict(acc=2)):
        assert backward(**kw) == EINVAL, kw
    for kw in (dict(dout=P + 1), dict(dtable=P + 1), dict(scratch=P + 8)):
        assert backward(**kw) == EALIGN, kw
    assert backward(q_len=0, acc=1, dout=None) == 0
    assert B.lib.zero_relpos_forward(None, P, P, P, P, P, 12, P, 12, None) == EINVAL
    assert B.lib.zero_relpos_backward(None, P, P, P, P, 12, P, 0, P, 1 << 60, None) == EINVAL


def test_binding_checks_shapes_and_types(B):
    """Shapes and types are the binding's to check: the C call sees sizes only."""
    f = torch.zeros
    i = lambda n: f(n, dtype=torch.int32)
    for call in (
            lambda: B.zero_tensor_list([f(4)], [f(4), f(4)]),
            lambda: B.zero_tensor_list([f(4)], [f(5)]),
            lambda: B.zero_tensor_list([f(4)]),                      # pageable memory
            lambda: B.zero_tensors_clip([], 1.0, f(1), f(9728)),
            lambda: B.zero_group_norm_forward(f(8), f(8), None, f(1), groups=2),
            lambda: B.zero_group_norm_forward(f(2, 3, 8), f(2, 3, 8), None, f(1)),
            lambda: B.zero_group_norm_forward(f(2, 3, 8), f(2, 3, 8), None, f(1), groups=2,
                                              act="relu"),
            lambda: B.zero_group_norm_forward(f(2, 3, 8), f(2, 3, 8), f(2, 2, 3), f(1)),
            lambda: B.zero_relpos_forward(f(32, 4), f(1, 3, 5, 5)),
            lambda: B.zero_relpos_forward(f(32, 4), f(4, 5, 5)),
            lambda: B.zero_relpos_forward(f(32, 4), f(1, 4, 5, 5), starts=f(1)),
            lambda: B.zero_relpos_forward(f(32, 4), f(1, 4, 5, 5), q_lengths=i(2)),
            lambda: B.zero_relpos_backward(f(1, 4, 5, 5), f(32, 4).double(), f(1)),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.ZeroError):
        B.zero_group_norm_scratch_bytes(1, 1, 8, 3)
    with pytest.raises(B.ZeroError):
        B.zero_relpos_scratch_bytes(1, 1, 8, 3, 1)


class Fake:
    """A tensor of a given place in device memory."""

    def __init__(self, at, n, dtype=torch.float32):
        self.at, self.n, self.dtype = at, n, dtype
        self.is_cuda, self.shape = True, (n,)
        self.nbytes = n * torch.empty(0, dtype=dtype).element_size()

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def test_tensor_list_refuses_overlaps(B):
    a, b = Fake(P, 100), Fake(P + 400, 100)
    assert B.zero_tensor_list([a, b]).n == 2
    assert B.zero_tensor_list([a, a], [Fake(2 * P, 100), Fake(3 * P, 100)]).n == 2
    assert B.zero_tensor_list([a, b], [Fake(2 * P, 100), Fake(2 * P + 400, 100)]).n == 2
    assert B.zero_tensor_list([a, Fake(P + 40, 0)]).n == 2
    for src, dst in (([a, a], None), ([a, Fake(P + 396, 5)], None), ([a], [Fake(P + 4, 100)]),
                     ([a, b], [b, a]), ([a, b], [Fake(2 * P, 100), Fake(2 * P + 396, 100)]),
                     ([a, b], [a, Fake(P + 396, 100)]), ([a], [Fake(P, 100, torch.bfloat16)])):
        with pytest.raises(ValueError):
            B.zero_tensor_list(src, dst)
