"""Refusals of the model operators, on the CPU: every bad argument is answered by
an error code (or the binding's ValueError) before anything is launched."""
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


def test_embed_forward_refuses(B):
    good = dict(table=P, tt=1, V=100, D=8, ids=P, it=4, n=5, scale=1.0, out=P, ot=2)

    def call(**kw):
        a = dict(good, **kw)
        return B.lib.zero_embed_forward(a["table"], a["tt"], a["V"], a["D"], a["ids"], a["it"],
                                        a["n"], a["scale"], a["out"], a["ot"], None)

    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(tt=0), dict(tt=3),
               dict(ot=4), dict(it=1), dict(V=0), dict(D=0), dict(n=-1), dict(V=1 << 31),
               dict(n=(1 << 30) + 1)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(table=P + 1), dict(ids=P + 4), dict(out=P + 2)):
        assert call(**kw) == EALIGN, kw
    assert call(n=0, ids=None, out=None) == 0


def test_embed_backward_refuses(B):
    assert B.lib.zero_embed_scratch_bytes(-1, 10, 10) == EINVAL
    assert B.lib.zero_embed_scratch_bytes(10, 0, 10) == EINVAL
    need = B.lib.zero_embed_scratch_bytes(5, 100, 8)
    good = dict(dout=P, dt=1, ids=P, it=4, n=5, dtable=P, gt=1, V=100, D=8, acc=0, scratch=P,
                bytes=need)

    def call(**kw):
        a = dict(good, **kw)
        return B.lib.zero_embed_backward(a["dout"], a["dt"], a["ids"], a["it"], a["n"], 1.0,
                                         a["dtable"], a["gt"], a["V"], a["D"], a["acc"],
                                         a["scratch"], a["bytes"], None)

    for kw in (dict(dout=None), dict(ids=None), dict(dtable=None), dict(scratch=None),
               dict(bytes=need - 1), dict(dt=5), dict(gt=4), dict(it=2), dict(acc=2), dict(n=-1),
               dict(V=0), dict(D=(1 << 22) + 1), dict(D=(1 << 20) + 1)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dout=P + 1), dict(ids=P + 4), dict(dtable=P + 1), dict(scratch=P + 8)):
        assert call(**kw) == EALIGN, kw
    assert call(n=0, dout=None, ids=None, acc=1) == 0


def spec(B, **kw):
    a = dict(n_rows=4, dim=64, rows_per_gate=4, kind=0, post_norm=1, pre_norm=1, act_type=1,
             res_type=1, param_type=1, gate_type=1, eps=1e-6, residual_scale=1.0,
             branch_scale=1.0)
    a.update(kw)
    return B.zero_block_norm_t(**a)


BAD_SPECS = [dict(n_rows=-1), dict(dim=0), dict(dim=16385), dict(rows_per_gate=0), dict(kind=2),
             dict(post_norm=2), dict(pre_norm=-1), dict(act_type=0), dict(res_type=3),
             dict(param_type=4), dict(gate_type=0), dict(act_type=2, res_type=1), dict(eps=0.0),
             dict(eps=float("nan")), dict(eps=1e-60), dict(residual_scale=float("inf")),
             dict(branch_scale=float("nan"))]


def test_block_norm_forward_refuses(B):
    def call(s=None, x=P, branch=P, gate=P, pw=P, pb=P, qw=P, qb=P, y=P, u=P, **kw):
        s = s if s is not None else spec(B, **kw)
        return B.lib.zero_block_norm_forward(C.byref(s), x, branch, gate, pw, pb, qw, qb, y, u,
                                             None)

    for kw in BAD_SPECS:
        assert call(**kw) == EINVAL, kw
    assert B.lib.zero_block_norm_forward(None, P, P, P, P, P, P, P, P, P, None) == EINVAL
    for kw in (dict(x=None), dict(y=None), dict(u=None), dict(branch=None),
               dict(branch=None, y=None, gate=None), dict(pre_norm=0, qw=None, qb=None),
               dict(pre_norm=0, u=None), dict(post_norm=0),
               dict(branch=None, y=None, post_norm=0, pw=None, pb=None)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(x=P + 1), dict(branch=P + 1), dict(gate=P + 1), dict(pw=P + 1), dict(y=P + 1),
               dict(u=P + 1), dict(qb=P + 1)):
        assert call(**kw) == EALIGN, kw
    assert call(n_rows=0, x=None) == 0


def test_block_norm_backward_refuses(B):
    need = B.lib.zero_block_norm_scratch_bytes(4, 64, 4)
    assert need > 0 and B.lib.zero_block_norm_scratch_bytes(4, 0, 4) == EINVAL
    assert B.lib.zero_block_norm_scratch_bytes(4, 64, 0) == EINVAL

    def grads(**kw):
        a = dict(dgate=P, dpost_weight=P, dpost_bias=P, dpre_weight=P, dpre_bias=P, dgate_type=1,
                 grad_type=1)
        a.update(kw)
        return B.zero_block_norm_grads_t(**a)

    def call(g=None, dy=P, du=P, y=P, branch=P, gate=P, pw=P, pb=P, qw=P, dx=P, dh=P, scratch=P,
             bytes=need, **kw):
        s, g = spec(B, **kw), g or grads()
        return B.lib.zero_block_norm_backward(C.byref(s), dy, du, y, branch, gate, pw, pb, qw, dx,
                                              dh, C.byref(g), scratch, bytes, None)

    for kw in BAD_SPECS:
        assert call(**kw) == EINVAL, kw
    for kw in (dict(du=None), dict(y=None), dict(dh=None), dict(branch=None), dict(scratch=None),
               dict(bytes=need - 1), dict(gate=None), dict(pre_norm=0, du=None),
               dict(pre_norm=0, qw=None), dict(post_norm=0, pw=None, pb=None),
               dict(g=grads(grad_type=0)), dict(g=grads(dgate_type=3))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dy=P + 1), dict(du=P + 1), dict(dx=P + 1), dict(dh=P + 1),
               dict(scratch=P + 4), dict(g=grads(dgate=P + 1)),
               dict(g=grads(dpre_weight=P + 2, grad_type=2))):
        assert call(**kw) == EALIGN, kw


def test_distill_refuses(B):
    def call(grad=True, logits=P, t=P, ids=P, labels=P, w=P, ce=P, kl=P, dl=P, stride=100, s=None,
             **kw):
        a = dict(n_rows=4, vocab=100, logits_stride=100, top=5, logits_type=1, teacher_type=2,
                 id_type=3, label_type=4, temperature=1.0, ce_weight=0.5, kl_weight=0.5)
        a.update(kw)
        s = C.byref(B.zero_distill_t(**a))
        if grad:
            return B.lib.zero_distill_forward_backward(s, logits, t, ids, labels, w, ce, kl, dl,
                                                       stride, None)
        return B.lib.zero_distill_forward(s, logits, t, ids, labels, w, ce, kl, None)

    for grad in (False, True):
        for kw in (dict(n_rows=-1), dict(vocab=0), dict(vocab=1 << 31, logits_stride=1 << 32),
                   dict(logits_stride=99), dict(top=0), dict(top=1025), dict(logits_type=0),
                   dict(teacher_type=3), dict(id_type=2), dict(label_type=1),
                   dict(temperature=0.0), dict(temperature=float("nan")),
                   dict(temperature=1e4), dict(ce_weight=float("inf")), dict(logits=None),
                   dict(t=None), dict(ids=None), dict(ce=None), dict(kl=None)):
            assert call(grad, **kw) == EINVAL, kw
        for kw in (dict(logits=P + 1), dict(t=P + 2), dict(ids=P + 2), dict(labels=P + 4),
                   dict(w=P + 2), dict(ce=P + 1), dict(kl=P + 1)):
            assert call(grad, **kw) == EALIGN, kw
        assert call(grad, n_rows=0, logits=None) == 0
    assert call(dl=None) == EINVAL and call(stride=99) == EINVAL and call(dl=P + 1) == EALIGN
    assert call(dl=P, stride=104) == EINVAL  # in place, with another stride


def test_binding_checks_shapes_and_types(B):
    """Shapes and types are the binding's to check: the C call sees sizes only."""
    f = torch.zeros
    with pytest.raises(ValueError):
        B.zero_embed_forward(f(10, 8), f(3, dtype=torch.int64), f(3, 7))
    with pytest.raises(ValueError):
        B.zero_embed_forward(f(10, 8), f(3, dtype=torch.int64), f(3, 8))  # pageable memory
    with pytest.raises(ValueError):
        B.zero_embed_backward(f(3, 8), f(4, dtype=torch.int64), f(10, 8), f(1))
    with pytest.raises(ValueError):
        B.zero_block_norm_forward(f(4, 8), branch=f(4, 9), y=f(4, 8), u=f(4, 8))
    with pytest.raises(ValueError):
        B.zero_block_norm_forward(f(4, 8), branch=f(4, 8), gate=f(3, 8), y=f(4, 8), u=f(4, 8))
    with pytest.raises(ValueError):
        B.zero_block_norm_forward(f(4, 8), u=f(4, 8), kind="batch")
    with pytest.raises(ValueError):
        B.zero_block_norm_backward(f(4, 8), f(1), dy=f(4, 8).double())
    with pytest.raises(ValueError):
        B.zero_distill_forward(f(4, 8), f(4, 3), f(4, 2, dtype=torch.int32), f(4), f(4))
    with pytest.raises(ValueError):
        B.zero_distill_forward(f(8, 4).t(), f(4, 3), f(4, 3, dtype=torch.int32), f(4), f(4))
    with pytest.raises(B.ZeroError):
        B.zero_embed_scratch_bytes(-1, 5, 5)
    with pytest.raises(B.ZeroError):
        B.zero_block_norm_scratch_bytes(5, 1 << 20)
