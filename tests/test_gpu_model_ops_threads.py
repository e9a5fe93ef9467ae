"""The model operators called from two host threads at once, on sizes whose
launches ask for different amounts of shared memory from the same kernel: the
calls are re-entrant, so each gives what it gives alone.  The C calls are made
with arguments prepared beforehand, so that the threads are inside them most of
the time (a foreign call does not hold the interpreter's lock)."""
import ctypes as C
import threading

import pytest
import torch

from fsdp_sharded_optimizer_gb300 import _binding as B

pytestmark = pytest.mark.gpu
CALLS = 4000


def distill(V):
    R, K = 80, 8
    s = torch.randn(R, V, device="cuda").bfloat16()
    t = torch.randn(R, K, device="cuda")
    ids = torch.arange(R * K, device="cuda").view(R, K)
    ce, kl, g = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda"), torch.zeros_like(s)
    spec = B.zero_distill_t(R, V, V, K, 1, 2, 4, 4, 1.0, 0.0, 1.0)
    at = [x.data_ptr() for x in (s, t, ids)]
    args = (C.byref(spec), *at, None, None, ce.data_ptr(), kl.data_ptr(), g.data_ptr(), V)
    return [ce, kl, g], (s, t, ids, spec), B.lib.zero_distill_forward_backward, args


def embed(V):
    n, D = 64, 64
    d = torch.randn(n, D, device="cuda").bfloat16()
    ids = torch.randint(0, V, (n,), device="cuda")
    scratch = torch.empty(B.zero_embed_scratch_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    g = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    args = (d.data_ptr(), 1, ids.data_ptr(), 4, n, 1.0, g.data_ptr(), 1, V, D, 0,
            scratch.data_ptr(), scratch.nbytes)
    return [g], (d, ids, scratch), B.lib.zero_embed_backward, args


def norm(shape):
    R, D = shape
    y, du = (torch.randn(shape, device="cuda").bfloat16() for _ in range(2))
    dx, dw = torch.zeros_like(y), torch.zeros(D, device="cuda")
    scratch = torch.empty(B.zero_block_norm_scratch_bytes(*shape), dtype=torch.uint8, device="cuda")
    spec = B.zero_block_norm_t(R, D, R, 0, 0, 1, 1, 1, 1, 1, 1e-6, 1.0, 1.0)
    grads = B.zero_block_norm_grads_t(None, None, None, dw.data_ptr(), None, 1, 2)
    args = (C.byref(spec), None, du.data_ptr(), y.data_ptr(), None, None, None, None, None,
            dx.data_ptr(), None, C.byref(grads), scratch.data_ptr(), scratch.nbytes)
    return [dx, dw], (y, du, scratch, spec, grads), B.lib.zero_block_norm_backward, args


@pytest.mark.parametrize("make,sizes", [
    (distill, (34000, 24000)), (embed, (100000, 70000)), (norm, ((200, 4096), (5000, 256)))],
    ids=["distill", "embed", "norm"])
def test_two_threads(make, sizes):
    jobs = [make(size) for size in sizes]
    alone = []
    for out, _, call, args in jobs:
        assert call(*args, torch.cuda.current_stream().cuda_stream) == 0
        alone.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def work(call, args):
        stream = torch.cuda.Stream()
        args = (*args, stream.cuda_stream)
        start.wait()
        for i in range(CALLS):
            rc = call(*args)
            if rc != 0:
                failed.append((i, rc))
            if i % 500 == 499:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=job[2:]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, "%d calls failed, the first (call, status): %s" % (len(failed), failed[0])
    for job, want in zip(jobs, alone):
        for t, w in zip(job[0], want):
            assert torch.equal(t, w)
