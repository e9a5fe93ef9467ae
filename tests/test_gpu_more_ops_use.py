"""The group norm, the relative position bias and the clip over many tensors as a training
program uses them: one step of a small encoder whose gradients are tensors of their own,
clipped into the ranks' flat gradients and taken by the sharded step; from two host
threads; in graphs that share a scratch; on pinned host memory."""
import ctypes as C
import math
import threading

import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z
from fsdp_sharded_optimizer_gb300 import _binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

N, P, CH, GROUPS, HEADS, BUCKETS, OUT = 3, 70, 48, 6, 4, 32, 10


def make_weights(gen):
    r = lambda *s, k=1.0: torch.randn(s, generator=gen, device="cuda") * k
    return {"gamma": 1 + 0.1 * r(CH), "beta": 0.1 * r(CH), "table": 0.5 * r(BUCKETS, HEADS),
            "q": r(CH, CH, k=CH ** -0.5), "k": r(CH, CH, k=CH ** -0.5),
            "v": r(CH, CH, k=CH ** -0.5), "o": r(OUT, CH, k=CH ** -0.5)}


def heads(t):
    return t.view(N, P, HEADS, CH // HEADS).transpose(1, 2)


def encoder_grads(w, x, target, lengths):
    """Loss and gradients with the library's operators around the matrix products (fp32)."""
    u, stats = torch.zeros_like(x), torch.empty((N, GROUPS, 2), device="cuda")
    s_norm = torch.empty(Z.zero_group_norm_scratch_bytes(N, P, CH, GROUPS), dtype=torch.uint8,
                         device="cuda")
    norm = dict(weight=w["gamma"], bias=w["beta"], lengths=lengths, act="silu")
    Z.zero_group_norm_forward(x, u, stats, s_norm, **norm)
    q, k, v = (heads(u @ w[n].t()) for n in "qkv")
    scores = (q @ k.transpose(2, 3)).contiguous()
    place = dict(q_lengths=lengths, k_lengths=lengths, bidirectional=True)
    Z.zero_relpos_forward(w["table"], scores, scores=scores, **place)  # in place, padded keys -inf
    live = (torch.arange(P, device="cuda") < lengths[:, None]).view(N, 1, P, 1)
    p = torch.where(live, torch.softmax(scores, -1), 0.0)
    mixed = (p @ v).transpose(1, 2).reshape(N, P, CH)
    y = mixed @ w["o"].t()
    dy = torch.where(live.view(N, P, 1), y - target, 0.0)
    g = {"o": torch.einsum("npo,npc->oc", dy, mixed)}
    dmixed = heads(dy @ w["o"])
    dp = dmixed @ v.transpose(2, 3)
    ds = (p * (dp - (p * dp).sum(-1, keepdim=True))).contiguous()
    g["table"] = torch.empty_like(w["table"])
    s_table = torch.empty(Z.zero_relpos_scratch_bytes(N, HEADS, P, P, BUCKETS), dtype=torch.uint8,
                          device="cuda")
    Z.zero_relpos_backward(ds, g["table"], s_table, **place)
    flat = lambda t: t.transpose(1, 2).reshape(N, P, CH)
    dq, dk, dv = flat(ds @ k), flat(ds.transpose(2, 3) @ q), flat(p.transpose(2, 3) @ dmixed)
    for n, d in zip("qkv", (dq, dk, dv)):
        g[n] = torch.einsum("npo,npc->oc", d, u)
    du = dq @ w["q"] + dk @ w["k"] + dv @ w["v"]
    g["gamma"], g["beta"], dx = (torch.empty_like(t) for t in (w["gamma"], w["beta"], x))
    Z.zero_group_norm_backward(x, du, stats, dx, s_norm, dweight=g["gamma"], dbias=g["beta"], **norm)
    return g, dx


def encoder_autograd(w, x, target, lengths):
    """The same by torch in fp64."""
    w = {n: t.double().requires_grad_() for n, t in w.items()}
    x = x.double().requires_grad_()
    per = CH // GROUPS
    u = []
    for n in range(N):
        L = int(lengths[n])
        v = x[n, :L].view(L, GROUPS, per)
        mean = v.mean((0, 2), keepdim=True)
        h = (v - mean) / torch.sqrt(((v - mean) ** 2).mean((0, 2), keepdim=True) + 1e-5)
        z = h.reshape(L, CH) * w["gamma"] + w["beta"]
        u.append(torch.cat([z * torch.sigmoid(z), z.new_zeros((P - L, CH))]))
    u = torch.stack(u)
    q, k, v = (heads(u @ w[n].t()) for n in "qkv")
    ahead = torch.arange(P)[None] - torch.arange(P)[:, None]
    half, n = BUCKETS // 2, ahead.abs()
    small = half // 2
    far = small + (torch.log(n.clamp(min=1) / small) / math.log(128 / small) * (half - small) + 1e-9).floor().long()
    at = torch.where(n < small, n, far.clamp(max=half - 1)) + half * (ahead > 0)
    live = torch.arange(P, device="cuda") < lengths[:, None]
    s = q @ k.transpose(2, 3) + w["table"][at.cuda()].permute(2, 0, 1)
    p = torch.softmax(s.masked_fill(~live[:, None, None], -math.inf), -1)
    y = (p @ v).transpose(1, 2).reshape(N, P, CH) @ w["o"].t()
    loss = (0.5 * (y - target.double()) ** 2 * live[:, :, None]).sum()
    loss.backward()
    return {n: t.grad for n, t in w.items()}, x.grad


def test_a_step_of_an_encoder():
    gen = torch.Generator(device="cuda").manual_seed(11)
    w = make_weights(gen)
    lengths = torch.tensor([P, 41, 1], dtype=torch.int32, device="cuda")
    sizes = [t.numel() for t in w.values()]
    (unit,), _ = Z.zero_layout([sum(sizes)], 2)
    grads = torch.zeros((2, unit.n_padded), dtype=torch.bfloat16, device="cuda")
    s, nc = torch.empty(Z.zero_clip_scratch_bytes(), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    backend = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        for rank in range(2):
            x = torch.randn((N, P, CH), generator=gen, device="cuda")
            target = torch.randn((N, P, OUT), generator=gen, device="cuda")
            got, dx = encoder_grads(w, x, target, lengths)
            want, dx64 = encoder_autograd(w, x, target, lengths)
            # fp32 chains of some 10 operators and sums of up to 210 terms: 1e-4 of the norm
            for n in w:
                assert float((got[n] - want[n]).norm() / want[n].norm()) < 1e-4, n
            for i in range(N):
                L = int(lengths[i])
                assert float((dx[i, :L] - dx64[i, :L]).norm()) <= 1e-4 * float(dx64.norm())
            places = [p.view(t.shape) for p, t in zip(grads[rank, :sum(sizes)].split(sizes), w.values())]
            Z.zero_tensors_clip(Z.zero_tensor_list([got[n] for n in w], places), 1.0, nc, s)
            norm = math.sqrt(sum(float(got[n].double().square().sum()) for n in w))
            assert abs(float(nc[0]) / norm - 1) <= 6.5 * U
            for n, p in zip(w, places):
                one = got[n].double() / (norm + 1e-6)
                assert torch.all((p.double() - one).abs() <= one.abs() * (torch.finfo(p.dtype).eps / 2 + 9 * U) + 1e-38)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = backend
    assert int(torch.count_nonzero(grads[:, sum(sizes):])) == 0
    master = torch.zeros((2, unit.shard_len), device="cuda")
    torch.cat([t.reshape(-1) for t in w.values()], out=(flat := torch.zeros(sum(sizes), device="cuda")))
    master.view(-1)[:sum(sizes)] = flat
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    params = torch.empty(unit.n_padded, dtype=torch.bfloat16, device="cuda")
    Z.zero_step_stage12(2, grads, master, m, v, params, Z.hparams(lr=1e-2, weight_decay=0.0))
    # the first AdamW step moves each weight by lr against its gradient's sign
    mean = grads.float().mean(0)[:sum(sizes)]
    moved = master.view(-1)[:sum(sizes)] - flat
    big = mean.abs() > 1e-5
    assert torch.equal(torch.sign(moved[big]), -torch.sign(mean[big])) and bool(big.any())


def group_norm_job(shape):
    n, p, c, g = shape
    x, dy = (torch.randn((n, p, c), device="cuda").bfloat16() for _ in range(2))
    stats = torch.rand((n, g, 2), device="cuda") + 0.5
    dx, dw = torch.zeros_like(x), torch.zeros(c, device="cuda")
    s = torch.empty(Z.zero_group_norm_scratch_bytes(n, p, c, g), dtype=torch.uint8, device="cuda")
    spec = B.zero_group_norm_t(n, p, c, c, c, g, 1, 1, 2, 1, 1e-5)
    args = (C.byref(spec), x.data_ptr(), dy.data_ptr(), None, None, None, stats.data_ptr(),
            dx.data_ptr(), dw.data_ptr(), None, s.data_ptr(), s.nbytes)
    return [dx, dw], (x, dy, stats, s, spec), B.lib.zero_group_norm_backward, args


def relpos_job(shape):
    b, h, k, buckets, distance = shape
    out = torch.zeros((b, h, k, k), device="cuda")
    table = torch.randn((buckets, h), device="cuda")
    spec = B.zero_relpos_t(b, h, k, k, 0, distance, buckets, 1, 0, 2, 2)
    args = (C.byref(spec), table.data_ptr(), None, None, None, None, 0, out.data_ptr(), k)
    return [out], (table, spec), B.lib.zero_relpos_forward, args


def clip_job(sizes):
    src = [torch.randn(n, device="cuda") for n in sizes]
    dst = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
    tl = Z.zero_tensor_list(src, dst)
    nc = torch.zeros(2, device="cuda")
    s = torch.empty(Z.zero_clip_scratch_bytes(), dtype=torch.uint8, device="cuda")
    args = (tl.array, tl.n, 1.0, nc.data_ptr(), s.data_ptr(), s.nbytes)
    return [*dst, nc], (tl, s), B.lib.zero_tensors_clip, args


@pytest.mark.parametrize("make,sizes", [
    (group_norm_job, ((2, 400, 64, 8), (1, 90, 256, 4))),
    (group_norm_job, ((1, 5000, 64, 8), (2, 64, 40, 4))),
    (relpos_job, ((1, 2, 64, 32, 128), (1, 2, 64, 512, 8192))),
    (clip_job, ([1000, 7], [5] * 300))], ids=["held", "passes", "relpos", "clip"])
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
        for i in range(1500):
            rc = call(*args)
            if rc != 0:
                failed.append((i, rc))
            if i % 300 == 299:
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


def test_graphs_that_share_a_scratch():
    """Two captured calls with one scratch, replayed in turn on one stream."""
    shapes = [(2, 3000, 64, 8), (3, 200, 128, 4)]
    need = max(Z.zero_group_norm_scratch_bytes(*s) for s in shapes)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    jobs = []
    for n, p, c, g in shapes:
        x, dy = (torch.randn((n, p, c), device="cuda").bfloat16() for _ in range(2))
        y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty((n, g, 2), device="cuda")
        dw, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")

        def call(x=x, dy=dy, y=y, dx=dx, stats=stats, dw=dw, db=db):
            Z.zero_group_norm_forward(x, y, stats, scratch)
            Z.zero_group_norm_backward(x, dy, stats, dx, scratch, dweight=dw, dbias=db)

        call()
        torch.cuda.synchronize()
        outs = (y, stats, dx, dw, db)
        want = [t.clone() for t in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        jobs.append((graph, outs, want, call))  # the call keeps the captured inputs
    for _ in range(3):
        for _, outs, _, _ in jobs:
            for t in outs:
                t.zero_()
        for graph, _, _, _ in jobs:
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _ in jobs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_pinned_host_memory():
    """Inputs and outputs in page-locked host memory, as every kernel of the library takes them."""
    pin = lambda t: t.cpu().pin_memory()
    x = torch.randn((2, 50, 32), device="cuda")
    scratch = torch.empty(Z.zero_group_norm_scratch_bytes(2, 50, 32, 4), dtype=torch.uint8, device="cuda")
    y, stats = torch.empty_like(x), torch.empty((2, 4, 2), device="cuda")
    Z.zero_group_norm_forward(x, y, stats, scratch)
    hx, hy = pin(x), pin(torch.zeros_like(x))
    Z.zero_group_norm_forward(hx, hy, stats, scratch)
    torch.cuda.synchronize()
    assert torch.equal(hy.cuda(), y)
    s, nc = torch.empty(Z.zero_clip_scratch_bytes(), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    Z.zero_tensors_clip([x], 0.5, nc, s)
    Z.zero_tensors_clip([hx], 0.5, nc, s)
    torch.cuda.synchronize()
    assert torch.equal(hx.cuda(), x)
    table, out = torch.randn((32, 2), device="cuda"), torch.empty((1, 2, 9, 9), device="cuda")
    Z.zero_relpos_forward(table, out)
    ht, ho = pin(table), pin(torch.zeros_like(out))
    Z.zero_relpos_forward(ht, ho)
    torch.cuda.synchronize()
    assert torch.equal(ho.cuda(), out)
