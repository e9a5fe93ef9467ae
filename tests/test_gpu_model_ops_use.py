"""The model operators as a program uses them: in a CUDA graph with other
launches, and on tensors whose offsets pass 2^31 elements (compared, bit for
bit, with the same rows on their own, at the same alignment to 16 bytes, on which
the order of a loss's sums depends)."""
import pytest
import torch

from fsdp_sharded_optimizer_gb300 import _binding as B

pytestmark = pytest.mark.gpu


def test_graph_replay_equals_calls():
    """Captured once, replayed on new inputs: the same bits as direct calls."""
    T, V, D, K = 700, 3001, 256, 16
    dev = dict(device="cuda")
    ids = torch.empty(T, dtype=torch.int64, **dev)
    dout = torch.empty(T, D, dtype=torch.bfloat16, **dev)
    y, du = torch.empty_like(dout), torch.empty_like(dout)
    logits = torch.empty(T, V, dtype=torch.bfloat16, **dev)
    tl = torch.empty(T, K, **dev)
    ti = torch.empty(T, K, dtype=torch.int32, **dev)
    w = torch.ones(D, dtype=torch.bfloat16, **dev)
    out = dict(x=torch.empty_like(dout), table=torch.empty(V, D, dtype=torch.bfloat16, **dev),
               dx=torch.empty_like(dout), dw=torch.empty(D, **dev),
               u=torch.empty_like(dout), g=torch.empty_like(logits), ce=torch.empty(T, **dev),
               kl=torch.empty(T, **dev))
    s1 = torch.empty(B.zero_embed_scratch_bytes(T, V, D), dtype=torch.uint8, **dev)
    s2 = torch.empty(B.zero_block_norm_scratch_bytes(T, D), dtype=torch.uint8, **dev)
    table = torch.randn(V, D, **dev).bfloat16()

    def fill(seed):
        torch.manual_seed(seed)
        ids.copy_(torch.randint(-1, V, (T,), **dev))
        for t in (dout, y, du, logits):
            t.copy_(torch.randn(t.shape, **dev))
        tl.copy_(torch.randn(T, K, **dev))
        ti.copy_(torch.randint(0, V, (T, K), **dev).to(torch.int32))

    def calls():
        B.zero_embed_forward(table, ids, out["x"], scale=16.0)
        B.zero_embed_backward(dout, ids, out["table"], s1, scale=16.0)
        B.zero_block_norm_forward(y, pre_weight=w, u=out["u"])
        B.zero_block_norm_backward(y, s2, du=du, dy=dout, pre_weight=w, dx=out["dx"],
                                   dpre_weight=out["dw"])
        B.zero_distill_forward_backward(logits, tl, ti, out["ce"], out["kl"], out["g"],
                                        temperature=2.0)

    fill(0)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    fill(1)
    graph.replay()
    torch.cuda.synchronize()
    replayed = {k: v.clone() for k, v in out.items()}
    for v in out.values():
        v.fill_(3.0)
    calls()
    for k, v in out.items():
        assert torch.equal(v, replayed[k]), k


def test_norm_and_embedding_past_2_31_elements():
    D = 4096
    R = (1 << 31) // D + 37
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    for a in range(0, R, 1 << 16):
        x[a:a + (1 << 16)].normal_()
    w = torch.randn(D, device="cuda").bfloat16()
    u = torch.empty_like(x)
    B.zero_block_norm_forward(x, pre_weight=w, u=u)
    few = torch.empty(37, D, dtype=torch.bfloat16, device="cuda")
    B.zero_block_norm_forward(x[-37:], pre_weight=w, u=few)
    assert torch.equal(u[-37:], few)
    scratch = torch.empty(B.zero_block_norm_scratch_bytes(R, D), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    B.zero_block_norm_backward(x, scratch, du=u, pre_weight=w, dx=dx)
    part = torch.empty_like(few)
    B.zero_block_norm_backward(x[-37:], scratch, du=few, pre_weight=w, dx=part)
    assert torch.equal(dx[-37:], part)
    ids = torch.arange(R, device="cuda") % 1000
    B.zero_embed_forward(x[:1000], ids, u, scale=0.5)
    B.zero_embed_forward(x[:1000], ids[-37:], few, scale=0.5)
    assert torch.equal(u[-37:], few)


def test_distillation_past_2_31_elements():
    V, K = 50257, 8
    R = (1 << 31) // V + 20
    x = torch.empty(R, V, dtype=torch.bfloat16, device="cuda")
    for a in range(0, R, 4096):
        x[a:a + 4096].normal_()
    ti = torch.randint(0, V, (R, K), device="cuda", dtype=torch.int32)
    tl = torch.randn(R, K, device="cuda")
    ce, kl = (torch.empty(R, device="cuda") for _ in range(2))
    tail = x[-20:].clone()
    B.zero_distill_forward_backward(x, tl, ti, ce, kl, x, temperature=2.0)
    # the same split of a row over blocks as with many rows: 20 rows alone would
    # use more blocks a row, and another order of the sums
    shift = x[-20].data_ptr() % 16 // 2
    many = torch.empty(160 * V + 8, dtype=torch.bfloat16, device="cuda")[shift:shift + 160 * V]
    many = many.view(160, V)
    many.copy_(tail.repeat(8, 1))
    a, b = (torch.empty(160, device="cuda") for _ in range(2))
    B.zero_distill_forward_backward(many, tl[-20:].repeat(8, 1), ti[-20:].repeat(8, 1), a, b, many,
                                    temperature=2.0)
    assert torch.equal(many[:20], x[-20:]) and torch.equal(b[:20], kl[-20:])
