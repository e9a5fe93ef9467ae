"""zero_relpos_forward and zero_relpos_backward against their definition.

Forward: one fp32 sum, rounded once: the same bits as the definition's.  Backward:
gradients that are small whole numbers have sums that fp32 holds exactly, so those are
compared for equality; for others a sum of n terms in fp32 is right to (roundings of a
term on its way) * 2^-24 of the sum of magnitudes: a thread adds at most one place in
eight rows of a diagonal (times the batch), then 8 warps, 9 + 5 steps of a bucket's
sum, flushes and parts follow: rows * batch + 1024 covers them.
"""
import functools
import math

import pytest
import torch

import fsdp_sharded_optimizer_gb300 as Z

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@functools.lru_cache(None)
def bucket(ahead, buckets, distance, both):
    """The definition, in whole numbers."""
    n_one = buckets // 2 if both else buckets
    first = n_one if both and ahead > 0 else 0
    n = abs(ahead) if both else max(0, -ahead)
    half = n_one // 2
    if n < half:
        return first + n
    parts, j = n_one - half, 0
    while j + 1 < parts and n ** parts * half ** (j + 1) >= distance ** (j + 1) * half ** parts:
        j += 1
    return first + half + j


def buckets_of(Q, K, start, buckets, distance, both):
    line = torch.tensor([bucket(d, buckets, distance, both)
                         for d in range(-start - Q + 1, K - start)])
    at = torch.arange(K)[None, :] - torch.arange(Q)[:, None] + Q - 1
    return line[at].cuda()


def strided(shape, dtype, pad, offset, fill=7.0):
    """A tensor whose rows are `pad` elements further apart than they are long."""
    B, H, Q, K = shape
    buf = torch.full((offset + B * H * Q * (K + pad) + 16,), fill, dtype=dtype, device="cuda")
    t = buf[offset:offset + B * H * Q * (K + pad)].view(B, H, Q, K + pad)[..., :K]
    return buf, t


class Case:
    def __init__(self, B=1, H=2, Q=16, K=16, buckets=32, distance=128, both=True, causal=False,
                 ragged=False, start=0, starts=None, type="bf16", table="bf16", pad=0, offset=0):
        self.__dict__.update(B=B, H=H, Q=Q, K=K, buckets=buckets, distance=distance, both=both,
                             causal=causal, start=start, type=TYPES[type], table_type=TYPES[table],
                             pad=pad, offset=offset)
        self.gen = torch.Generator(device="cuda").manual_seed(B * 7 + Q * 31 + K)
        self.starts = None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda()
        self.q_lengths = self.k_lengths = None
        if ragged:
            # some empty, some whole, some beyond what there is (held within it)
            self.q_lengths = torch.tensor([(Q, 0, Q // 2, Q + 5, 1)[b % 5] for b in range(B)],
                                          dtype=torch.int32).cuda()
            self.k_lengths = torch.tensor([(K // 2, K, 0, K + 9, -3, 1)[b % 6] for b in range(B)],
                                          dtype=torch.int32).cuda()

    def args(self):
        return dict(start=self.start, starts=self.starts, q_lengths=self.q_lengths,
                    k_lengths=self.k_lengths, max_distance=self.distance,
                    bidirectional=self.both, causal=self.causal)

    def masks(self, b):
        """Bucket of each place, which keys count, which rows do."""
        start = self.start if self.starts is None else int(self.starts[b])
        at = buckets_of(self.Q, self.K, start, self.buckets, self.distance, self.both)
        on = torch.ones((self.Q, self.K), dtype=torch.bool, device="cuda")
        if self.causal:
            on &= (torch.arange(self.K).cuda()[None] <= torch.arange(self.Q).cuda()[:, None] + start)
        if self.k_lengths is not None:
            on[:, min(self.K, max(0, int(self.k_lengths[b]))):] = False
        rows = self.Q
        if self.q_lengths is not None:
            rows = min(self.Q, max(0, int(self.q_lengths[b])))
        return at, on, rows


CASES = [
    dict(Q=1, K=1), dict(Q=1, K=37, start=36, both=False, causal=True),
    dict(Q=1, K=1021, start=1020, both=False, causal=True, B=4, H=12, ragged=True, type="f32"),
    dict(Q=5, K=3), dict(Q=3, K=5, H=1), dict(Q=16, K=16, B=3), dict(Q=77, K=333, B=2, H=3),
    dict(Q=333, K=333, B=6, H=2, ragged=True, buckets=320, distance=800),
    dict(Q=256, K=256, causal=True, both=False, B=5, ragged=True),
    dict(Q=200, K=264, start=64, causal=True, both=False), dict(Q=64, K=64, start=-30, causal=True),
    dict(Q=64, K=64, start=-100, causal=True, both=False), dict(Q=40, K=48, start=1000),
    dict(Q=40, K=48, start=-1000, both=False), dict(Q=40, K=48, start=1 << 39),
    dict(Q=9, K=600, start=300, buckets=64, distance=256),
    dict(Q=50, K=50, start=3, B=7, starts=[0, 3, -5, 1 << 30, -(1 << 30), 100, 49], ragged=True),
    dict(Q=33, K=129, B=4, starts=[96, 95, 0, 50], causal=True, both=False),
    dict(Q=24, K=72, B=3, starts=[48, 48, 40], type="f32", causal=True, both=True),
    dict(Q=128, K=128, pad=8), dict(Q=65, K=121, pad=7), dict(Q=65, K=121, pad=2, type="f32"),
    dict(Q=30, K=64, offset=1), dict(Q=30, K=61, offset=3, type="f32"),
    dict(Q=30, K=1, B=3), dict(Q=700, K=2, buckets=16, distance=64),
    dict(Q=20, K=20, buckets=2, both=False, distance=2), dict(Q=20, K=20, buckets=3, both=False),
    dict(Q=20, K=30, buckets=4, distance=2), dict(Q=100, K=100, buckets=6, distance=9),
    dict(Q=100, K=90, buckets=512, distance=8192), dict(Q=60, K=60, buckets=320, distance=100),
    dict(Q=1024, K=1024, H=1), dict(Q=2000, K=300, H=1, table="f32"),
    dict(Q=2, K=20000, H=1, buckets=512, distance=8192, start=9000, table="f32"),
    dict(B=70000, H=1, Q=2, K=3), dict(B=3, H=40, Q=8, K=8, table="f32"),
]
IDS = ["-".join("%s%s" % kv for kv in c.items() if kv[0] != "starts") for c in CASES]


@pytest.mark.parametrize("with_scores", [False, True, "in place", "other stride"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, with_scores):
    c = Case(**case)
    table = torch.randn((c.buckets, c.H), generator=c.gen, device="cuda").to(c.table_type)
    shape = (c.B, c.H, c.Q, c.K)
    buf, out = strided(shape, c.type, c.pad, c.offset)
    scores = None
    if with_scores:
        value = torch.randn(shape, generator=c.gen, device="cuda").to(c.type)
        for b in range(min(c.B, 8)):  # what is masked may hold anything
            _, on, _ = c.masks(b)
            value[b, :, ~on] = math.nan
        if with_scores == "in place":
            scores = out
        else:
            scores = strided(shape, c.type, c.pad + (with_scores == "other stride"), c.offset)[1]
        scores.copy_(value)
    before = out.clone()
    Z.zero_relpos_forward(table, out, scores=scores, **c.args())
    for b in range(c.B) if c.B < 100 else (0, 1, c.B - 1):
        at, on, rows = c.masks(b)
        want = table.float()[at].permute(2, 0, 1)
        if with_scores:
            want = value[b].float() + want
        want = torch.where(on, want, -math.inf).to(c.type)
        assert torch.equal(out[b, :, :rows], want[:, :rows]), b
        assert torch.equal(out[b, :, rows:].isnan(), before[b, :, rows:].isnan())
        assert torch.equal(out[b, :, rows:].nan_to_num(), before[b, :, rows:].nan_to_num())
    n = c.B * c.H * c.Q
    gaps = buf[c.offset:c.offset + n * (c.K + c.pad)].view(n, -1)[:, c.K:]
    assert torch.all(gaps == 7) and torch.all(buf[:c.offset] == 7) and torch.all(buf[-16:] == 7)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_is_exact_for_whole_numbers(case, accumulate):
    c = Case(**case)
    shape = (c.B, c.H, c.Q, c.K)
    value = torch.randint(-8, 9, shape, generator=c.gen, device="cuda").float()
    _, dout = strided(shape, c.type, c.pad, c.offset, fill=math.nan)
    dout.copy_(value)
    want = torch.zeros((c.buckets, c.H), dtype=torch.float64, device="cuda")
    if c.B > 100:  # all sequences alike
        at, on, rows = c.masks(0)
        total = value.double().sum(0)
        for q in range(c.buckets):
            want[q] = torch.where(at == q, total, 0.0).sum((1, 2))
    else:
        for b in range(c.B):
            at, on, rows = c.masks(b)
            live = on & (torch.arange(c.Q).cuda() < rows)[:, None]
            dout[b, :, ~live] = math.nan
            want.index_add_(0, at[live], value[b][:, live].double().t().contiguous())
    old = torch.randint(-9, 10, want.shape, generator=c.gen, device="cuda").to(c.table_type)
    dtable = old.clone()
    need = Z.zero_relpos_scratch_bytes(c.B, c.H, c.Q, c.K, c.buckets)
    scratch = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    Z.zero_relpos_backward(dout, dtable, scratch[:need], accumulate=accumulate, **c.args())
    assert float(want.abs().max()) < 2 ** 24
    if accumulate:
        want = want + old.double()
    assert torch.equal(dtable, want.to(c.table_type))
    assert torch.all(scratch[need:] == 255)
    again = old.clone()
    Z.zero_relpos_backward(dout, again, scratch[:need], accumulate=accumulate, **c.args())
    assert torch.equal(dtable, again)


@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_backward_of_real_gradients(type):
    c = Case(B=3, H=4, Q=700, K=513, type=type, table="f32", ragged=True)
    dout = torch.randn((c.B, c.H, c.Q, c.K), generator=c.gen, device="cuda").to(c.type)
    want = torch.zeros((c.buckets, c.H), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for b in range(c.B):
        at, on, rows = c.masks(b)
        live = on & (torch.arange(c.Q).cuda() < rows)[:, None]
        v = dout[b][:, live].double().t().contiguous()
        want.index_add_(0, at[live], v)
        size.index_add_(0, at[live], v.abs())
    dtable = torch.empty((c.buckets, c.H), device="cuda")
    scratch = torch.empty(Z.zero_relpos_scratch_bytes(c.B, c.H, c.Q, c.K, c.buckets),
                          dtype=torch.uint8, device="cuda")
    Z.zero_relpos_backward(dout, dtable, scratch, **c.args())
    assert torch.all((dtable.double() - want).abs() <= (c.Q * c.B + 1024) * U * size)


def test_gradient_against_differences():
    """The table's gradient of sum(dout * out): out is linear in the table, so the
    difference of two forward calls is the gradient's product with the step."""
    c = Case(B=2, H=3, Q=45, K=70, type="f32", table="f32", start=25, causal=True, both=False)
    gen = c.gen
    table = torch.randint(-4, 5, (c.buckets, c.H), generator=gen, device="cuda").float()
    dout = torch.randint(-4, 5, (c.B, c.H, c.Q, c.K), generator=gen, device="cuda").float()
    scratch = torch.empty(Z.zero_relpos_scratch_bytes(c.B, c.H, c.Q, c.K, c.buckets),
                          dtype=torch.uint8, device="cuda")
    dtable = torch.empty_like(table)
    Z.zero_relpos_backward(dout, dtable, scratch, **c.args())
    step = torch.randint(-2, 3, table.shape, generator=gen, device="cuda").float()
    value = []
    for t in (table, table + step):
        out = torch.zeros_like(dout)
        Z.zero_relpos_forward(t, out, **c.args())
        value.append(torch.where(out > -math.inf, out.double() * dout.double(), 0.0).sum())
    assert float(value[1] - value[0]) == float((dtable.double() * step.double()).sum())


def test_empty_sizes():
    table = torch.ones((32, 2), device="cuda")
    scratch = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for shape in ((0, 2, 4, 4), (1, 2, 0, 4), (1, 2, 4, 0)):
        out = torch.empty(shape, device="cuda")
        Z.zero_relpos_forward(table, out)
        d = torch.full_like(table, 3.0)
        Z.zero_relpos_backward(out, d, scratch, accumulate=True)
        assert torch.all(d == 3)
        Z.zero_relpos_backward(out, d, scratch)
        assert torch.all(d == 0)


def test_captured_and_on_another_stream():
    c = Case(B=2, H=3, Q=100, K=100, type="f32", table="f32", causal=True)
    table = torch.randn((c.buckets, c.H), generator=c.gen, device="cuda")
    dout = torch.randint(-4, 5, (c.B, c.H, c.Q, c.K), generator=c.gen, device="cuda").float()
    out, dtable = torch.empty_like(dout), torch.empty_like(table)
    scratch = torch.empty(Z.zero_relpos_scratch_bytes(c.B, c.H, c.Q, c.K, c.buckets),
                          dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        Z.zero_relpos_forward(table, out, **c.args())
        Z.zero_relpos_backward(dout, dtable, scratch, **c.args())
    stream.synchronize()
    want = out.clone(), dtable.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_relpos_forward(table, out, **c.args())
        Z.zero_relpos_backward(dout, dtable, scratch, **c.args())
    for _ in range(2):
        out.zero_()
        dtable.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dtable, want[1])


def test_past_2_31_elements():
    """Planes whose places are beyond 32 bits."""
    B, H, Q, K = 3, 16, 8192, 8192
    dout = torch.zeros((B, H, Q, K), dtype=torch.bfloat16, device="cuda")
    assert dout.numel() > 1 << 31
    dout[2, 15, 8191, 8191] = 2.0
    dout[2, 15, 8191, 0] = 3.0
    dout[2, 15, 0, 8191] = 4.0
    dtable = torch.empty((32, H), device="cuda")
    scratch = torch.empty(Z.zero_relpos_scratch_bytes(B, H, Q, K, 32), dtype=torch.uint8,
                          device="cuda")
    Z.zero_relpos_backward(dout, dtable, scratch)
    want = torch.zeros_like(dtable)
    want[0, 15], want[15, 15], want[31, 15] = 2.0, 3.0, 4.0
    assert torch.equal(dtable, want)
    table = torch.arange(32 * H, device="cuda").float().view(32, H)
    Z.zero_relpos_forward(table, dout)
    for (i, j), v in (((8191, 8191), 0), ((8191, 0), 15), ((0, 8191), 31), ((8000, 7999), 1)):
        assert float(dout[2, 15, i, j]) == float(table[v, 15].bfloat16())
