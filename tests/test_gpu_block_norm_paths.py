"""Paths of the block norms' gradient that need many rows: workers that take
several rows, at every width's kernel, and shared gate rows that are found by
the ends of the workers' runs.  References and bounds are those of
test_gpu_block_norm."""
import pytest
import torch

from test_gpu_block_norm import Case, backward64, close, forward64, run_backward

from fsdp_sharded_optimizer_gb300 import _binding as B

pytestmark = pytest.mark.gpu
BIASED = dict(kind="layer", bias=True)
SPECS = [
    dict(rows=8000, dim=64, span=3), dict(rows=1500, dim=2048, span=4),  # found by their ends
    dict(rows=8000, dim=64, span=3, **BIASED), dict(rows=2000, dim=2044, span=5),
    dict(rows=20000, dim=256), dict(rows=20000, dim=256, **BIASED),
    dict(rows=2001, dim=4096, res="f32", span=500), dict(rows=2001, dim=4096, span=2000, **BIASED),
    dict(rows=611, dim=5000), dict(rows=611, dim=5000, span=7), dict(rows=611, dim=5000, span=7, **BIASED),
    dict(rows=611, dim=8192, act="f32", res="f32", span=1), dict(rows=611, dim=5001, **BIASED),
    dict(rows=400, dim=8200, span=150), dict(rows=400, dim=16384, **BIASED),
    dict(rows=400, dim=16380, res="f32", span=1), dict(rows=400, dim=12001),
]
IDS = ["-".join("%s%s" % (k[:4], v) for k, v in c.items()) for c in SPECS]


@pytest.mark.parametrize("spec", SPECS, ids=IDS)
def test_many_rows(spec):
    c = Case(**spec)
    y = torch.empty((c.rows, c.dim), dtype=c.res, device="cuda")
    u = torch.empty((c.rows, c.dim), dtype=c.act, device="cuda")
    B.zero_block_norm_forward(c.x, pre_bias=c.qb, y=y, u=u, **c.common())
    wy, by, wu, bu = forward64(c)
    close(y, wy, by, c.res, "y")
    close(u, wu, bu, c.act, "u")
    want = backward64(c)
    bufs = run_backward(c, torch.float32, want)
    again = run_backward(c, torch.float32, want)
    for name, (_, t) in bufs.items():
        close(t, *want[name], t.dtype, name)
        assert torch.equal(t, again[name][1]), name


@pytest.mark.parametrize("spec", [
    dict(rows=3000, dim=256, span=3), dict(rows=3000, dim=100, act="f32", res="f32"),
    dict(rows=1000, dim=1001, span=1, **BIASED), dict(rows=700, dim=520, span=100, offset=1),
    dict(rows=611, dim=4096), dict(rows=400, dim=5000, **BIASED), dict(rows=400, dim=8200)],
    ids=lambda c: "-".join("%s%s" % (k[:4], v) for k, v in c.items()))
def test_gradients_in_place(spec):
    """dx in dy's place and dbranch in du's: the same bits as apart."""
    c = Case(**spec)
    want = {k: t for k, (_, t) in run_backward(c, torch.float32, backward64(c)).items()}
    scratch = torch.empty(B.zero_block_norm_scratch_bytes(c.rows, c.dim, c.span), dtype=torch.uint8,
                          device="cuda")
    sums = {k: torch.empty_like(t) for k, t in want.items() if k not in ("dx", "dbranch")}
    B.zero_block_norm_backward(c.x, scratch, dy=c.dy, du=c.du, dx=c.dy, dbranch=c.du, **c.common(), **sums)
    assert torch.equal(c.dy, want["dx"]) and torch.equal(c.du, want["dbranch"])
    for k, t in sums.items():
        assert torch.equal(t, want[k]), k
