"""The exchange of words among the blocks of a cluster: every turn's words are that
turn's, and once a limited wait has run out the result is NaN for good, on the
block whose wait it was and, from the next turn at the latest, on all."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from fsdp_sharded_optimizer_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def run_turns(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("exchange") / "exchange.so")
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "exchange_kernel.cu")
    subprocess.run([build.nvcc()] + build.ARCH + build.COMMON + ["-shared", "-o", lib, source], check=True)
    call = C.CDLL(lib).run_turns
    call.argtypes = [C.c_int] * 4 + [C.c_void_p] * 2

    def run(ranks, turns, late=-1, at=0):
        out = torch.zeros(turns, ranks, 64, device="cuda")
        assert call(ranks, turns, late, at, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        i = torch.arange(turns)
        each = ranks * (ranks - 1) // 2
        want = ranks * (100.0 * (i % 64) + i % 7) + 2 * each
        return out.cpu(), want[:, None, None].expand(turns, ranks, 64)

    return run


@pytest.mark.parametrize("ranks", [1, 2, 4, 8])
def test_every_turn(run_turns, ranks):
    out, want = run_turns(ranks, 5001)
    assert torch.equal(out, want)


@pytest.mark.parametrize("ranks,late,at", [(2, 1, 3), (4, 0, 0), (8, 5, 4)])
def test_lost_for_good(run_turns, ranks, late, at):
    out, want = run_turns(ranks, 9, late, at)
    assert torch.equal(out[:at], want[:at])
    others = [r for r in range(ranks) if r != late]
    assert torch.isnan(out[at, others]).all()
    assert (torch.isnan(out[at, late]) | (out[at, late] == want[at, late])).all()
    assert torch.isnan(out[at + 1:]).all()
