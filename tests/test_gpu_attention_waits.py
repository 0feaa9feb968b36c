"""The limit of an in-kernel wait is a matter of one unit of work, not of all that a block does: calls whose
longest unit is well below a limit that the whole call is well above."""
import pytest
import torch

import async_rl_b200 as bi
from async_rl_b200 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def _timed(run, limit_ns):
    """Milliseconds of a second run, with that limit on each wait."""
    bi.check_status(run()[-1])
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    _lib.load().bi_debug_attn_wait_limit_once(limit_ns)
    a.record()
    status = run()[-1]
    b.record()
    torch.cuda.synchronize()
    bi.check_status(status)
    return a.elapsed_time(b)


def test_a_short_sequence_behind_a_long_one(cuda_device):
    """65,536 tokens (no ragged tile) and 100 (ragged, the last units of the list).  A forward unit takes 1.3 ms of
    about 32, one of dK, dV 3.5 ms and one of dQ 1 of about 100."""
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(0)
    T, Hq, Hkv, D = 65536 + 100, 32, 8, 128
    q, k, v, dout = (torch.randn(T, h, D, generator=gen, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq))
    offs = torch.tensor([0, 65536, T], device=dev)
    kept = {}

    def fwd():
        kept["out"], kept["lse"], st = bi.attn_fwd(q, k, v, offs)
        return kept["out"], st

    assert _timed(fwd, 8_000_000) > 16
    assert _timed(lambda: bi.attn_bwd(dout, q, k, v, kept["out"], kept["lse"], offs), 12_000_000) > 30


def test_a_wait_that_runs_out_is_reported(cuda_device):
    """262,244 tokens, the last tile ragged: the warp that clears it waits for its unit's other tiles, 5 ms, with a
    limit of 0.2 ms.  The status says so, and the next call is whole."""
    dev = cuda_device
    T = 262144 + 100
    q, k, v = (torch.ones(T, h, 128, dtype=torch.bfloat16, device=dev) for h in (4, 1, 1))
    offs = torch.tensor([0, T], device=dev)
    _lib.load().bi_debug_attn_wait_limit_once(200_000)
    with pytest.raises(bi.BiError, match="TIMEOUT"):
        bi.check_status(bi.attn_fwd(q, k, v, offs)[-1])
    out, lse, st = bi.attn_fwd(q, k, v, offs)
    bi.check_status(st)
    # equal scores: every row is the mean of ones, summed up with terms of 1 (exact), and lse = s + log(keys)
    assert torch.all(out == 1)
