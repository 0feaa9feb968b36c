"""Sizes at the edge of what the attention's entry points take: refused calls and workspace sizes, no GPU."""
import pytest

from async_rl_b200 import _lib
from async_rl_b200.build import build
from tests.test_layer_refusals_cpu import ARG, BWD, FWD, _call

MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


@pytest.mark.parametrize("S,Tq,Tk,Hq", [(MOST, 0, 0, 1), (MOST, 1000, 1000, 1), (MOST - 500, 10, 1 << 20, 1),
                                        (1 << 30, (1 << 31) - 600, 1 << 20, 128)])
def test_units_past_31_bits_are_refused(lib, S, Tq, Tk, Hq):
    """Units are counted in 32 bits: one for each sequence and tile at most."""
    assert lib.bi_attn_fwd_workspace_bytes(Tq, Tk, S, Hq, 1, 64) == 0
    assert lib.bi_attn_bwd_workspace_bytes(Tq, Tk, S, Hq, 1, 64) == 0
    big = dict(S=S, Tq=Tq, Tk=Tk, Hq=Hq, Hkv=1, D=64, n=1 << 60, q_ld=64 * Hq, k_ld=64, v_ld=64)
    assert _call(lib.bi_attn_fwd, FWD, **big) == ARG
    assert _call(lib.bi_attn_bwd, BWD, **{**big, "do_ld": 64 * Hq, "dq_ld": 64 * Hq, "dk_ld": 64, "dv_ld": 64}) == ARG


@pytest.mark.parametrize("S,Tq,Tk", [(1 << 30, 1 << 20, 1 << 20), (1, (1 << 31) - 600, 1000), (64, 1000, (1 << 31) - 600)])
def test_workspaces_hold_every_unit(lib, S, Tq, Tk):
    """40 bytes of each sequence and 16 of each unit."""
    for fn in (lib.bi_attn_fwd_workspace_bytes, lib.bi_attn_bwd_workspace_bytes):
        assert fn(Tq, Tk, S, 1, 1, 64) > 40 * S + 16 * (S + Tq // 128)
