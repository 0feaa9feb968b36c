"""What the attention layer's and the update's entry points refuse, before any CUDA call (no GPU needed):
return codes through the C ABI with made-up addresses, and the binding's checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from async_rl_b200 import _lib
from async_rl_b200.build import build

OK, ARG, SHAPE, WS = 0, 1, 2, 3
A = [(1 << 20) * (i + 1) for i in range(32)]  # 1 MiB-aligned addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


QK = dict(q=A[0], k=A[1], q_ld=1536, k_ld=256, gq=A[2], gk=A[3], pos=A[4], inv=A[5], eps=1e-6, T=8, Hq=12, Hkv=2, D=128,
          R=128, qo=A[6], ko=A[7], qo_ld=1536, ko_ld=256, st=A[8], s=None)
QKB = dict(dqo=A[0], dko=A[1], dqo_ld=1536, dko_ld=256, q=A[2], k=A[3], q_ld=1536, k_ld=256, gq=A[4], gk=A[5], pos=A[6],
           inv=A[7], eps=1e-6, T=8, Hq=12, Hkv=2, D=128, R=128, dq=A[8], dk=A[9], dq_ld=1536, dk_ld=256, dgq=A[10],
           dgk=A[11], st=A[12], ws=A[13], n=1 << 30, s=None)
FWD = dict(q=A[0], k=A[1], v=A[2], q_ld=1536, k_ld=256, v_ld=256, qo=A[3], ko=A[4], kl=None, S=2, Tq=64, Tk=64, Hq=12,
           Hkv=2, D=128, causal=1, scale=0.1, out=A[5], lse=A[6], st=A[7], ws=A[8], n=1 << 40, s=None)
BWD = dict(do=A[0], do_ld=1536, q=A[1], k=A[2], v=A[3], q_ld=1536, k_ld=256, v_ld=256, out=A[4], lse=A[5], qo=A[6],
           ko=A[7], kl=None, S=2, Tq=64, Tk=64, Hq=12, Hkv=2, D=128, causal=1, scale=0.1, dq=A[8], dk=A[9], dv=A[10],
           dq_ld=1536, dk_ld=256, dv_ld=256, st=A[11], ws=A[12], n=1 << 40, s=None)


def _call(fn, base, **change):
    assert set(change) <= set(base)
    return fn(*{**base, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(st=None), ARG), (dict(T=-1), ARG), (dict(T=1 << 31), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.inf), ARG),
    (dict(eps=math.nan), ARG), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=4097), SHAPE), (dict(D=72), SHAPE),
    (dict(D=272), SHAPE), (dict(R=144), SHAPE), (dict(R=8), SHAPE), (dict(R=0), SHAPE), (dict(gk=None), ARG),
    (dict(gq=A[2] + 2), ARG), (dict(q=None), ARG), (dict(q=A[0] + 8), ARG), (dict(q_ld=1528), ARG),
    (dict(q_ld=1540), ARG), (dict(k_ld=248), ARG), (dict(qo=A[0]), ARG), (dict(ko=A[1]), ARG), (dict(ko=A[6]), ARG),
    (dict(pos=None), ARG), (dict(inv=None), ARG)])
def test_qk_norm_rope_refuses(lib, change, code):
    assert _call(lib.bi_qk_norm_rope, QK, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(st=None), ARG), (dict(T=-1), ARG), (dict(D=40), SHAPE), (dict(dgq=None), ARG), (dict(dq=A[0]), ARG),
    (dict(dk=A[3]), ARG), (dict(dk=A[8]), ARG), (dict(q=None), ARG), (dict(dko_ld=250), ARG), (dict(ws=None), WS),
    (dict(ws=A[13] + 128), WS), (dict(n=1000), WS)])
def test_qk_norm_rope_bwd_refuses(lib, change, code):
    assert _call(lib.bi_qk_norm_rope_bwd, QKB, **change) == code


COMMON = [
    (dict(st=None), ARG), (dict(S=-1), ARG), (dict(Tq=-1), ARG), (dict(Tk=1 << 31), ARG), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(D=96), SHAPE),
    (dict(D=256), SHAPE), (dict(Hq=13), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hq=2 * 129), SHAPE),
    (dict(qo=None), ARG), (dict(ko=None), ARG), (dict(q=None), ARG), (dict(k=A[1] + 4), ARG), (dict(v_ld=250), ARG),
    (dict(q_ld=1000), ARG), (dict(out=None), ARG), (dict(lse=None), ARG), (dict(ws=None), WS), (dict(n=100), WS)]


@pytest.mark.parametrize("change,code", COMMON + [(dict(ws=A[8] + 16), WS), (dict(out=A[5] + 2), ARG),
                                                   (dict(out=A[0]), ARG), (dict(out=A[1]), ARG), (dict(out=A[2]), ARG)])
def test_attn_fwd_refuses(lib, change, code):
    assert _call(lib.bi_attn_fwd, FWD, **change) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(do=None), ARG), (dict(do_ld=1000), ARG), (dict(dq=None), ARG), (dict(dq_ld=12), ARG), (dict(dv=A[9]), ARG),
    (dict(dq=A[1]), ARG), (dict(dq=A[0]), ARG), (dict(dk=A[3]), ARG), (dict(dv=A[8]), ARG), (dict(ws=A[12] + 32), WS)])
def test_attn_bwd_refuses(lib, change, code):
    assert _call(lib.bi_attn_bwd, BWD, **change) == code


def test_attn_workspaces(lib):
    f, b = lib.bi_attn_fwd_workspace_bytes, lib.bi_attn_bwd_workspace_bytes
    for fn in (f, b):
        assert fn(64, 64, 2, 12, 2, 96) == 0 and fn(64, 64, 2, 13, 2, 128) == 0 and fn(-1, 64, 2, 12, 2, 128) == 0
        assert 0 < fn(0, 0, 0, 12, 2, 128) <= fn(64, 64, 2, 12, 2, 128) <= fn(100000, 100000, 2, 12, 2, 128)
    # nothing that grows with queries times keys
    assert b(1 << 20, 1 << 20, 1, 32, 8, 128) < 4 << 30 and f(1 << 20, 1 << 20, 1, 32, 8, 128) < 1 << 30


def _adamw(lib, rows=None, count=1, **cfg):
    row = [A[0], A[1], A[2], A[3], A[4], 0, 0, 1000]
    table = np.array([row] if rows is None else rows, dtype=np.int64)
    c = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, state_bits=32, param_bf16=1, grad_bf16=0,
             reserved=0)
    extra = {k: cfg.pop(k) for k in ("grad_scale", "step_dev", "st") if k in cfg}
    c.update(cfg)
    s = _lib.AdamWCfg(*c.values())
    return lib.bi_adamw_step(table.ctypes.data, count, ctypes.addressof(s), extra.get("grad_scale"), extra.get("step_dev"),
                             extra.get("st", A[20]), None)


@pytest.mark.parametrize("cfg", [
    dict(st=None), dict(count=-1), dict(state_bits=16), dict(param_bf16=2), dict(grad_bf16=-1), dict(reserved=1),
    dict(lr=-1.0), dict(lr=math.nan), dict(eps=-1e-8), dict(weight_decay=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
    dict(beta2=1.5), dict(beta2=math.nan), dict(step=0), dict(grad_scale=A[0] + 2), dict(step_dev=A[0] + 4),
    dict(param_bf16=0), dict(state_bits=8),
    dict(rows=[[0, A[1], A[2], A[3], A[4], 0, 0, 5]]), dict(rows=[[A[0], A[1], 0, A[3], A[4], 0, 0, 5]]),
    dict(rows=[[A[0], A[1], A[2], A[3] + 2, A[4], 0, 0, 5]]), dict(rows=[[A[0], A[1], A[2], A[3], A[4], 0, 0, -5]]),
    dict(rows=[[A[0], A[1], A[2], A[3], A[4], 0, 0, 5], [A[5], 0, A[6], A[7], A[8], 0, 0, 5]], count=2)])
def test_adamw_refuses(lib, cfg):
    assert _adamw(lib, **cfg) == ARG


def test_the_binding_refuses_host_tensors():
    """Host memory never reaches the library."""
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    o, lse = torch.tensor([0, 4]), torch.zeros(2, 4)
    pos, inv = torch.zeros(4, dtype=torch.int32), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        bi.qk_norm_rope(q, k, None, None, pos, inv, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        bi.qk_norm_rope_bwd(q, k, q, k, None, None, pos, inv, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        bi.attn_fwd(q, k, k, o)
    with pytest.raises(ValueError, match="CUDA"):
        bi.attn_bwd(q, q, k, k, q, lse, o)
    p = [torch.zeros(8)]
    with pytest.raises(ValueError, match="CUDA"):
        bi.AdamWState(p, None, [torch.zeros(8)], [torch.zeros(8)])
    for bad in (dict(params=[], masters=None, exp_avg=[], exp_avg_sq=[]),
                dict(params=[torch.zeros(8, dtype=torch.float16)], masters=None, exp_avg=p, exp_avg_sq=p)):
        with pytest.raises(ValueError):
            bi.AdamWState(**bad)
