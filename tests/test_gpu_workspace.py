"""What a workspace held before a call reaches no result: zeros, NaN of bf16 and fp32, infinities, all ones."""
import pytest
import torch

import async_rl_b200 as bi
from async_rl_b200 import _lib
from tests.test_gpu_attention import _offs, _rand
from workloads import make_batch, spec_for

pytestmark = pytest.mark.gpu
FILLS = [0, 0x7FC07FC0, 0x7FC00000, 0x7F807F80, -1]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def _filled(n, fill, dev):
    ws = torch.empty(-(-n // 256) * 256, dtype=torch.uint8, device=dev)
    ws.view(torch.int32).fill_(fill)
    return ws


def _same(run):
    want = run(FILLS[0])
    for fill in FILLS[1:]:
        for a, b in zip(want, run(fill)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), hex(fill)


@pytest.mark.parametrize("prompt_len", [0, 3, 40])
@pytest.mark.parametrize("pstore", [False, True])
def test_loss(prompt_len, pstore, cuda_device):
    b = make_batch(spec_for("tiny", prompt_len=prompt_len)).to(cuda_device)
    mu = torch.full((b.n_rows,), -6.0, device=cuda_device)
    T, H, V = *b.hidden.shape, b.w.shape[0]
    n = bi.workspace_bytes(T, H, V, b.R, pstore=pstore)

    def run(fill):
        o = bi.is_loss_fwd_bwd(b.hidden, b.w, b.targets, mu, b.rewards, b.resp_offsets, b.group_offsets, b.prompt_lens,
                               ws=_filled(n, fill, cuda_device), pstore=pstore)
        bi.check_status(o.status)
        return [o.loss, o.logprob, o.grad_hidden, o.grad_w]

    _same(run)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([130, 0, 70], 6, 2, 128), ([5000], 2, 1, 64), ([1, 1], 8, 8, 64)])
def test_attention_layer(lens, Hq, Hkv, D, cuda_device):
    dev = cuda_device
    T = sum(lens)
    q, k, v, dout = (_rand(T, h, D, i).to(dev) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    o = _offs(lens).to(dev)
    g, pos = torch.ones(D, dtype=torch.bfloat16, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    inv = torch.ones(D // 2, device=dev)
    lib = _lib.load()
    sizes = [fn(T, T, len(lens), Hq, Hkv, D) for fn in (lib.bi_attn_fwd_workspace_bytes, lib.bi_attn_bwd_workspace_bytes)]

    def run(fill):
        out, lse, s0 = bi.attn_fwd(q, k, v, o, ws=_filled(sizes[0], fill, dev))
        dq, dk, dv, s1 = bi.attn_bwd(dout, q, k, v, out, lse, o, ws=_filled(sizes[1], fill, dev))
        back = bi.qk_norm_rope_bwd(dq, dk, q, k, g, g, pos, inv, 1e-6,
                                   ws=_filled(lib.bi_qk_norm_rope_bwd_workspace_bytes(D), fill, dev))
        for s in (s0, s1, back[4]):
            bi.check_status(s)
        return [out, lse, dq, dk, dv, *back[:4]]

    _same(run)
