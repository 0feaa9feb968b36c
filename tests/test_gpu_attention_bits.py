"""A row's bits in a prefill, alone over a cache, among its last neighbours and in another batch, on scores that
make the softmax raise its reference: every tile, now and then, and by less than the threshold."""
import pytest
import torch

import async_rl_b200 as bi
from tests.test_gpu_attention import _offs, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def _inputs(kind, T, Hq, Hkv, D):
    """q and k whose scores (scale 1) rise by `slope` a key, or are large and of both signs."""
    q, k, v = _rand(T, Hq, D, 1).float(), _rand(T, Hkv, D, 2).float(), _rand(T, Hkv, D, 3)
    if kind == "peaked":
        return (q * 2).to(torch.bfloat16), k.to(torch.bfloat16), v
    slope = dict(every_tile=0.125, some_tiles=0.02, falling=-0.05)[kind]
    q, k = q * 0.3, k * 0.3
    q[:, :, 0] = 4.0
    k[:, :, 0] = (torch.arange(T) * (slope / 4.0))[:, None]
    return q.to(torch.bfloat16), k.to(torch.bfloat16), v


@pytest.mark.parametrize("kind", ["every_tile", "some_tiles", "falling", "peaked"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 12, 2), (64, 8, 8), (128, 5, 1)])
def test_prefill_decode_and_batch(kind, D, Hq, Hkv, cuda_device):
    dev = cuda_device
    lens = [130, 2047, 2049, 4500, 6200]
    q, k, v = (t.to(dev) for t in _inputs(kind, max(lens), Hq, Hkv, D))
    q, k, v = (torch.cat([t[:n] for n in lens]) for t in (q, k, v))
    o = _offs(lens).to(dev)
    out, lse, st = bi.attn_fwd(q, k, v, o, scale=1.0)
    bi.check_status(st)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    gen = torch.Generator().manual_seed(0)
    starts = o[:-1]
    for trial in range(6):
        at = [n - 1 if trial == 0 else int(torch.randint(0, n, (1,), generator=gen)) for n in lens]
        rows = starts + torch.tensor(at, device=dev)
        # all sequences' single tokens, then one alone, which is split over SMs
        d, dl, st = bi.attn_fwd(q[rows].contiguous(), k, v, torch.arange(len(lens) + 1, device=dev), k_offsets=o, scale=1.0,
                                k_lens=torch.tensor([a + 1 for a in at], dtype=torch.int32, device=dev))
        bi.check_status(st)
        assert torch.equal(d, out[rows]) and torch.equal(dl, lse[:, rows])
        i = trial % len(lens)
        r, a, b = int(rows[i]), int(o[i]), int(o[i]) + at[i] + 1
        d, dl, st = bi.attn_fwd(q[r:r + 1], k[a:b], v[a:b], torch.tensor([0, 1], device=dev),
                                k_offsets=torch.tensor([0, b - a], device=dev), scale=1.0)
        bi.check_status(st)
        assert torch.equal(d[0], out[r]) and torch.equal(dl[:, 0], lse[:, r])
    # the last 70 queries of each sequence (units of two row tiles), and each sequence by itself
    for i, n in enumerate(lens):
        a, b = int(o[i]), int(o[i + 1])
        for m in (70, n):
            d, dl, st = bi.attn_fwd(q[b - m:b], k[a:b], v[a:b], torch.tensor([0, m], device=dev),
                                    k_offsets=torch.tensor([0, n], device=dev), scale=1.0)
            bi.check_status(st)
            assert torch.equal(d, out[b - m:b]) and torch.equal(dl, lse[:, b - m:b])
