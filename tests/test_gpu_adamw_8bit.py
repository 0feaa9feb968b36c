"""The 8-bit states of the AdamW step where the format is at its ends: blocks that have almost vanished,
elements that are not finite.  The rule is evaluated beside it in fp32, one rounded operation at a time, so that
codes and scales have to be equal; tolerances count e4m3's half step (2^-4 relative)."""
import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from tests.test_gpu_adamw import _sqrt

pytestmark = pytest.mark.gpu
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def hold(x, root):
    """The documented format of x [blocks, 256]: (codes as floats, scales)."""
    most = x.abs().amax(1)
    inv = most.reciprocal() * 448.0
    gone = torch.isinf(inv)
    inv, most = torch.where(gone, 0.0, inv), torch.where(gone, 0.0, most)
    y = x * inv[:, None]
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).float(), most * torch.tensor(1 / 448.0)


def state(p, m, root, dev):
    """A handle over p [blocks, 256] with held m and sqrt(v)."""
    (cm, sm), (cv, sv) = hold(m, False), hold(root, True)
    c = lambda t: [t.contiguous().to(dev)]  # noqa: E731
    f8 = lambda t: [t.to(torch.float8_e4m3fn).contiguous().to(dev)]  # noqa: E731
    return bi.AdamWState(c(p), None, f8(cm), f8(cv), c(sm), c(sv))


def test_blocks_that_have_almost_vanished(cuda_device):
    """Maxima from 1e-34 down to the smallest subnormal: held by the rule, as zeros where 448 / max is infinite, and
    never as codes that do not belong to their scale."""
    gen = torch.Generator().manual_seed(0)
    tops = torch.tensor([1e-34, 3e-36, 1.4e-36, 1.32e-36, 1.3e-36, 1e-36, 1e-37, 2e-38, 1e-38, 1e-40, 1.4e-45, 0.0])
    grad = torch.rand(len(tops), 256, generator=gen) * 0.9 * tops[:, None]
    grad[:, 7] = tops
    grad[:, ::2] *= -1
    zero = torch.zeros_like(grad)
    st = state(zero, zero, zero, cuda_device)
    bi.check_status(bi.adamw_step(st, [grad.to(cuda_device)], 1, **HYPER))
    m = grad * torch.tensor(1 - HYPER["beta1"], dtype=torch.float64).float()
    codes, scale = hold(m, False)
    assert torch.equal(st.exp_avg[0].cpu().float(), codes) and torch.equal(st.exp_avg_scale[0].cpu(), scale)
    held, want = codes.double() * scale.double()[:, None], m.double()
    assert torch.all((scale > 0) | (m.abs().amax(1) < 1.32e-36))
    for h, w, s in zip(held, want, scale.double()):
        # half a code's step, or half of the smallest one; a scale below the normal range has lost 3 bits at most
        assert s == 0 or torch.all((h - w).abs() <= torch.maximum(2.0 ** -4 * w.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -18))


def test_a_block_without_gradients_decays_to_zero(cuda_device):
    """900 steps with no gradient: the maximum keeps the code 448, so the scale shrinks by beta1 and a code c comes
    back as c (1 + 2^-18) at most, which rounds to c, until the block is zeros (0.9^794 = 1e-36)."""
    gen = torch.Generator().manual_seed(1)
    zero = torch.zeros(1, 256)
    st = state(zero, torch.randn(1, 256, generator=gen), zero + 1.0, cuda_device)
    g = [zero.to(cuda_device)]
    first = st.exp_avg[0].float().cpu().double()  # codes: the largest stays 448 while the scale decays
    for t in range(1, 901):
        bi.check_status(bi.adamw_step(st, g, t, **HYPER))
        if t % 60 == 0:
            codes, scale = st.exp_avg[0].float().cpu().double(), st.exp_avg_scale[0].cpu().double()
            if float(scale) == 0:
                assert torch.all(codes == 0)
            else:
                assert torch.equal(codes, first), t
    assert float(scale) == 0


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 1e25])
def test_elements_that_are_not_finite_stay_their_own(bad, cuda_device):
    """One gradient of a block is infinite, NaN or has an infinite square: the block's other elements have the
    bits of a block whose element has no gradient, in that step and in later ones.  (1e25 is a finite m and the
    block's maximum, before which the others vanish; they stay finite.)"""
    gen = torch.Generator().manual_seed(2)
    n, at = 600, [5, 300]
    grads = [torch.randn(n, generator=gen) * 1e-3 for _ in range(4)]
    w = torch.randn(n, generator=gen)
    runs = []
    for worst in (0.0, bad):
        st = bi.AdamWState.allocate([w.clone().to(cuda_device)], state_bits=8)
        for t, g in enumerate(grads, 1):
            g = g.clone()
            g[at] = worst if t == 2 else 0.0
            bi.check_status(bi.adamw_step(st, [g.to(cuda_device)], t, **HYPER))
        runs.append([st.params[0].cpu(), st.exp_avg[0].cpu().float(), st.exp_avg_sq[0].cpu().float(),
                     st.exp_avg_scale[0].cpu(), st.exp_avg_sq_scale[0].cpu()])
    keep = torch.ones(n, dtype=torch.bool)
    keep[at] = False
    for a, b in zip(*runs):
        k = keep if a.numel() == n else slice(None)
        assert torch.isfinite(b[k]).all()
        assert bad == 1e25 or torch.equal(a[k], b[k])
    assert torch.isnan(runs[1][2][at]).all()
