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


def bits(n, t):
    """The documented 32 bits of elements 0 .. n - 1 at step t."""
    M = 0xffffffff
    i = np.arange(n, dtype=np.uint64)
    x = ((i & M) * 0x9E3779B9 + (i >> np.uint64(32)) * 0x510E527F + (t & M) * 0x6A09E667 + (t >> 32) * 0x1F83D9AB) & M
    x ^= x >> np.uint64(16)
    x = (x * 0xBB67AE85) & M
    x ^= x >> np.uint64(15)
    x = (x * 0x9B05688D) & M
    return torch.from_numpy((x ^ (x >> np.uint64(16))).astype(np.int64))


def hold_dithered(x, root, r):
    """As hold(), rounded by r (0 .. 65535)."""
    most = x.abs().amax(1)
    inv = most.reciprocal() * 448.0
    gone = torch.isinf(inv)
    inv, most = torch.where(gone, 0.0, inv), torch.where(gone, 0.0, most)
    y = x * inv[:, None]
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    exponent = torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 1  # |y| in [2^e, 2^(e + 1))
    spacing = torch.ldexp(torch.ones_like(y), exponent - 3)
    c = torch.floor(y.abs() / spacing + r.float() / 65536) * spacing
    return torch.copysign(c, y).to(torch.float8_e4m3fn).float(), most * torch.tensor(1 / 448.0)


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.95, 0.95), (0.95, 0.99), (17 / 18, 0.96)])
@pytest.mark.parametrize("step", [1, 7, (1 << 33) + 5])
def test_dithered_codes_are_the_documented_ones(beta1, beta2, step, cuda_device):
    gen = torch.Generator().manual_seed(3)
    n = 70 * 256
    p, grad = torch.randn(70, 256, generator=gen), torch.randn(70, 256, generator=gen) * 3e-3
    m, root = torch.randn(70, 256, generator=gen) * 1e-3, torch.rand(70, 256, generator=gen) * 3e-3
    m[3] *= torch.logspace(0, -7, 256)
    root[3] *= torch.logspace(0, -7, 256)
    root[4] = 0.0
    grad[4, ::2] = 0.0
    m[5] = grad[5] = 0.0
    st = state(p, m, root, cuda_device)
    (cm, sm), (cv, sv) = hold(m, False), hold(root, True)
    bi.check_status(bi.adamw_step(st, [grad.to(cuda_device)], step, 1e-3, beta1=beta1, beta2=beta2))
    f = lambda x: torch.tensor(x, dtype=torch.float64).float()  # noqa: E731
    v = cv * sv[:, None]
    m = (cm * sm[:, None]) * f(beta1) + grad * f(1 - beta1)
    v = _sqrt((v * v) * f(beta2) + (grad * grad) * f(1 - beta2))
    r = bits(n, step).view(70, 256)
    for x, pos, dither, part, codes, scale in (
            (m, False, beta1 > 17 / 18, r & 0xffff, st.exp_avg[0], st.exp_avg_scale[0]),
            (v, True, beta2 > 0.96, r >> 16, st.exp_avg_sq[0], st.exp_avg_sq_scale[0])):
        c, s = hold_dithered(x, pos, part) if dither else hold(x, pos)
        assert torch.equal(scale.cpu(), s) and torch.equal(codes.cpu().float(), c)
        # a code next to the value: within a whole step of e4m3, not half
        assert torch.all((c * s[:, None] - x).abs() <= torch.maximum(2.0 ** -3 * x.abs(), 2.0 ** -9 * s[:, None]) * (1 + 2.0 ** -18))


@pytest.mark.parametrize("beta2,steps", [(0.95, 400), (0.96, 400), (0.99, 1000), (0.999, 4000)])
def test_sqrt_v_follows_the_gradients(beta2, steps, cuda_device):
    """Gradients change their scales; `steps` later the held sqrt(v) is set against that of 32-bit states.

    Scatter, dithered: a step moves sqrt(v), and the grid under it with the block's maximum, by c = (1 - b2) / 2
    |g^2 / v - 1| each, E|g^2 / v - 1| = 0.97; rounding a move of c on codes d apart (relative, 1/8 at most) has the
    variance d c at most, and a deviation goes back by 1 - b2 a step: variance d 2 (0.97 (1 - b2) / 2) /
    (2 (1 - b2)) = 0.06, deviation 0.25.  10% and 90% of the elements are 1.28 deviations out, 1% and 99% 2.33, on a
    distribution between a normal and a log-normal one: 0.68 .. 1.37 and 0.42 .. 1.77; the median within d / 2."""
    gen = torch.Generator(device=cuda_device).manual_seed(4)
    n = 1 << 16
    scales = torch.exp(torch.randn(2, n, generator=gen, device=cuda_device))
    p = [torch.zeros(n, device=cuda_device) for _ in range(2)]
    held, true = (bi.AdamWState.allocate([x], state_bits=b) for x, b in zip(p, (8, 32)))
    for t in range(1, 2 * steps + 1):
        g = [torch.randn(n, generator=gen, device=cuda_device) * scales[int(t > steps)]]
        for st in (held, true):
            s = bi.adamw_step(st, g, t, 1e-3, beta2=beta2)
    bi.check_status(s)
    ratio = held.exp_avg_sq[0].float().view(-1, 256) * held.exp_avg_sq_scale[0][:, None]
    ratio = (ratio.view(-1) / true.exp_avg_sq[0].sqrt()).cpu()
    q = torch.quantile(ratio, torch.tensor([0.01, 0.1, 0.5, 0.9, 0.99]))
    low, high = torch.tensor([0.42, 0.68, 0.9375, 0.68, 0.42]), torch.tensor([1.77, 1.37, 1.0625, 1.37, 1.77])
    assert torch.all(q >= low) and torch.all(q <= high), q.tolist()


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.98])
def test_m_of_elements_without_gradients_decays(beta1, cuda_device):
    """A quarter of each block's elements lose their gradients while the others keep the block's scale.  The mean
    square of a dithered m shrinks by beta1^2 + (1 - beta1) / 8 a step (its own move and the rounding's variance), to
    nearest by less than (17/18)^2 between codes; both end at a few of the smallest codes, 2^-9 of 448."""
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    n = 1 << 14
    st = bi.AdamWState.allocate([torch.zeros(n, device=cuda_device)], state_bits=8)
    for t in range(1, 701):
        g = torch.randn(n, generator=gen, device=cuda_device)
        if t > 200:
            g[::4] = 0.0
        s = bi.adamw_step(st, [g], t, 1e-3, beta1=beta1, beta2=0.95)
        if t == 200:
            first = (st.exp_avg[0].float().view(-1, 256) * st.exp_avg_scale[0][:, None]).view(-1)[::4].square().mean()
    bi.check_status(s)
    last = (st.exp_avg[0].float().view(-1, 256) * st.exp_avg_scale[0][:, None]).view(-1)[::4].square().mean()
    # 0.9629^500 = 6e-9 for beta1 = 0.98; four smallest codes of a maximum of 4 deviations: (4 2^-9 4 / 448)^2 = 5e-9
    assert float(last / first) < 1e-6


def test_dither_in_a_replayed_graph_and_among_other_tensors(cuda_device):
    """With the step on the device, captured once, and with another tensor in front: the same bits."""
    gen = torch.Generator().manual_seed(6)
    p, g = torch.randn(1000, generator=gen).to(cuda_device), torch.randn(1000, generator=gen).to(cuda_device)
    extra = torch.ones(300, device=cuda_device)
    one = bi.AdamWState.allocate([p.clone()], state_bits=8)
    two = bi.AdamWState.allocate([extra.clone(), p.clone()], state_bits=8)
    live = bi.AdamWState.allocate([p.clone()], state_bits=8)
    step = torch.ones(1, dtype=torch.int64, device=cuda_device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status = bi.adamw_step(live, [g], step, 1e-3)
    for t in range(1, 30):
        step.fill_(t)
        graph.replay()
        bi.adamw_step(one, [g], t, 1e-3)
        bi.adamw_step(two, [extra, g], t, 1e-3)
        for a, b, c in zip(one.tensors(), live.tensors(), two.tensors()[1::2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    bi.check_status(status)
