"""The AdamW step against the fp64 oracle and against the same fp32 operations in torch, over its
types, odd sizes and addresses, graphs, and the 8-bit states' format.

Tolerances (u = 2^-24): with the hyper-parameters' factors rounded once,
* m = b1 m + c1 g: a factor, a product and the sum round: 3 u (|b1 m| + |c1 g|) (one more with a scale);
* v: 5 u v;
* the update u = m rate / (sqrt(v) root + eps): den is within 8 u, the quotient within 12 u of |u|
  and what m's error gives; p: 3 u |p| + 13 u |u| + rate / den times m's bound; bf16: 2^-8 |p| more.
"""
import itertools

import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 255, 256, 257, 4096, 4097, 12345, 70001]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def _f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def _quantise(x, positive):
    """The 8-bit format, on the CPU in fp32: (codes, scales)."""
    n = x.numel()
    b = torch.zeros(-(-n // 256) * 256)
    b[:n] = x
    b = b.view(-1, 256)
    most = b.abs().amax(1)
    inv = torch.where(most > 0, most.reciprocal() * 448.0, 0.0)
    y = b * inv[:, None]
    if positive:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).view(-1)[:n].clone(), most * torch.tensor(1 / 448.0)


def _widen(codes, scale):
    return codes.float() * scale.repeat_interleave(256)[:codes.numel()]


def _make(sizes, ptype, master, gtype, bits, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda n, s: torch.randn(n, generator=gen) * s  # noqa: E731
    d = dict(p=[], master=[] if master else None, g=[], m=[], v=[], ms=[] if bits == 8 else None,
             vs=[] if bits == 8 else None)
    for n in sizes:
        w = r(n, 0.02)
        d["p"].append(w.to(ptype))
        if master:
            d["master"].append(w.clone())
        g = r(n, 3e-3)
        if n > 20:
            g[3] = 0.0
        d["g"].append(g.to(gtype))
        m, v = r(n, 1e-3), torch.rand(n, generator=gen) * 1e-5
        if n > 300:
            m[256:] *= 1e-6
            v[256:] *= 1e-9
            v[300] = 0.0
        if bits == 32:
            d["m"].append(m)
            d["v"].append(v)
        else:
            for x, c, s, pos in ((m, "m", "ms", False), (v.sqrt(), "v", "vs", True)):
                codes, scale = _quantise(x, pos)
                d[c].append(codes)
                d[s].append(scale)
    return d


def _sqrt(x):
    """Correctly rounded (torch's CPU square root is not): the fp64 root of an fp32 value, rounded."""
    return x.double().sqrt().float()


def _plain(d, i, step, gs=None):
    """The documented fp32 operations, one torch operation each, on the CPU."""
    f = lambda x: torch.tensor(x, dtype=torch.float64).float()  # noqa: E731
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    rate, root = f(HYPER["lr"] / (1 - b1 ** step)), f(1 / np.sqrt(1 - b2 ** step))
    keep = f(1 - HYPER["lr"] * HYPER["weight_decay"])
    g = d["g"][i].float()
    if gs is not None:
        g = g * torch.tensor(gs)
    if d["ms"] is None:
        m, v = d["m"][i], d["v"][i]
    else:
        m, v = _widen(d["m"][i], d["ms"][i]), _widen(d["v"][i], d["vs"][i])
        v = v * v
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    w = d["master"][i] if d["master"] is not None else d["p"][i].float()
    w = w * keep - (m * rate) / (_sqrt(v) * root + f(HYPER["eps"]))
    return w, m, v


def _state(d, dev):
    c = lambda ts: None if ts is None else [t.to(dev) for t in ts]  # noqa: E731
    return bi.AdamWState(c(d["p"]), c(d["master"]), c(d["m"]), c(d["v"]), c(d["ms"]), c(d["vs"])), c(d["g"])


def _check(d, st, step, gs=None):
    for i in range(len(d["p"])):
        w, m, v = _plain(d, i, step, gs)
        got_p = st.params[i].cpu()
        if st.masters is not None:
            assert torch.equal(st.masters[i].cpu(), w)
        assert torch.equal(got_p, w.to(got_p.dtype))
        if st.state_bits == 32:
            assert torch.equal(st.exp_avg[i].cpu(), m) and torch.equal(st.exp_avg_sq[i].cpu(), v)
        else:
            for x, pos, codes, scale in ((m, False, st.exp_avg[i], st.exp_avg_scale[i]),
                                         (_sqrt(v), True, st.exp_avg_sq[i], st.exp_avg_sq_scale[i])):
                c, s = _quantise(x, pos)
                assert torch.equal(scale.cpu(), s)
                assert torch.equal(codes.cpu().view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("ptype,master,gtype,bits", [
    (p, ma, g, b) for (p, ma), g, b in itertools.product(
        [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)],
        [torch.float32, torch.bfloat16], [32, 8])])
def test_step_has_the_documented_operations_bits(ptype, master, gtype, bits, cuda_device):
    d = _make(SIZES, ptype, master, gtype, bits, seed=bits)
    st, g = _state(d, cuda_device)
    status = bi.adamw_step(st, g, 3, **HYPER)
    torch.cuda.synchronize()
    bi.check_status(status)
    _check(d, st, 3)


def test_step_matches_oracle(cuda_device):
    d = _make(SIZES, torch.float32, False, torch.float32, 32, seed=1)
    st, g = _state(d, cuda_device)
    for step in (1, 1000):
        before = [(_f64(a), _f64(b), _f64(c)) for a, b, c in zip(st.params, st.exp_avg, st.exp_avg_sq)]
        bi.check_status(bi.adamw_step(st, g, step, **HYPER))
        for i, (p, m, v) in enumerate(before):
            rp, rm, rv, u, den = ao.adamw(p, d["g"][i], m, v, step, **HYPER)
            bm = 3 * U * (np.abs(HYPER["beta1"] * m) + np.abs((1 - HYPER["beta1"]) * _f64(d["g"][i])))
            rate = HYPER["lr"] / (1 - HYPER["beta1"] ** step)
            bp = 3 * U * np.abs(rp) + 13 * U * np.abs(u) + rate / den * bm
            # zero states and gradients apart, v is normal: 1e-14 at the least here
            assert np.all(np.abs(_f64(st.exp_avg[i]) - rm) <= bm + 1e-44)
            assert np.all(np.abs(_f64(st.exp_avg_sq[i]) - rv) <= 5 * U * rv + 1e-44)
            assert np.all(np.abs(_f64(st.params[i]) - rp) <= bp + 2 * U * np.abs(p))


def test_eight_bit_format_error(cuda_device):
    """A held value is within half a step of e4m3 of the value itself: 2^-4 relative, or half of the
    smallest step, 2^-10, of the block's scale; a sqrt(v) above zero is held above zero."""
    d = _make([100000], torch.bfloat16, True, torch.float32, 8, seed=4)
    d["g"][0][:256] = 0
    d["g"][0][5] = 1e-12
    d["m"][0] = torch.zeros(100000, dtype=torch.uint8).view(torch.float8_e4m3fn)
    d["v"][0] = torch.zeros(100000, dtype=torch.uint8).view(torch.float8_e4m3fn)
    st, g = _state(d, cuda_device)
    bi.check_status(bi.adamw_step(st, g, 1, **HYPER))
    g64 = _f64(d["g"][0])
    for codes, scale, ref in ((st.exp_avg[0], st.exp_avg_scale[0], 0.1 * g64),
                              (st.exp_avg_sq[0], st.exp_avg_sq_scale[0], np.sqrt(0.05) * np.abs(g64))):
        got = _f64(_widen(codes.cpu(), scale.cpu()))
        s = _f64(scale).repeat(256)[:got.size]
        low = np.where(np.abs(ref) > 0, 2.0 ** -9, 2.0 ** -10) * s  # raised to the smallest code
        assert np.all(np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), low) * (1 + 2.0 ** -20))
    root = _f64(st.exp_avg_sq[0].float())
    assert np.all((root > 0) == (g64 != 0))


@pytest.mark.parametrize("bits", [32, 8])
def test_odd_addresses_and_many_tensors(bits, cuda_device):
    """Views at odd elements (no vector access), tensors without elements, and more tensors than one
    launch takes."""
    sizes = [0, 300, 1, 5000] + [3, 40, 0] * 300
    d = _make(sizes, torch.bfloat16, True, torch.float32, bits, seed=9)
    total = sum(sizes)

    def packed(ts, dtype, pad=1):
        flat = torch.zeros(total + pad * len(sizes) + 1, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                           device=cuda_device)
        flat = flat.view(dtype) if dtype == torch.float8_e4m3fn else flat
        out, at = [], 1
        for t in ts:
            v = flat[at:at + t.numel()]
            v.view(torch.uint8 if dtype == torch.float8_e4m3fn else dtype).copy_(
                t.view(torch.uint8 if dtype == torch.float8_e4m3fn else dtype))
            out.append(v)
            at += t.numel() + pad
        return out

    held = torch.float32 if bits == 32 else torch.float8_e4m3fn
    c = lambda ts: None if ts is None else [t.to(cuda_device) for t in ts]  # noqa: E731
    st = bi.AdamWState(packed(d["p"], torch.bfloat16), packed(d["master"], torch.float32), packed(d["m"], held),
                       packed(d["v"], held), c(d["ms"]), c(d["vs"]))
    status = bi.adamw_step(st, packed(d["g"], torch.float32), 5, **HYPER)
    torch.cuda.synchronize()
    bi.check_status(status)
    _check(d, st, 5)


def test_graph_replays_with_a_device_step_and_a_gradient_scale(cuda_device):
    d = _make([1000, 77], torch.bfloat16, True, torch.bfloat16, 32, seed=6)
    st, g = _state(d, cuda_device)
    eager, g2 = _state(d, cuda_device)
    step = torch.ones(1, dtype=torch.int64, device=cuda_device)
    scale = torch.tensor([0.5], device=cuda_device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status = bi.adamw_step(st, g, step, grad_scale=scale, **HYPER)
    for t in (1, 2, 3):
        step.fill_(t)
        scale.fill_(0.25 * t)
        graph.replay()
        bi.check_status(bi.adamw_step(eager, g2, t, grad_scale=scale, **HYPER))
        for a, b in zip(st.tensors(), eager.tensors()):
            assert torch.equal(a, b)
    bi.check_status(status)
    step.fill_(0)  # no such step: refused on the device, nothing is touched
    graph.replay()
    with pytest.raises(bi.BiError, match="INVALID_ARG"):
        bi.check_status(status)
    for a, b in zip(st.tensors(), eager.tensors()):
        assert torch.equal(a, b)


def test_nonfinite_gradients_stay_in_their_elements(cuda_device):
    d = _make([600], torch.float32, False, torch.float32, 32, seed=12)
    clean, g = _state(d, cuda_device)
    bi.adamw_step(clean, g, 2, **HYPER)
    d["g"][0][100] = float("nan")
    d["g"][0][101] = float("inf")
    st, g = _state(d, cuda_device)
    bi.adamw_step(st, g, 2, **HYPER)
    ok = torch.ones(600, dtype=torch.bool, device=cuda_device)
    ok[100:102] = False
    assert torch.equal(st.params[0][ok], clean.params[0][ok]) and not torch.isfinite(st.params[0][~ok]).any()


def test_allocated_state_and_refusals(cuda_device):
    p = [torch.randn(40, 3, device=cuda_device).to(torch.bfloat16)]
    st = bi.AdamWState.allocate(p, state_bits=8, master=True)
    g = [torch.randn(40, 3, device=cuda_device)]
    bi.check_status(bi.adamw_step(st, g, 1, 1e-3))
    assert torch.equal(p[0], st.masters[0].to(torch.bfloat16))
    with pytest.raises(ValueError, match="overlap"):
        bi.AdamWState([p[0], p[0]], None, [x.float() for x in p * 2], [x.float() for x in p * 2])
    with pytest.raises(ValueError, match="shape"):
        bi.adamw_step(st, [g[0].t().contiguous()], 1, 1e-3)
    with pytest.raises(bi.BiError):
        bi.adamw_step(st, g, 0, 1e-3)
    with pytest.raises(bi.BiError):
        bi.adamw_step(st, g, 1, 1e-3, beta1=1.0)


def test_a_replaced_storage_is_followed(cuda_device):
    """``param.data = ...`` between two steps: the new storage is updated, the old one left alone; one of
    another size or type is refused."""
    d = _make([300, 1000], torch.float32, False, torch.float32, 32, seed=5)
    st, g = _state(d, cuda_device)
    old = st.params[1].data
    fresh = old.clone()
    st.params[1].data = fresh
    kept = old.clone()
    bi.check_status(bi.adamw_step(st, g, 3, **HYPER))
    assert torch.equal(old, kept) and st.params[1].data_ptr() == fresh.data_ptr()
    _check(d, st, 3)
    st.params[0].data = torch.zeros(299, device=cuda_device)
    with pytest.raises(ValueError):
        bi.adamw_step(st, g, 4, **HYPER)


@pytest.mark.parametrize("count", [16, 17, 96, 97, 440, 441])
def test_as_many_tensors_as_a_launch_takes_and_one_more(count, cuda_device):
    d = _make([1 + 7 * (i % 40) for i in range(count)], torch.bfloat16, True, torch.bfloat16, 8, seed=count)
    st, g = _state(d, cuda_device)
    bi.check_status(bi.adamw_step(st, g, 3, **HYPER))
    _check(d, st, 3)
