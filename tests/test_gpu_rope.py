"""The per-head RMS norm with rotation and its gradient against the fp64 oracle, row by row
independence, and what the entry points allow: slices of a projection, partial rotation, no norm,
far positions, the smallest and odd sizes, graphs and streams.

Tolerances, from the arithmetic (u = 2^-24, fp32; a rounding to bf16 is off by at most 2^-8):
* z: the sum of D squares is within D u (relative), so r within (D / 2 + 4) u; a product more for the
  gain; the angle's remainder and sincospif within 4 u absolute; each of the two products of a
  rotated pair and their sum a rounding.  |error| <= 2^-8 |z| + (D + 32) u (|y_i| + |y_i'|).
* dx = r (dn - n mean(dn n)): the same pieces, the mean within D u of its absolute terms:
  |error| <= 2^-8 |dx| + (2 D + 64) u r (|dn|_pair + |n| mean |dn n|).
* dg: N = T heads terms in fp32 in any order: |error| <= (N + D + 64) u sum |dy n|, |dy| by its pair.
"""
import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def _f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def _inputs(T, Hq, Hkv, D, R, seed, far=4096, sliced=True):
    gen = torch.Generator().manual_seed(seed)
    scale = torch.exp(torch.randn(1, Hq + Hkv, 1, generator=gen))
    x = (torch.randn(T, Hq + Hkv, D, generator=gen) * scale).to(torch.bfloat16)
    dz = torch.randn(T, Hq + Hkv, D, generator=gen).to(torch.bfloat16)
    gq, gk = (1 + 0.3 * torch.randn(2, D, generator=gen)).to(torch.bfloat16)
    pos = torch.randint(0, far, (T,), generator=gen, dtype=torch.int32)
    inv = (1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float()
    return x, dz, gq, gk, pos, inv


def _pair_abs(y, R):
    a = np.abs(y)
    h = R // 2
    s = a[..., :h] + a[..., h:R]
    return np.concatenate([s, s, a[..., R:]], -1)


def _check_fwd(x, g, pos, inv, eps, z):
    D = x.shape[-1]
    ref = ao.qk_norm_rope(x, g, pos, inv, eps)
    y, _ = ao.head_norm(x, g, eps)
    bound = 2.0 ** -8 * np.abs(ref) + (D + 32) * U * _pair_abs(y, 2 * len(inv)) * (1 + 2.0 ** -8)
    err = np.abs(_f64(z) - ref)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))


def _check_bwd(dz, x, g, pos, inv, eps, dx, dg):
    D, R = x.shape[-1], 2 * len(inv)
    ref, dgr = ao.qk_norm_rope_bwd(dz, x, g, pos, inv, eps)
    if g is None:
        bound = 2.0 ** -8 * np.abs(ref) + 16 * U * _pair_abs(_f64(dz), R)
    else:
        _, r = ao.head_norm(x, g, eps)
        n = _f64(x) * r
        dya = _pair_abs(_f64(dz), R)
        dna = dya * np.abs(_f64(g))
        bound = 2.0 ** -8 * np.abs(ref) + (2 * D + 64) * U * r * (dna + np.abs(n) * np.mean(dna * np.abs(n), -1, keepdims=True))
        gb = (x.shape[0] * x.shape[1] + D + 64) * U * (dya * np.abs(n)).sum((0, 1))
        gerr = np.abs(_f64(dg) - dgr)
        assert np.all(gerr <= gb), float(np.max(gerr / np.maximum(gb, 1e-300)))
    err = np.abs(_f64(dx) - ref)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))


def _run(dev, x, dz, gq, gk, pos, inv, Hq, eps, norm=True):
    c = lambda t: None if t is None else t.to(dev)  # noqa: E731
    x, dz = x.to(dev), dz.to(dev)
    gq, gk = (c(gq), c(gk)) if norm else (None, None)
    q, k = x[:, :Hq], x[:, Hq:]
    zq, zk, st = bi.qk_norm_rope(q, k, gq, gk, c(pos), c(inv), eps)
    dq, dk, dgq, dgk, st2 = bi.qk_norm_rope_bwd(dz[:, :Hq], dz[:, Hq:], q, k, gq, gk, c(pos), c(inv), eps)
    torch.cuda.synchronize()
    bi.check_status(st)
    bi.check_status(st2)
    return zq, zk, dq, dk, dgq, dgk


@pytest.mark.parametrize("T,Hq,Hkv,D,R,norm", [
    (1, 12, 2, 128, 128, True), (1, 1, 1, 16, 16, True), (5, 3, 1, 80, 32, True), (37, 6, 2, 64, 64, True),
    (130, 5, 5, 96, 48, True), (300, 32, 8, 128, 128, True), (9, 4, 4, 256, 256, True), (64, 7, 1, 32, 16, True),
    (33, 12, 2, 128, 64, False), (3000, 6, 2, 48, 48, True), (2500, 4, 2, 128, 128, False)])
def test_matches_oracle(T, Hq, Hkv, D, R, norm, cuda_device):
    x, dz, gq, gk, pos, inv = _inputs(T, Hq, Hkv, D, R, seed=T + D)
    eps = 1e-6
    zq, zk, dq, dk, dgq, dgk = _run(cuda_device, x, dz, gq, gk, pos, inv, Hq, eps, norm)
    if not norm:
        gq = gk = None
        assert dgq is None and dgk is None
    _check_fwd(x[:, :Hq], gq, pos, inv, eps, zq)
    _check_fwd(x[:, Hq:], gk, pos, inv, eps, zk)
    _check_bwd(dz[:, :Hq], x[:, :Hq], gq, pos, inv, eps, dq, dgq)
    _check_bwd(dz[:, Hq:], x[:, Hq:], gk, pos, inv, eps, dk, dgk)


@pytest.mark.parametrize("far", [1 << 20, 1 << 24, (1 << 31) - 1])
def test_far_positions_keep_their_phase(far, cuda_device):
    """Positions past 2^24, which fp32 cannot hold, and negative ones.  The fp64 angle in turns is
    off by at most two roundings, 2^-52 of |position| inv_freq / 2 pi: below 2^-24 for all of these."""
    x, dz, gq, gk, pos, inv = _inputs(64, 2, 1, 64, 64, seed=far & 1023)
    pos = torch.randint(far // 2, far, (64,), generator=torch.Generator().manual_seed(1), dtype=torch.int64).to(torch.int32)
    pos[::3] = -pos[::3]
    zq, zk, dq, dk, dgq, dgk = _run(cuda_device, x, dz, gq, gk, pos, inv, 2, 1e-6)
    _check_fwd(x[:, :2], gq, pos, inv, 1e-6, zq)
    _check_bwd(dz[:, 2:], x[:, 2:], gk, pos, inv, 1e-6, dk, dgk)


def test_gradient_against_differences(cuda_device):
    """The oracle's gradient (which the kernels are held to) against central differences of the oracle."""
    x, dz, gq, _, pos, inv = _inputs(3, 2, 1, 32, 32, seed=3)
    X, G, dZ = _f64(x), _f64(gq), _f64(dz)
    f = lambda a, b: float((ao.qk_norm_rope(a, b, pos, inv, 1e-5) * dZ).sum())  # noqa: E731
    dx, dg = ao.qk_norm_rope_bwd(dZ, X, G, pos, inv, 1e-5)
    rng = np.random.default_rng(0)
    for _ in range(20):
        i = tuple(rng.integers(0, s) for s in X.shape)
        e = np.zeros_like(X)
        e[i] = 1e-6
        assert abs((f(X + e, G) - f(X - e, G)) / 2e-6 - dx[i]) <= 1e-6 * (1 + abs(dx[i]))
        j = int(rng.integers(0, G.shape[0]))
        e = np.zeros_like(G)
        e[j] = 1e-6
        assert abs((f(X, G + e) - f(X, G - e)) / 2e-6 - dg[j]) <= 1e-6 * (1 + abs(dg[j]))


def test_rows_bitwise_independent_of_the_batch(cuda_device):
    """A token's outputs and input gradients have the same bits alone (a decode step) and among
    thousands, where a warp takes a token's heads together."""
    x, dz, gq, gk, pos, inv = _inputs(5000, 12, 2, 128, 128, seed=8)
    full = _run(cuda_device, x, dz, gq, gk, pos, inv, 12, 1e-6)
    for t in (0, 17, 4999):
        one = _run(cuda_device, x[t:t + 1], dz[t:t + 1], gq, gk, pos[t:t + 1], inv, 12, 1e-6)
        for a, b in zip(full[:4], one[:4]):
            assert torch.equal(a[t:t + 1], b)
    again = _run(cuda_device, x, dz, gq, gk, pos, inv, 12, 1e-6)
    for a, b in zip(full, again):
        assert torch.equal(a, b)


def test_empty_zero_rows_and_nonfinite_rows(cuda_device):
    x, dz, gq, gk, pos, inv = _inputs(6, 2, 1, 64, 64, seed=2)
    e = _run(cuda_device, x[:0], dz[:0], gq, gk, pos[:0], inv, 2, 1e-6)
    assert e[0].shape == (0, 2, 64) and torch.all(e[4] == 0) and torch.all(e[5] == 0)
    clean = _run(cuda_device, x, dz, gq, gk, pos, inv, 2, 1e-6)
    x[1] = 0
    x[3, 0, 5] = float("nan")
    out = _run(cuda_device, x, dz, gq, gk, pos, inv, 2, 1e-6)
    assert torch.all(out[0][1] == 0) and torch.isfinite(out[2][1].float()).all()
    assert torch.isnan(out[0][3, 0]).all()
    assert torch.equal(out[0][3, 1], clean[0][3, 1])  # the other heads and tokens are untouched
    assert torch.equal(out[0][4:], clean[0][4:]) and torch.equal(out[2][4:], clean[2][4:])


def test_strided_outputs_streams_and_graphs(cuda_device):
    """Outputs written into slices of one buffer (the rest left as it was), on another stream, and
    captured into a graph that is replayed with new inputs."""
    Hq, Hkv, D = 4, 2, 128
    x, dz, gq, gk, pos, inv = (t.to(cuda_device) for t in _inputs(50, Hq, Hkv, D, D, seed=5))
    q, k = x[:, :Hq], x[:, Hq:]
    zq, zk, _ = bi.qk_norm_rope(q, k, gq, gk, pos, inv, 1e-6)
    buf = torch.full((50, Hq + Hkv + 3, D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bi.qk_norm_rope(q, k, gq, gk, pos, inv, 1e-6, q_out=buf[:, 1:1 + Hq], k_out=buf[:, 2 + Hq:2 + Hq + Hkv])
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(buf[:, 1:1 + Hq], zq) and torch.equal(buf[:, 2 + Hq:2 + Hq + Hkv], zk)
    for rest in (buf[:, 0], buf[:, 1 + Hq], buf[:, 2 + Hq + Hkv:]):
        assert torch.all(rest == 7.0)
    ref = bi.qk_norm_rope_bwd(dz[:, :Hq], dz[:, Hq:], q, k, gq, gk, pos, inv, 1e-6)
    live = dz.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = bi.qk_norm_rope_bwd(live[:, :Hq], live[:, Hq:], q, k, gq, gk, pos, inv, 1e-6)
    live.zero_()
    g.replay()
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0)
    live.copy_(dz)
    g.replay()
    for a, b in zip(out, ref):
        assert torch.equal(a, b)
