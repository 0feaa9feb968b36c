"""Softmax attention against the fp64 oracle: lengths from none to several chunks of keys, head groups,
masks that leave rows empty, caches, and the bits of a row in a prefill, a decode step and any batch.

Tolerances, from the arithmetic (u = 2^-24; a rounding to bf16 is off by at most 2^-8):
* a score is a sum of D exact products in fp32: within (D + 4) u s_abs, s_abs = scale sum |q k|; the
  exponent's fma rounds (|x| <= 2^7 here: 2^-17) and ex2 is within 2^-21: relative error of a term
  d = (D + 4) u s_abs + 2^-16.
* the terms are rounded to bf16 (2^-8), n products are added in fp32 (n 2^-23), l has d as well, out is
  rounded: |error| <= (2^-8 + 3 d + n 2^-23) sum p |v| + 2^-8 |out|, the last two terms compounded
  (factor 1 + 2^-6).
* lse: d + n u for the sum, and its own rounding: d + n u + 2^-22 (1 + |lse|).
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


def _offs(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64)


def _rand(T, H, D, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=gen) * scale).to(torch.bfloat16)


def check_fwd(q, k, v, seqs, causal, scale, out, lse):
    D = q.shape[-1]
    r = ao.attention(q, k, v, seqs, causal, scale)
    n = max([s[3] for s in seqs] + [1])
    d = ((D + 4) * U * r["s_abs"] + 2.0 ** -16).T[..., None]
    bound = ((2.0 ** -8 + 3 * d + n * 2.0 ** -23) * r["out_abs"] + 2.0 ** -8 * np.abs(r["out"])) * (1 + 2.0 ** -6)
    rows = np.concatenate([np.arange(s[0], s[0] + s[1]) for s in seqs]).astype(int)
    err = np.abs(_f64(out) - r["out"])[rows]
    assert np.all(err <= bound[rows]), float(np.max(err / np.maximum(bound[rows], 1e-300)))
    got, ref = _f64(lse)[:, rows], r["lse"][:, rows]
    empty = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), empty)
    lb = d[..., 0].T[:, rows] + n * U + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, ref)))
    assert np.all(np.abs(np.where(empty, 0, got) - np.where(empty, 0, ref)) <= lb)
    return r


def _packed(lens, Hq, Hkv, D, causal, seed, dev, scale=None, qscale=1.0):
    T = sum(lens)
    x = _rand(T, Hq + 2 * Hkv, D, seed)
    x[:, :Hq] *= qscale
    xd = x.to(dev)
    o = _offs(lens)
    out, lse, st = bi.attn_fwd(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], o.to(dev), causal=causal, scale=scale)
    torch.cuda.synchronize()
    bi.check_status(st)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    check_fwd(q, k, v, ao.sequences(o), causal, D ** -0.5 if scale is None else scale, out, lse)
    return out, lse


@pytest.mark.parametrize("lens,Hq,Hkv,D,causal", [
    ([1], 1, 1, 64, True), ([1], 12, 2, 128, True), ([5, 0, 3], 2, 1, 64, True), ([127], 1, 1, 128, True),
    ([128], 1, 1, 128, True), ([129], 1, 1, 128, True), ([257, 1, 64], 6, 1, 128, True), ([300, 41], 4, 4, 64, False),
    ([77, 500, 0, 130], 12, 2, 128, True), ([200], 128, 1, 64, True), ([333], 35, 5, 128, False),
    ([1000, 24], 8, 8, 64, True), ([2048], 2, 1, 128, True), ([2049], 2, 2, 64, True), ([4500, 100], 1, 1, 128, True),
    ([2500], 3, 1, 64, False)])
def test_packed_matches_oracle(lens, Hq, Hkv, D, causal, cuda_device):
    _packed(lens, Hq, Hkv, D, causal, sum(lens) + Hq, cuda_device)


def test_peaked_scores(cuda_device):
    """Large scores: the reference has to rise many times, most terms underflow."""
    _packed([700], 4, 2, 128, True, 3, cuda_device, qscale=8.0)
    _packed([700], 4, 2, 64, False, 4, cuda_device, scale=0.9)


def _rising(T, H, D, dev):
    """Keys whose scores rise along the sequence, so that every tile raises the reference."""
    q = torch.zeros(T, H, D)
    q[:, :, 0] = 4.0
    k = _rand(T, H, D, 5).float() * 0.1
    k[:, :, 0] = torch.arange(T)[:, None] / 32.0
    return q.to(torch.bfloat16), k.to(torch.bfloat16), _rand(T, H, D, 6)


def test_reference_rises_with_every_tile(cuda_device):
    q, k, v = _rising(1500, 2, 128, cuda_device)
    o = _offs([1500])
    out, lse, st = bi.attn_fwd(q.to(cuda_device), k.to(cuda_device), v.to(cuda_device), o.to(cuda_device), scale=1.0)
    torch.cuda.synchronize()
    bi.check_status(st)
    check_fwd(q, k, v, ao.sequences(o), True, 1.0, out, lse)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,causal", [
    ([5], [3], 2, 1, 64, True), ([300], [100], 4, 1, 128, True), ([1, 2, 0, 4], [0, 700, 9, 2100], 6, 2, 128, True),
    ([130], [900], 8, 2, 64, True), ([3], [0], 2, 2, 128, False), ([33, 1], [4097, 5000], 4, 1, 128, True)])
def test_keys_of_their_own_and_empty_rows(lq, lk, Hq, Hkv, D, causal, cuda_device):
    """More keys than queries (a prefix), fewer (rows that see nothing), none."""
    q, k, v = _rand(sum(lq), Hq, D, 1), _rand(sum(lk), Hkv, D, 2), _rand(sum(lk), Hkv, D, 3)
    qo, ko = _offs(lq), _offs(lk)
    dev = cuda_device
    out, lse, st = bi.attn_fwd(q.to(dev), k.to(dev), v.to(dev), qo.to(dev), k_offsets=ko.to(dev), causal=causal)
    torch.cuda.synchronize()
    bi.check_status(st)
    check_fwd(q, k, v, ao.sequences(qo, ko), causal, D ** -0.5, out, lse)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 12, 2), (64, 8, 8)])
def test_cache_decode_has_the_prefill_bits(D, Hq, Hkv, cuda_device):
    """Each query of a prefill, recomputed alone over a cache whose spare rows hold NaN (one or several
    chunks, split over SMs), among others and by itself: the same bits."""
    dev = cuda_device
    lens = [40, 2047, 2048, 2049, 4500, 6200]
    T = sum(lens)
    q, k, v = (_rand(T, h, D, s).to(dev) for h, s in ((Hq, 1), (Hkv, 2), (Hkv, 3)))
    o = _offs(lens).to(dev)
    out, lse, st = bi.attn_fwd(q, k, v, o)
    bi.check_status(st)
    room = 6500
    kc = torch.full((room * len(lens), Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
    vc = kc.clone()
    for i, n in enumerate(lens):
        kc[i * room:i * room + n] = k[o[i]:o[i + 1]]
        vc[i * room:i * room + n] = v[o[i]:o[i + 1]]
    ko = torch.arange(len(lens) + 1, dtype=torch.int64, device=dev) * room
    gen = torch.Generator().manual_seed(0)
    for trial in range(4):
        at = [n - 1 if trial == 0 else int(torch.randint(0, n, (1,), generator=gen)) for n in lens]
        rows = torch.tensor([int(o[i]) + a for i, a in enumerate(at)], device=dev)
        kl = torch.tensor([a + 1 for a in at], dtype=torch.int32, device=dev)
        d, dl, st = bi.attn_fwd(q[rows].contiguous(), kc, vc, torch.arange(len(lens) + 1, device=dev), k_offsets=ko,
                                k_lens=kl)
        bi.check_status(st)
        assert torch.equal(d, out[rows]) and torch.equal(dl, lse[:, rows])
    # one sequence alone, and its last 9 queries together
    i = 5
    qs = q[o[i + 1] - 9:o[i + 1]].contiguous()
    one = torch.tensor([0, 9], device=dev)
    d, dl, st = bi.attn_fwd(qs, kc[i * room:], vc[i * room:], one, k_offsets=torch.tensor([0, room], device=dev),
                            k_lens=torch.tensor([lens[i]], dtype=torch.int32, device=dev))
    bi.check_status(st)
    assert torch.equal(d, out[o[i + 1] - 9:o[i + 1]]) and torch.equal(dl, lse[:, o[i + 1] - 9:o[i + 1]])


def test_rows_do_not_depend_on_the_batch(cuda_device):
    dev = cuda_device
    lens = [300, 17, 900, 2500]
    x = _rand(sum(lens), 12 + 4, 128, 11).to(dev)
    o = _offs(lens).to(dev)
    sl = lambda y: (y[:, :12], y[:, 12:14], y[:, 14:])  # noqa: E731
    out, lse, _ = bi.attn_fwd(*sl(x), o)
    for i in range(len(lens)):
        y = x[o[i]:o[i + 1]].contiguous()
        a, b, st = bi.attn_fwd(*sl(y), torch.tensor([0, lens[i]], device=dev))
        bi.check_status(st)
        assert torch.equal(a, out[o[i]:o[i + 1]]) and torch.equal(b, lse[:, o[i]:o[i + 1]])
    # one sequence's NaN stays its own
    x[int(o[1]) + 3] = float("nan")
    out2, lse2, _ = bi.attn_fwd(*sl(x), o)
    keep = torch.ones(sum(lens), dtype=torch.bool, device=dev)
    keep[o[1]:o[2]] = False
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
    assert torch.isnan(out2[o[1] + 3:o[2]].float()).all()


def test_rows_in_no_sequence_and_bad_offsets(cuda_device):
    dev = cuda_device
    q, k, v = (_rand(200, h, 64, h).to(dev) for h in (4, 2, 2))
    out = torch.full((200, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((4, 200), 3.0, device=dev)
    _, _, st = bi.attn_fwd(q, k, v, torch.tensor([10, 60, 150], device=dev), out=out, lse=lse)
    bi.check_status(st)
    for rest in (out[:10], out[150:], lse[:, :10], lse[:, 150:]):
        assert torch.all(rest == 3.0)
    out.fill_(3.0)
    lse.fill_(3.0)
    for offs, kw in (([0, 100, 50], {}), ([0, 100, 201], {}), ([-1, 100, 200], {}),
                     ([0, 100, 200], dict(k_lens=torch.tensor([50, 101], dtype=torch.int32, device=dev))),
                     ([0, 100, 200], dict(k_lens=torch.tensor([-1, 10], dtype=torch.int32, device=dev)))):
        _, _, st = bi.attn_fwd(q, k, v, torch.tensor(offs, device=dev), out=out, lse=lse, **kw)
        with pytest.raises(bi.BiError, match="BAD_OFFSETS"):
            bi.check_status(st)
        assert torch.all(out == 3.0) and torch.all(lse == 3.0)
    # no sequences, no queries
    _, _, st = bi.attn_fwd(q, k, v, torch.tensor([0], device=dev), out=out, lse=lse)
    bi.check_status(st)
    e, _, st = bi.attn_fwd(q[:0], k[:0], v[:0], torch.tensor([0, 0], device=dev))
    bi.check_status(st)
    assert e.shape == (0, 4, 64)


def test_streams_and_a_graph_with_new_lengths(cuda_device):
    dev = cuda_device
    q, k, v = (_rand(5000, h, 128, h).to(dev) for h in (6, 1, 1))
    offs = torch.tensor([0, 5, 4000, 5000], device=dev)
    ref = bi.attn_fwd(q, k, v, offs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = bi.attn_fwd(q, k, v, offs)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ref[0], other[0]) and torch.equal(ref[1], other[1])
    live = offs.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bi.attn_fwd(q, k, v, live)
    for new in ([0, 5, 4000, 5000], [0, 2500, 2501, 5000], [0, 0, 0, 5000]):
        live.copy_(torch.tensor(new, device=dev))
        g.replay()
        want = bi.attn_fwd(q, k, v, live)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        bi.check_status(out[2])
