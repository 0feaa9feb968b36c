"""The gradient of softmax attention against the fp64 oracle: lengths, head groups, masks that leave rows
and keys empty, strides, bits, streams and graphs.

Tolerances, from the arithmetic (u = 2^-24; a rounding to bf16 is off by at most 2^-8; d as in the forward's
tests: (D + 4) u s_abs + 2^-16):
* p = exp2(c s - lse log2 e): d for the score and the exponential, lse itself is off by
  d + n u + 2^-22 (1 + |lse|) and its product by u |lse| log2 e: e_p = 2 d + n u + 2^-21 (1 + |lse|).
* dv: p is rounded (2^-8), m fp32 additions (m 2^-23), dv is rounded:
  (2^-8 + e_p + m 2^-23) sum p |do| + 2^-8 |dv|.
* ds = p (dp - delta): dp within (D + 4) u |do| |v|; delta from the rounded out, which is off by
  (2^-8 + 3 d + n 2^-23) sum p |v| + 2^-8 |out|, and a sum of D products; ds is rounded.  Relative to the sum
  of all terms' magnitudes A = p (|do| |v| + sum p |do| |v|):
  e_s = e_p + 3 2^-8 + 3 d + n 2^-23 + (2 D + 8) u;   dq, dk: (e_s + m 2^-23) sum A |k or q| + 2^-8 |result|.
Compounded: factor 1 + 2^-5.
"""
import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from oracle import attn_oracle as ao
from tests.test_gpu_attention import U, _f64, _offs, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


def check_bwd(q, k, v, dout, seqs, causal, scale, dq, dk, dv):
    D = q.shape[-1]
    r = ao.attention(q, k, v, seqs, causal, scale, dout=dout)
    n = max([s[3] for s in seqs] + [1])
    m = max([s[1] for s in seqs] + [1]) * (q.shape[1] // k.shape[1])
    qr = np.concatenate([np.arange(s[0], s[0] + s[1]) for s in seqs]).astype(int)
    kr = np.concatenate([np.arange(s[2], s[2] + s[3]) for s in seqs]).astype(int)
    d = (D + 4) * U * (r["s_abs"][:, qr].max() if len(qr) else 0.0) + 2.0 ** -16
    lse = np.abs(r["lse"][:, qr])
    lse = lse[np.isfinite(lse)].max(initial=0.0)
    ep = 2 * d + n * U + 2.0 ** -21 * (1 + lse)
    es = ep + 3 * 2.0 ** -8 + 3 * d + n * 2.0 ** -23 + (2 * D + 8) * U
    for name, got, rows, e in (("dv", dv, kr, ep + 2.0 ** -8 + m * 2.0 ** -23), ("dk", dk, kr, es + m * 2.0 ** -23),
                               ("dq", dq, qr, es + n * 2.0 ** -23)):
        bound = (e * r[name + "_abs"] + 2.0 ** -8 * np.abs(r[name]))[rows] * (1 + 2.0 ** -5)
        err = np.abs(_f64(got) - r[name])[rows]
        assert np.all(err <= bound), (name, float(np.max(err / np.maximum(bound, 1e-300))))
        # the bound allows for the worst signs; as a whole the result is far nearer
        norm = np.sqrt((r[name][rows] ** 2).sum())
        assert np.sqrt((err ** 2).sum()) <= 2.0 ** -6 * norm + np.sqrt((bound ** 2).sum()) / 8, name
    return r


def _run(q, k, v, dout, qo, ko, causal, dev, scale=None, **kw):
    t = [x.to(dev) for x in (q, k, v)]
    args = dict(k_offsets=None if ko is None else ko.to(dev), causal=causal, scale=scale)
    if "k_lens" in kw:
        args["k_lens"] = kw.pop("k_lens").to(dev)
    out, lse, st = bi.attn_fwd(*t, qo.to(dev), **args)
    bi.check_status(st)
    dq, dk, dv, st = bi.attn_bwd(dout.to(dev), *t, out, lse, qo.to(dev), **args, **kw)
    torch.cuda.synchronize()
    bi.check_status(st)
    return dq, dk, dv


@pytest.mark.parametrize("lens,Hq,Hkv,D,causal", [
    ([1], 1, 1, 64, True), ([1], 12, 2, 128, True), ([5, 0, 3], 2, 1, 64, True), ([127], 1, 1, 128, True),
    ([128], 1, 1, 128, True), ([129], 1, 1, 128, False), ([257, 1, 64], 6, 1, 128, True), ([300, 41], 4, 4, 64, False),
    ([77, 500, 0, 130], 12, 2, 128, True), ([200], 128, 1, 64, True), ([333], 35, 5, 128, False),
    ([1000, 24], 8, 8, 64, True), ([700], 7, 1, 128, True), ([1500, 100], 1, 1, 128, True)])
def test_packed_matches_oracle(lens, Hq, Hkv, D, causal, cuda_device):
    T = sum(lens)
    x = _rand(T, Hq + 2 * Hkv, D, sum(lens) + Hq)
    dout = _rand(T, Hq, D, 99, 0.1)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    o = _offs(lens)
    xd = x.to(cuda_device)
    sl = (xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:])
    out, lse, st = bi.attn_fwd(*sl, o.to(cuda_device), causal=causal)
    bi.check_status(st)
    # gradients into the slices of one buffer, as the projection's gradient wants them
    g = torch.full_like(xd, float("nan"))
    _, _, _, st = bi.attn_bwd(dout.to(cuda_device), *sl, out, lse, o.to(cuda_device), causal=causal, dq=g[:, :Hq],
                              dk=g[:, Hq:Hq + Hkv], dv=g[:, Hq + Hkv:])
    torch.cuda.synchronize()
    bi.check_status(st)
    assert not torch.isnan(g.float()).any()
    check_bwd(q, k, v, dout, ao.sequences(o), causal, D ** -0.5, g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:])


def test_peaked_scores(cuda_device):
    x = _rand(400, 8, 128, 3)
    x[:, :4] *= 8
    q, k, v, o = x[:, :4].contiguous(), x[:, 4:6].contiguous(), x[:, 6:].contiguous(), _offs([400])
    dout = _rand(400, 4, 128, 4)
    got = _run(q, k, v, dout, o, None, True, cuda_device)
    check_bwd(q, k, v, dout, ao.sequences(o), True, 128 ** -0.5, *got)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,causal", [
    ([5], [3], 2, 1, 64, True), ([300], [100], 4, 1, 128, True), ([1, 2, 0, 4], [0, 300, 9, 500], 6, 2, 128, True),
    ([130], [900], 8, 2, 64, True), ([3], [0], 2, 2, 128, False), ([0, 0], [5, 200], 2, 2, 128, True),
    ([33, 1], [257, 600], 4, 1, 128, True), ([64], [200], 3, 3, 64, False)])
def test_keys_of_their_own_and_empty_rows(lq, lk, Hq, Hkv, D, causal, cuda_device):
    q, k, v = _rand(sum(lq), Hq, D, 1), _rand(sum(lk), Hkv, D, 2), _rand(sum(lk), Hkv, D, 3)
    dout = _rand(sum(lq), Hq, D, 5)
    qo, ko = _offs(lq), _offs(lk)
    got = _run(q, k, v, dout, qo, ko, causal, cuda_device)
    check_bwd(q, k, v, dout, ao.sequences(qo, ko), causal, D ** -0.5, *got)


def test_rows_around_a_sequence_may_hold_anything(cuda_device):
    """NaN in rows of no sequence, in cache rows behind the keys and in another sequence: they reach nothing."""
    dev = cuda_device
    Hq, Hkv, D = 6, 2, 128
    q, k, v, dout = _rand(300, Hq, D, 1), _rand(700, Hkv, D, 2), _rand(700, Hkv, D, 3), _rand(300, Hq, D, 4)
    qo, ko = torch.tensor([10, 90, 250]), torch.tensor([5, 350, 700])
    kl = torch.tensor([130, 300], dtype=torch.int32)
    for t, used in ((q, [(10, 250)]), (dout, [(10, 250)]), (k, [(5, 135), (350, 650)]), (v, [(5, 135), (350, 650)])):
        keep = torch.zeros(t.shape[0], dtype=torch.bool)
        for a, b in used:
            keep[a:b] = True
        t[~keep] = float("nan")
    outs = [torch.full(s, 3.0, dtype=torch.bfloat16, device=dev) for s in (q.shape, k.shape, k.shape)]
    dq, dk, dv = _run(q, k, v, dout, qo, ko, True, dev, k_lens=kl, dq=outs[0], dk=outs[1], dv=outs[2])
    for t, used in ((dq, [(10, 250)]), (dk, [(5, 135), (350, 650)]), (dv, [(5, 135), (350, 650)])):
        keep = torch.zeros(t.shape[0], dtype=torch.bool, device=dev)
        for a, b in used:
            keep[a:b] = True
        assert torch.all(t[~keep] == 3.0) and torch.isfinite(t[keep].float()).all()
    clean = lambda t: torch.nan_to_num(t.float()).to(torch.bfloat16)  # noqa: E731
    check_bwd(clean(q), clean(k), clean(v), clean(dout), ao.sequences(qo, ko, kl), True, D ** -0.5, dq, dk, dv)
    # a sequence's NaN stays its own
    q2 = q.clone()
    q2[20] = float("nan")
    eq, ek, ev = _run(q2, k, v, dout, qo, ko, True, dev, k_lens=kl)
    assert torch.equal(eq[90:250], dq[90:250]) and torch.equal(ek[350:650], dk[350:650])
    assert torch.equal(ev[350:650], dv[350:650]) and torch.isnan(ek[5:135].float()).any()


def test_a_sequence_has_the_same_bits_in_any_batch(cuda_device):
    dev = cuda_device
    lens = [300, 17, 900, 1500]
    Hq, Hkv, D = 12, 2, 128
    T = sum(lens)
    q, k, v, dout = _rand(T, Hq, D, 1), _rand(T, Hkv, D, 2), _rand(T, Hkv, D, 3), _rand(T, Hq, D, 4)
    o = _offs(lens)
    whole = _run(q, k, v, dout, o, None, True, dev)
    again = _run(q, k, v, dout, o, None, True, dev)
    assert all(torch.equal(a, b) for a, b in zip(whole, again))
    for i, n in enumerate(lens):
        r = slice(int(o[i]), int(o[i + 1]))
        one = _run(q[r], k[r], v[r], dout[r], torch.tensor([0, n]), None, True, dev)
        assert all(torch.equal(a, b[r]) for a, b in zip(one, whole))


def test_bad_offsets_write_nothing(cuda_device):
    dev = cuda_device
    q, k, v, dout = (_rand(200, h, 64, h).to(dev) for h in (4, 2, 2, 4))
    out, lse, _ = bi.attn_fwd(q, k, v, torch.tensor([0, 200], device=dev))
    g = [torch.full_like(t, 3.0) for t in (q, k, v)]
    for offs, kw in (([0, 100, 50], {}), ([0, 100, 201], {}), ([-1, 100, 200], {}),
                     ([0, 100, 200], dict(k_lens=torch.tensor([50, 101], dtype=torch.int32, device=dev)))):
        _, _, _, st = bi.attn_bwd(dout, q, k, v, out, lse, torch.tensor(offs, device=dev), dq=g[0], dk=g[1], dv=g[2],
                                  **kw)
        with pytest.raises(bi.BiError, match="BAD_OFFSETS"):
            bi.check_status(st)
        assert all(torch.all(t == 3.0) for t in g)
    for n in (0, 1):  # no sequences; one without tokens
        *_, st = bi.attn_bwd(dout[:0], q[:0], k[:0], v[:0], out[:0], lse[:, :0].contiguous(),
                             torch.zeros(n + 1, dtype=torch.int64, device=dev))
        bi.check_status(st)


def test_streams_and_a_graph_with_new_lengths(cuda_device):
    dev = cuda_device
    q, k, v, dout = (_rand(3000, h, 128, h).to(dev) for h in (6, 1, 1, 6))
    live = torch.tensor([0, 5, 2000, 3000], device=dev)

    def both():
        out, lse, _ = bi.attn_fwd(q, k, v, live)
        return bi.attn_bwd(dout, q, k, v, out, lse, live)

    ref = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    for new in ([0, 5, 2000, 3000], [0, 1500, 1501, 3000], [0, 0, 0, 3000]):
        live.copy_(torch.tensor(new, device=dev))
        g.replay()
        want = both()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        bi.check_status(held[3])


def test_many_short_sequences(cuda_device):
    """More sequences than the plan's threads, most of them empty or a few tokens long, forward and backward."""
    from tests.test_gpu_attention import check_fwd
    dev = cuda_device
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 5, (2600,), generator=gen).tolist()
    lens[7], lens[2599] = 300, 150
    Hq, Hkv, D = 3, 1, 64
    T = sum(lens)
    q, k, v, dout = _rand(T, Hq, D, 1), _rand(T, Hkv, D, 2), _rand(T, Hkv, D, 3), _rand(T, Hq, D, 4)
    o = _offs(lens)
    t = [x.to(dev) for x in (q, k, v)]
    out, lse, st = bi.attn_fwd(*t, o.to(dev))
    bi.check_status(st)
    check_fwd(q, k, v, ao.sequences(o), True, D ** -0.5, out, lse)
    dq, dk, dv, st = bi.attn_bwd(dout.to(dev), *t, out, lse, o.to(dev))
    bi.check_status(st)
    check_bwd(q, k, v, dout, ao.sequences(o), True, D ** -0.5, dq, dk, dv)


def test_one_query_over_a_long_cache(cuda_device):
    """35 chunks of keys joined, and their gradients."""
    from tests.test_gpu_attention import check_fwd
    dev = cuda_device
    q, k, v, dout = _rand(1, 4, 64, 1), _rand(70001, 1, 64, 2), _rand(70001, 1, 64, 3), _rand(1, 4, 64, 4)
    qo, ko = torch.tensor([0, 1]), torch.tensor([0, 70001])
    t = [x.to(dev) for x in (q, k, v)]
    out, lse, st = bi.attn_fwd(*t, qo.to(dev), k_offsets=ko.to(dev))
    bi.check_status(st)
    check_fwd(q, k, v, ao.sequences(qo, ko), True, 64 ** -0.5, out, lse)
    got = bi.attn_bwd(dout.to(dev), *t, out, lse, qo.to(dev), k_offsets=ko.to(dev))
    bi.check_status(got[3])
    check_bwd(q, k, v, dout, ao.sequences(qo, ko), True, 64 ** -0.5, *got[:3])
