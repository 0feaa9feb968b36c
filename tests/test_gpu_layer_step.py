"""The attention layer's operators and the update as a learner and a rollout engine use them together: norm
with rotation on a projection's slices, attention, its gradient, the gradient of the norm into the slices of
one buffer, and the step of the gains; eager, captured and replayed, on two streams at once, and a decode step
whose bits are the prefill's.  Every stage is held to its own tests' bounds, on the values that it got."""
import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from oracle import attn_oracle as ao
from tests.test_gpu_attention import _f64, _offs, _rand, check_fwd
from tests.test_gpu_attention_bwd import check_bwd
from tests.test_gpu_rope import _check_bwd, _check_fwd

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from async_rl_b200.build import build
    build()


class Layer:
    """One attention layer's training step on packed sequences."""

    def __init__(self, lens, Hq, Hkv, D, dev, seed):
        self.lens, self.Hq, self.Hkv, self.D = lens, Hq, Hkv, D
        T = sum(lens)
        self.x = _rand(T, Hq + 2 * Hkv, D, seed).to(dev)
        self.dout = _rand(T, Hq, D, seed + 1, 0.1).to(dev)
        gen = torch.Generator().manual_seed(seed + 2)
        self.gains = [(1 + 0.2 * torch.randn(D, generator=gen)).to(torch.bfloat16).to(dev) for _ in range(2)]
        self.opt = bi.AdamWState.allocate(self.gains, state_bits=32, master=True)
        self.pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(dev)
        self.inv = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(dev)
        self.offs = _offs(lens).to(dev)
        self.step = torch.ones(1, dtype=torch.int64, device=dev)

    def parts(self, t):
        a, b = self.Hq, self.Hq + self.Hkv
        return t[:, :a], t[:, a:b], t[:, b:]

    def run(self):
        q, k, v = self.parts(self.x)
        r = {}
        r["gains"] = [g.clone() for g in self.gains]
        r["q"], r["k"], s0 = bi.qk_norm_rope(q, k, *self.gains, self.pos, self.inv, EPS)
        r["out"], r["lse"], s1 = bi.attn_fwd(r["q"], r["k"], v, self.offs)
        r["dx"] = torch.empty_like(self.x)
        dq, dk, dv = self.parts(r["dx"])
        r["dq"], r["dk"], _, s2 = bi.attn_bwd(self.dout, r["q"], r["k"], v, r["out"], r["lse"], self.offs, dv=dv)
        _, _, r["dgq"], r["dgk"], s3 = bi.qk_norm_rope_bwd(r["dq"], r["dk"], q, k, *self.gains, self.pos, self.inv, EPS,
                                                           dq=dq, dk=dk)
        s4 = bi.adamw_step(self.opt, [r["dgq"], r["dgk"]], self.step, 1e-2)
        self.step += 1
        r["status"] = [s0, s1, s2, s3, s4]
        r["after"] = [g.clone() for g in self.gains]
        return r


def _same(a, b):
    if isinstance(a, list):
        return all(_same(x, y) for x, y in zip(a, b))
    return torch.equal(a.view(torch.uint8) if a.dtype == torch.bfloat16 else a,
                       b.view(torch.uint8) if b.dtype == torch.bfloat16 else b)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([130, 1, 65], 6, 2, 128), ([300], 4, 4, 64), ([1, 1, 1], 8, 1, 128)])
def test_every_stage_of_a_step(lens, Hq, Hkv, D, cuda_device):
    l = Layer(lens, Hq, Hkv, D, cuda_device, 7)
    r = l.run()
    torch.cuda.synchronize()
    for s in r["status"]:
        bi.check_status(s)
    c = lambda t: t.detach().cpu()  # noqa: E731
    q, k, v = (c(t) for t in l.parts(l.x))
    g, pos, inv = [c(t) for t in r["gains"]], c(l.pos), c(l.inv)
    for x, gain, z in ((q, g[0], r["q"]), (k, g[1], r["k"])):
        _check_fwd(x, gain, pos, inv, EPS, z)
    seqs = ao.sequences(c(l.offs))
    check_fwd(c(r["q"]), c(r["k"]), v, seqs, True, D ** -0.5, r["out"], r["lse"])
    dq, dk, dv = l.parts(r["dx"])
    check_bwd(c(r["q"]), c(r["k"]), v, c(l.dout), seqs, True, D ** -0.5, r["dq"], r["dk"], dv)
    for x, gain, dz, dx, dg in ((q, g[0], r["dq"], dq, r["dgq"]), (k, g[1], r["dk"], dk, r["dgk"])):
        _check_bwd(c(dz), x, gain, pos, inv, EPS, dx, dg)
    # first step from zero states: m / (1 - beta1) = g and sqrt(v / (1 - beta2)) = |g|, so that a gain moves by
    # lr g / (|g| + eps) and its decay (an update of at most lr, in a few fp32 roundings: 1e-6 is ample)
    for before, after, dg in zip(r["gains"], r["after"], (r["dgq"], r["dgk"])):
        g64 = _f64(dg)
        w = _f64(before) * (1 - 1e-2 * 0.01) - 1e-2 * g64 / (np.abs(g64) + 1e-8)
        assert np.all(np.abs(_f64(after) - w) <= 2.0 ** -8 * np.abs(w) + 1e-6)


def test_replays_and_two_streams_have_the_eager_bits(cuda_device):
    """Two layers of different shapes, each captured, replayed together on two streams; three steps each."""
    shapes = [([200, 31, 70], 12, 2, 128), ([150, 90], 8, 4, 64)]
    eager = []
    for i, s in enumerate(shapes):
        l = Layer(*s, cuda_device, 20 + i)
        eager.append([l.run() for _ in range(3)])
    torch.cuda.synchronize()
    layers = [Layer(*s, cuda_device, 20 + i) for i, s in enumerate(shapes)]
    graphs, held = [], []
    for l in layers:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(l.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in layers]
    for i in range(3):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for e, h in zip(eager, held):
            for key in e[i]:
                assert _same(e[i][key], h[key]), (i, key)


@pytest.mark.parametrize("Hq,Hkv,D", [(12, 2, 128), (8, 8, 64)])
def test_decode_step_has_the_prefill_bits(Hq, Hkv, D, cuda_device):
    """The last token of each sequence alone, its norm and rotation and its attention over the cache."""
    lens = [40, 1, 300, 2100]
    l = Layer(lens, Hq, Hkv, D, cuda_device, 3)
    r = l.run()
    l.gains[0].copy_(r["gains"][0])
    l.gains[1].copy_(r["gains"][1])
    last = l.offs[1:] - 1
    x = l.x[last].contiguous()
    q, k, v = l.parts(x)
    q1, k1, _ = bi.qk_norm_rope(q, k, *l.gains, l.pos[last].contiguous(), l.inv, EPS)
    assert _same(q1, r["q"][last]) and _same(k1, r["k"][last])
    room = max(lens) + 5
    cache = torch.full((2, len(lens) * room, Hkv, D), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    vs = l.parts(l.x)[2]
    for i, n in enumerate(lens):
        a, b = int(l.offs[i]), int(l.offs[i + 1])
        cache[0, i * room:i * room + n - 1] = r["k"][a:b - 1]
        cache[1, i * room:i * room + n - 1] = vs[a:b - 1]
        cache[0, i * room + n - 1], cache[1, i * room + n - 1] = k1[i], v[i]  # the step's own key and value
    out, lse, st = bi.attn_fwd(q1, cache[0], cache[1], torch.arange(len(lens) + 1, device=cuda_device),
                               k_offsets=torch.arange(len(lens) + 1, device=cuda_device) * room,
                               k_lens=torch.tensor(lens, dtype=torch.int32, device=cuda_device))
    bi.check_status(st)
    assert _same(out, r["out"][last]) and torch.equal(lse, r["lse"][:, last])


def test_a_process_may_capture_its_first_call(cuda_device):
    import os
    import subprocess
    import sys
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "capture_first_call.py")
    p = subprocess.run([sys.executable, path], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "captured first calls ok" in p.stdout, p.stderr[-2000:]
