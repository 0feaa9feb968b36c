"""Run by the tests in a process of its own: the process's first calls of the layer's and the update's entry
points are captured into a graph, replayed, and compared with eager ones."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import async_rl_b200 as bi  # noqa: E402


def main():
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    x, dout, g = r(150, 8, 64), r(150, 4, 64), r(64)
    pos, inv = torch.arange(150, dtype=torch.int32, device=dev), torch.ones(32, device=dev)
    offs = torch.tensor([0, 100, 150], device=dev)
    w = [torch.ones(1000, device=dev)]
    opt = bi.AdamWState.allocate(w)
    grad, step = [torch.ones(1000, device=dev)], torch.ones(1, dtype=torch.int64, device=dev)

    def run():
        q, k, st = bi.qk_norm_rope(x[:, :4], x[:, 4:6], g, g, pos, inv, 1e-6)
        out, lse, s1 = bi.attn_fwd(q, k, x[:, 6:], offs)
        dq, dk, dv, s2 = bi.attn_bwd(dout, q, k, x[:, 6:], out, lse, offs)
        back = bi.qk_norm_rope_bwd(dq, dk, x[:, :4], x[:, 4:6], g, g, pos, inv, 1e-6)
        s3 = bi.adamw_step(opt, grad, step, 1e-3)
        return [q, k, out, lse, dq, dk, dv, *back[:4]], [st, s1, s2, back[4], s3]

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held, status = run()
    graph.replay()
    torch.cuda.synchronize()
    for s in status:
        bi.check_status(s)
    first = w[0].clone()
    want, _ = run()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert torch.all(first < 1) and torch.all(w[0] < first)
    print("captured first calls ok")


if __name__ == "__main__":
    main()
