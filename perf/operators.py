"""Cases of the operators of the policy model's attention layer and of its update, to be timed and compared.

  qk     RMS norm of each query and key head with the rotation of its positions in the same pass, and its backward
  attn   softmax attention over packed sequences or key/value caches, and its backward
  adamw  one AdamW step over many tensors, with 32-bit or 8-bit states

`run` computes an operator in its plain form, or calls async_rl_b200's where `own` is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0    # largest float8_e4m3fn
E4M3_TINY = 2.0 ** -9  # smallest positive float8_e4m3fn
STATE_BLOCK = 256   # elements that share a scale in the 8-bit states


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of eight sequences, far into their contexts
        dict(name="qk_fwd_decode", op="qk", dir="fwd", T=8, Hq=12, Hkv=2, D=128, R=128, norm=True, far=131072),
        # the packed rows of one learner step of the 1.5B shape (64 responses of 256..2048 tokens)
        dict(name="qk_fwd_step", op="qk", dir="fwd", T=76239, Hq=12, Hkv=2, D=128, R=128, norm=True, far=2048),
        # backward of half a long-context batch of the 4B shape
        dict(name="qk_bwd_long", op="qk", dir="bwd", T=131072, Hq=32, Hkv=8, D=128, R=128, norm=True, far=16384),
        # the packed causal responses of one learner step, ragged
        dict(name="attn_fwd_step", op="attn", dir="fwd", kind="packed", S=64, lo=256, hi=2048, pre=0, lens=1235,
             Hq=12, Hkv=2, D=128, causal=True),
        # one 16K context of the 4B shape
        dict(name="attn_fwd_16k", op="attn", dir="fwd", kind="packed", S=1, lo=16384, hi=16384, pre=0, lens=1, Hq=32,
             Hkv=8, D=128, causal=True),
        # a rollout engine's decode step: single tokens over caches of up to 8K keys
        dict(name="attn_fwd_decode", op="attn", dir="fwd", kind="cache", S=64, lo=1, hi=1, pre=8192, lens=7, Hq=32,
             Hkv=8, D=128, causal=True),
        # the gradient of a learner step's attention
        dict(name="attn_bwd_step", op="attn", dir="bwd", kind="packed", S=64, lo=256, hi=2048, pre=0, lens=1235,
             Hq=12, Hkv=2, D=128, causal=True),
        # the gradient of a few 8K responses, heads of 64
        dict(name="attn_bwd_8k_d64", op="attn", dir="bwd", kind="packed", S=3, lo=4097, hi=8191, pre=0, lens=5, Hq=16,
             Hkv=8, D=64, causal=True),
        # a smoke-sized update: the norm gains of a few layers
        dict(name="adamw_gains", op="adamw", n=57, lo=128, hi=2560, sizes=3, master=True, grad="float32", bits=32),
        # the LM head of the 1.5B shape, whose gradient is float32, with its master weights
        dict(name="adamw_head", op="adamw", n=1, lo=151936 * 1536, hi=151936 * 1536, sizes=1, master=True,
             grad="float32", bits=32),
        # the matrices of a model's layers with 8-bit states
        dict(name="adamw_layers_8bit", op="adamw", n=48, lo=1536, hi=1536 * 8960, sizes=2, master=True,
             grad="bfloat16", bits=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "attn", "attn", "adamw"])
    if op == "qk":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.randint(1, 8)
        return dict(op="qk", dir=rng.choice(["fwd", "bwd"]), T=_log(rng, 1, max(1, 131072 * 40 * 128 // ((Hq + Hkv) * D))),
                    Hq=Hq, Hkv=Hkv, D=D, R=D if rng.random() < 0.7 else D // 32 * 16, norm=rng.random() < 0.8,
                    far=_log(rng, 2, 1 << 20))
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.randint(1, 8)
        D = rng.choice([64, 128])
        kind = rng.choice(["packed", "packed", "cache"])
        back = kind == "packed" and rng.random() < 0.5
        if kind == "cache":
            S, hi, pre = _log(rng, 1, 128), rng.choice([1, 1, 4, 33]), _log(rng, 16, 16384)
        else:
            S, hi, pre = _log(rng, 1, 96), _log(rng, 1, 8192), rng.choice([0, 0, 0, 777])
        most = 3.2e9 if back else 8e9  # padded scores of the plain form
        while S > 1 and S * Hkv * G * hi * (hi + pre) > most:
            S = S // 2
        return dict(op="attn", dir="bwd" if back else "fwd", kind=kind, S=S, lo=rng.choice([0, 1, (hi + 1) // 2]) if hi > 1 else 1,
                    hi=hi, pre=pre, lens=rng.randrange(1 << 20), Hq=Hkv * G, Hkv=Hkv, D=D, causal=rng.random() < 0.8)
    n = _log(rng, 1, 300)
    return dict(op="adamw", n=n, lo=1, hi=_log(rng, 64, max(128, (1 << 27) // n)), sizes=rng.randrange(1 << 20),
                master=rng.random() < 0.6, grad=rng.choice(["float32", "bfloat16"]), bits=rng.choice([8, 32]))


def _lengths(c):
    """Query and key lengths of each sequence: `pre` is the longest earlier context (cache), or one that all share."""
    r = random.Random(c["lens"])
    lq = [r.randint(c["lo"], c["hi"]) for _ in range(c["S"])]
    if c["S"] > 0 and max(lq) < c["hi"]:
        lq[0] = c["hi"]
    if c["kind"] == "cache":
        return lq, [n + r.randint(c["pre"] // 32, c["pre"]) for n in lq]
    return lq, [n + c["pre"] for n in lq]


def _sizes(c):
    r = random.Random(c["sizes"])
    return [_log(r, c["lo"], c["hi"]) for _ in range(c["n"])]


def work(case):
    c = case
    if c["op"] == "qk":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        passes = 2 if c["dir"] == "fwd" else 3 if c["norm"] else 2
        return dict(bytes=passes * 2 * n + 4 * c["T"], flops=(8 if c["dir"] == "fwd" else 16) * n)
    if c["op"] == "attn":
        lq, lk = _lengths(c)
        pairs = 0
        for a, b in zip(lq, lk):  # queries are the last `a` of the `b` positions
            full = min(a, b)
            pairs += full * (b - full) + full * (full + 1) // 2 if c["causal"] else a * b
        tq, tk = sum(lq), sum(lk)
        q, kv = tq * c["Hq"] * c["D"] * 2, tk * c["Hkv"] * c["D"] * 2
        if c["dir"] == "fwd":
            return dict(bytes=2 * q + 2 * kv + 4 * tq * c["Hq"], flops=4 * pairs * c["Hq"] * c["D"])
        return dict(bytes=4 * q + 4 * kv + 4 * tq * c["Hq"], flops=10 * pairs * c["Hq"] * c["D"])
    n = sum(_sizes(c))
    held = 16 if c["bits"] == 32 else 4
    return dict(bytes=n * (held + (4 if c["grad"] == "float32" else 2) + (10 if c["master"] else 8)), flops=16 * n)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return dict({"qk": _prepare_qk, "attn": _prepare_attn, "adamw": _prepare_adamw}[case["op"]](case, gen), case=case)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _prepare_qk(c, gen):
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    # the projection's output: heads of different magnitudes, queries and keys side by side
    scale = torch.exp(_randn(gen, 1, Hq + Hkv, 1))
    x = (torch.randn(T, Hq + Hkv, D, generator=gen, device=DEV) * scale).to(torch.bfloat16)
    s = dict(q=x[:, :Hq], k=x[:, Hq:], eps=1e-6,
             positions=torch.randint(0, c["far"], (T,), generator=gen, device=DEV, dtype=torch.int32),
             inv_freq=(1e6 ** (-torch.arange(0, c["R"], 2, device=DEV, dtype=torch.float64) / c["R"])).float(),
             gq=(1 + 0.2 * _randn(gen, D)).to(torch.bfloat16) if c["norm"] else None,
             gk=(1 + 0.2 * _randn(gen, D)).to(torch.bfloat16) if c["norm"] else None)
    if c["dir"] == "bwd":
        s["dq"] = (_randn(gen, T, Hq, D) * 1e-2).to(torch.bfloat16)
        s["dk"] = (_randn(gen, T, Hkv, D) * 1e-2).to(torch.bfloat16)
    return s


def _offsets(lens):
    o = torch.zeros(len(lens) + 1, dtype=torch.int64)
    o[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    return o.to(DEV)


def _prepare_attn(c, gen):
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    lq, lk = _lengths(c)
    tq = sum(lq)
    s = dict(lq=max(lq), lk=max(lk), q_offsets=_offsets(lq), k_offsets=None, k_lens=None)
    if c["kind"] == "cache":  # each sequence's keys in a slot of its own, with room behind them
        room = c["pre"] + c["hi"]
        s["k_offsets"] = _offsets([room] * c["S"])
        s["k_lens"] = torch.tensor(lk, dtype=torch.int32, device=DEV)
        s["q"] = _randn(gen, tq, Hq, D).to(torch.bfloat16)
        s["k"] = _randn(gen, room * c["S"], Hkv, D).to(torch.bfloat16)
        s["v"] = _randn(gen, room * c["S"], Hkv, D).to(torch.bfloat16)
    elif c["pre"]:
        s["k_offsets"] = _offsets(lk)
        s["q"] = _randn(gen, tq, Hq, D).to(torch.bfloat16)
        s["k"] = _randn(gen, sum(lk), Hkv, D).to(torch.bfloat16)
        s["v"] = _randn(gen, sum(lk), Hkv, D).to(torch.bfloat16)
    else:  # slices of one projection's output
        x = _randn(gen, tq, Hq + 2 * Hkv, D).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if c["dir"] == "bwd":
        s["out"], s["lse"] = _attn_fwd(c, s)
        s["dout"] = (_randn(gen, tq, Hq, D) * 1e-2).to(torch.bfloat16)
    return s


def _prepare_adamw(c, gen):
    sizes = _sizes(c)
    starts, total = [], 0
    for n in sizes:  # the tensors lie in flat buffers, each at a block of its own
        starts.append(total)
        total += -(-n // STATE_BLOCK) * STATE_BLOCK
    part = lambda flat: [flat[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
    live = torch.zeros(total, device=DEV)
    for x in part(live):
        x.fill_(1.0)
    w = _randn(gen, total).mul_(0.02)
    m = _randn(gen, total).mul_(1e-3).mul_(live)
    v = torch.rand(total, generator=gen, device=DEV).mul_(1e-5).mul_(live)
    grad = _randn(gen, total).mul_(3e-3).to(getattr(torch, c["grad"]))
    s = dict(total=total, live=live.bool(), grad=grad, lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=11,
             w=w.to(torch.bfloat16) if c["master"] else w, master=w.to(torch.bfloat16).float() if c["master"] else None)
    if c["bits"] == 32:
        s.update(m=m, v=v, ms=None, vs=None)
    else:
        s["m"], s["ms"] = _pack(m)
        s["v"], s["vs"] = _pack(v.sqrt(), True)
    blocks = [(a // STATE_BLOCK, -(-n // STATE_BLOCK)) for a, n in zip(starts, sizes)]
    scales = lambda flat: None if flat is None else [flat[a:a + n] for a, n in blocks]  # noqa: E731
    s["lists"] = dict(params=part(s["w"]), masters=part(s["master"]) if c["master"] else None, exp_avg=part(s["m"]),
                      exp_avg_sq=part(s["v"]), exp_avg_scale=scales(s["ms"]), exp_avg_sq_scale=scales(s["vs"]))
    s["grads"] = part(grad)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "qk":
        return _qk_fwd(c, s) if c["dir"] == "fwd" else _qk_bwd(c, s)
    if c["op"] == "attn":
        return list(_attn_fwd(c, s) if c["dir"] == "fwd" else _attn_bwd(c, s))
    return _adamw(s)


def _run_own(s, c):
    import async_rl_b200 as bi
    if c["op"] == "qk":
        if c["dir"] == "fwd":
            return list(bi.qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], s["positions"], s["inv_freq"], s["eps"])[:2])
        dq, dk, dgq, dgk, _ = bi.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["gq"], s["gk"], s["positions"],
                                                  s["inv_freq"], s["eps"])
        return [dq, dk, dgq, dgk] if c["norm"] else [dq, dk]
    if c["op"] == "attn":
        seqs = dict(k_offsets=s["k_offsets"], k_lens=s["k_lens"], causal=c["causal"])
        if c["dir"] == "fwd":
            return list(bi.attn_fwd(s["q"], s["k"], s["v"], s["q_offsets"], **seqs)[:2])
        return list(bi.attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["q_offsets"], **seqs)[:3])
    if "opt" not in s:  # the handle that a training program keeps
        s["opt"] = bi.AdamWState(**s["lists"])
    bi.adamw_step(s["opt"], s["grads"], s["step"], s["lr"], s["beta1"], s["beta2"], s["eps"], s["weight_decay"])
    return _adamw_out(s)


def _adamw_out(s):
    return [x for x in (s["w"], s["master"], s["m"], s["v"], s["ms"], s["vs"]) if x is not None]


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _angles(s):
    # float64: a far position times a frequency needs more than 24 bits
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(y, cos, sin, R):
    a, b, rest = y[..., :R // 2], y[..., R // 2:R], y[..., R:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _qk_fwd(c, s):
    cos, sin = _angles(s)

    def one(x, g):
        y = x.float()
        if g is not None:
            y = y * (y.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * g.float()
        return _rotate(y, cos, sin, c["R"]).to(torch.bfloat16)

    return [one(s["q"], s["gq"]), one(s["k"], s["gk"])]


def _qk_bwd(c, s):
    cos, sin = _angles(s)

    def one(dz, x, g):
        dy = _rotate(dz.float(), cos, -sin, c["R"])
        if g is None:
            return dy.to(torch.bfloat16), None
        x = x.float()
        r = (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
        n = x * r
        dn = dy * g.float()
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), (dy * n).sum((0, 1))

    (dq, dgq), (dk, dgk) = one(s["dq"], s["q"], s["gq"]), one(s["dk"], s["k"], s["gk"])
    return [x for x in (dq, dk, dgq, dgk) if x is not None]


def _padded(x, starts, lens, most):
    """[T, H, D] -> float32 [S, H, most, D], zero behind each sequence, and which rows are real."""
    at = torch.arange(most, device=x.device)
    real = at < lens[:, None]
    rows = torch.where(real, starts[:, None] + at, 0)
    return (x[rows].float() * real[..., None, None]).transpose(1, 2).contiguous(), real


def _attn_inputs(c, s):
    G = c["Hq"] // c["Hkv"]
    qo = s["q_offsets"]
    ko = qo if s["k_offsets"] is None else s["k_offsets"]
    lq = qo.diff()
    lk = ko.diff() if s["k_lens"] is None else s["k_lens"].long()
    q, real = _padded(s["q"], qo[:-1], lq, s["lq"])
    k, _ = _padded(s["k"], ko[:-1], lk, s["lk"])
    v, _ = _padded(s["v"], ko[:-1], lk, s["lk"])
    key = torch.arange(s["lk"], device=q.device)
    hidden = (key >= lk[:, None])[:, None, :]
    if c["causal"]:
        last = torch.arange(s["lq"], device=q.device) + (lk - lq)[:, None]
        hidden = hidden | (key > last[..., None])
    S, Lq, D = q.shape[0], s["lq"], c["D"]
    group = lambda x: x.reshape(S, c["Hkv"], G * Lq, -1)  # noqa: E731
    return q, k, v, real, hidden, group


def _packed(x, real):
    return x.transpose(1, 2)[real]


def _attn_fwd(c, s):
    q, k, v, real, hidden, group = _attn_inputs(c, s)
    S, Hq, Lq, D = q.shape
    p = group(q) @ k.transpose(-1, -2)
    p = p.mul_(D ** -0.5).view(S, Hq, Lq, s["lk"]).masked_fill_(hidden[:, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (group(p) @ v).view(S, Hq, Lq, D) / total.clamp(min=1e-30)
    lse = m + total.log()
    return _packed(o, real).to(torch.bfloat16), _packed(lse, real)[..., 0].t().contiguous()


def _attn_bwd(c, s):
    q, k, v, real, hidden, group = _attn_inputs(c, s)
    S, Hq, Lq, D = q.shape
    qo = s["q_offsets"]
    do, _ = _padded(s["dout"], qo[:-1], qo.diff(), Lq)
    o, _ = _padded(s["out"], qo[:-1], qo.diff(), Lq)
    lse, _ = _padded(s["lse"].t()[..., None], qo[:-1], qo.diff(), Lq)
    lse = torch.where(lse == -math.inf, 0.0, lse)
    p = (group(q) @ k.transpose(-1, -2)).mul_(D ** -0.5).view(S, Hq, Lq, s["lk"])
    p = p.sub_(lse).exp_().masked_fill_(hidden[:, None], 0.0)
    dv = group(p).transpose(-1, -2) @ group(do)
    ds = (group(do) @ v.transpose(-1, -2)).view_as(p)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq = (group(ds) @ k).view(S, Hq, Lq, D)
    dk = group(ds).transpose(-1, -2) @ group(q)
    ko = qo if s["k_offsets"] is None else s["k_offsets"]
    lk = ko.diff() if s["k_lens"] is None else s["k_lens"].long()
    real_k = torch.arange(s["lk"], device=q.device) < lk[:, None]
    return (_packed(dq, real).to(torch.bfloat16), _packed(dk, real_k).to(torch.bfloat16),
            _packed(dv, real_k).to(torch.bfloat16))


def _pack(x, positive=False):
    """Blocks of 256 values as float8 e4m3 and one float32 scale each. `positive`: no value above zero becomes zero."""
    b = x.view(-1, STATE_BLOCK)
    most = b.abs().amax(1)
    inv = torch.where(most > 0, E4M3_MAX / most, 0.0)
    y = b * inv[:, None]
    if positive:
        y = torch.where(b > 0, y.clamp(min=E4M3_TINY), y)
    return y.to(torch.float8_e4m3fn).view(-1), most / E4M3_MAX


def _unpack(codes, scale):
    return (codes.float().view(-1, STATE_BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    f = lambda x: torch.tensor(x, dtype=torch.float64).float().item()  # noqa: E731
    b1, b2 = s["beta1"], s["beta2"]
    rate = f(s["lr"] / (1 - b1 ** s["step"]))
    root = f(1 / math.sqrt(1 - b2 ** s["step"]))
    keep = f(1 - s["lr"] * s["weight_decay"])
    g = s["grad"].float() * s["live"]
    m = s["m"] if s["ms"] is None else _unpack(s["m"], s["ms"])
    v = s["v"] if s["vs"] is None else _unpack(s["v"], s["vs"]).square()
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    w = s["w"] if s["master"] is None else s["master"]
    new = w * keep - (m * rate) / (v.sqrt() * root + f(s["eps"]))
    w.copy_(torch.where(s["live"], new, w))
    if s["master"] is not None:
        s["w"].copy_(torch.where(s["live"], w, s["w"].float()))
    if s["ms"] is None:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for x, y in zip((s["m"], s["ms"], s["v"], s["vs"]), _pack(m) + _pack(v.sqrt(), True)):
            x.copy_(y)
    return _adamw_out(s)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "attn": _exact_attn, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_qk(c, s):
    """Rows as complex pairs, turned by exp(i angle), a slice of tokens at a time."""
    T, R, h = c["T"], c["R"], c["R"] // 2
    new = lambda x: torch.empty(x.shape, dtype=torch.float64, device=DEV)  # noqa: E731
    back = c["dir"] == "bwd"
    outs, grads = [], []
    for name in ("q", "k"):
        x, g = s[name], s["g" + name]
        out, dg = new(x), torch.zeros(c["D"], dtype=torch.float64, device=DEV)
        for a in range(0, T, 8192):
            z = slice(a, min(T, a + 8192))
            turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                               s["positions"][z, None].double() * s["inv_freq"].double())[:, None]
            X = x[z].double()
            r = 1 / torch.sqrt((X * X).sum(-1, keepdim=True) / c["D"] + s["eps"])
            Y = s["d" + name][z].double() if back else X if g is None else X * r * g.double()
            pair = torch.complex(Y[..., :h], Y[..., h:R]) * (turn.conj() if back else turn)
            Y = torch.cat([pair.real, pair.imag, Y[..., R:]], -1)
            if back and g is not None:
                dg += (Y * X * r).sum((0, 1))
                Y = Y * g.double()
                Y = r * Y - X * r ** 3 * (Y * X).sum(-1, keepdim=True) / c["D"]
            out[z] = Y
        outs.append(out)
        grads.append(dg)
    return outs + (grads if back and c["norm"] else [])


def _exact_attn(c, s):
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G, back = Hq // Hkv, c["dir"] == "bwd"
    lq, lk = _lengths(c)
    qo = [0]
    for n in lq:
        qo.append(qo[-1] + n)
    ko = qo if s["k_offsets"] is None else s["k_offsets"].tolist()
    zeros = lambda *n: torch.zeros(*n, dtype=torch.float64, device=DEV)  # noqa: E731
    out, lse = zeros(qo[-1], Hq, D), zeros(Hq, qo[-1])
    dq = zeros(qo[-1], Hq, D) if back else None
    dk, dv = (zeros(s["k"].shape[0], Hkv, D) for _ in "kv") if back else (None, None)
    for b in range(c["S"]):
        rows, keys = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b] + lk[b])
        if lq[b] == 0 or lk[b] == 0:
            lse[:, rows] = -math.inf
            continue
        for h in range(Hq):
            q, k, v = (x.double() for x in (s["q"][rows, h], s["k"][keys, h // G], s["v"][keys, h // G]))
            t = q @ k.T / math.sqrt(D)
            if c["causal"]:
                t = t + torch.full_like(t, -math.inf).triu(lk[b] - lq[b] + 1)
            z = torch.logsumexp(t, 1)
            p = torch.exp(t - torch.where(z == -math.inf, 0.0, z)[:, None])
            o = p @ v
            out[rows, h], lse[h, rows] = o, z
            if back:
                g = s["dout"][rows, h].double()
                dt = p * (g @ v.T - (g * o).sum(1, keepdim=True)) / math.sqrt(D)
                dq[rows, h] = dt @ k
                dk[keys, h // G] += dt.T @ q
                dv[keys, h // G] += p.T @ g
    return [dq, dk, dv] if back else [out, lse]


def _exact_adamw(c, s):
    d = lambda x: None if x is None else x.double()  # noqa: E731
    wide = lambda x, scale: x if scale is None else x * scale.repeat_interleave(STATE_BLOCK)  # noqa: E731
    g = d(s["grad"]) * s["live"]
    b1, b2, t = s["beta1"], s["beta2"], s["step"]
    m = b1 * wide(d(s["m"]), d(s["ms"])) + (1 - b1) * g
    v = wide(d(s["v"]), d(s["vs"]))
    v = b2 * (v if c["bits"] == 32 else v * v) + (1 - b2) * g * g
    w = d(s["w"] if s["master"] is None else s["master"])
    step = s["lr"] * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + s["eps"]) + s["weight_decay"] * w)
    w = torch.where(s["live"], w - step, w)
    head = [w, w] if c["master"] else [w]
    if c["master"]:
        head[0] = torch.where(s["live"], w, d(s["w"]))
    if c["bits"] == 32:
        return head + [m, v]
    u = torch.sqrt(v)
    sm, su = (x.abs().view(-1, STATE_BLOCK).amax(1) / E4M3_MAX for x in (m, u))
    code = lambda x, y: (x / y.clamp(min=1e-300).repeat_interleave(STATE_BLOCK)).float()  # noqa: E731
    cm = code(m, sm).to(torch.float8_e4m3fn)
    cu = torch.where(u > 0, code(u, su).clamp(min=E4M3_TINY), 0.0).to(torch.float8_e4m3fn)
    return head + [d(cm.float()), d(cu.float()), sm, su]
