"""What the linear-attention and group-norm operators are measured on.

Five operators, each with a plain form (elementary torch operations in fp32) and
the library's own call:

  step      one token per sequence through linear attention with a decay for each head
  prefill   the same recurrence over whole prompts, dense or packed, with or without state slots
  grad      the gradients of the prefill
  norm      group norm with an activation, channels last (heads as groups, or long statistics)
  norm_grad its gradients

With g_h = exp(log_decay_h), per (sequence, head) and token t:
  S_t = g_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t
and per (sample n, group of channels) over all L positions:
  z = (x - mean) / sqrt(var + eps) * weight + bias;  y = act(z), or z * act(gate)

`own` selects which side `run` computes.
"""
import math
import random

import torch

own = False

EPS = 1e-5
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one user at decode time on a small model: launch latency is all there is
        dict(name="step_one", op="step", N=1, H=16, dk=64, dv=64, dtype="bf16", slots=False),
        # a full decode batch on a state pool, some rows padding (continuous batching)
        dict(name="step_batch", op="step", N=256, H=32, dk=128, dv=128, dtype="bf16", slots=True),
        # a short prompt of odd length
        dict(name="prefill_short", op="prefill", B=1, T=61, H=8, dk=64, dv=64, dtype="bf16", packed=0, slots=False),
        # the library's headline prefill size
        dict(name="prefill_8k", op="prefill", B=1, T=8192, H=32, dk=128, dv=128, dtype="bf16", packed=0,
             slots=False),
        # ragged prompts packed into one call, resumed from and written back to their slots
        dict(name="prefill_packed", op="prefill", B=1, T=16001, H=16, dk=128, dv=128, dtype="bf16", packed=9,
             slots=True),
        # fp32, unequal head sizes, a length that is no multiple of anything
        dict(name="prefill_f32", op="prefill", B=2, T=1003, H=8, dk=64, dv=128, dtype="f32", packed=0, slots=False),
        # a training step's backward at the headline size
        dict(name="grad_8k", op="grad", B=1, T=8192, H=32, dk=128, dv=128, dtype="bf16", packed=0),
        # a packed batch of short training sequences
        dict(name="grad_packed", op="grad", B=1, T=3001, H=6, dk=64, dv=128, dtype="bf16", packed=5),
        # the norm behind the headline prefill: one group per head, gated by a second projection
        dict(name="norm_heads", op="norm", N=8192, L=1, C=4096, G=32, dtype="bf16", act="silu", gate=True),
        # statistics over thousands of positions, ten channels a group
        dict(name="norm_long", op="norm", N=3, L=4096, C=320, G=32, dtype="bf16", act="silu", gate=False),
        # their gradients
        dict(name="norm_grad_heads", op="norm_grad", N=8192, L=1, C=4096, G=32, dtype="bf16", act="silu", gate=True),
        dict(name="norm_grad_long", op="norm_grad", N=2, L=1021, C=640, G=32, dtype="f32", act="silu", gate=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["step", "prefill", "prefill", "grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "step":
        H = _log(rng, 1, 32)
        return dict(op=op, N=_log(rng, 1, 256), H=H, dk=dk, dv=dv, dtype=dtype, slots=rng.random() < 0.5)
    if op in ("prefill", "grad"):
        H = _log(rng, 1, 32)
        tokens = _log(rng, 1, min(16384, (262144 if dtype == "bf16" else 32768) // H))
        c = dict(op=op, B=1, T=tokens, H=H, dk=dk, dv=dv, dtype=dtype, packed=0)
        how = rng.random()
        if how < 0.4:
            c["B"] = _log(rng, 1, 8)
            c["T"] = max(1, tokens // c["B"])
        elif how < 0.8:
            c["packed"] = _log(rng, 2, 16)
        if op == "prefill":
            c["slots"] = rng.random() < 0.4
        return c
    act = rng.choice(["none", "silu", "silu", "sigmoid"])
    if rng.random() < 0.5:      # one group per head
        H, D = _log(rng, 1, 32), rng.choice([64, 128])
        rows = _log(rng, 1, 8192)
        return dict(op=op, N=rows, L=1, C=H * D, G=H, dtype=dtype, act=act, gate=rng.random() < 0.7)
    G = rng.choice([1, 4, 8, 16, 32])
    C = G * _log(rng, 1, 1280 // G)
    N = _log(rng, 1, 8)
    return dict(op=op, N=N, L=_log(rng, 2, min(8192, (1 << 25) // (N * C))), C=C, G=G, dtype=dtype, act=act,
                gate=rng.random() < 0.3)


def _lengths(case):
    """Sequence lengths of a packed case: ragged, empty ones among them, summing to T."""
    n, total = case["packed"], case["T"]
    r = random.Random(1000 * n + total)
    w = [math.exp(r.uniform(0.0, 3.0)) for _ in range(n)]
    cut, at = [], 0.0
    for x in w[:-1]:
        at += x
        cut.append(int(total * at / sum(w)))
    if n >= 4:
        cut[1] = cut[0]
    cu = [0] + cut + [total]
    return [b - a for a, b in zip(cu, cu[1:])]


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=gen).to(dtype)

    def unit(*shape, dtype):
        x = normal(*shape)
        return (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)).to(dtype)

    dt = DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if case["op"] in ("norm", "norm_grad"):
        N, L, C = case["N"], case["L"], case["C"]
        shape = (N, C) if L == 1 else (N, L, C)
        s["x"] = normal(*shape, mean=0.3, dtype=dt)
        s["weight"] = normal(C, std=0.2, mean=1.0)
        s["bias"] = normal(C, std=0.2)
        s["gate"] = normal(*shape, dtype=dt) if case["gate"] else None
        if case["op"] == "norm_grad":
            s["dy"] = normal(*shape, dtype=dt)
            # what the forward pass kept: statistics of x, rounded to fp32
            m, r = _statistics(s["x"].to(torch.float64), case["G"])
            s["mean"], s["rstd"] = m.to(torch.float32), r.to(torch.float32)
        return s
    H, dk, dv = case["H"], case["dk"], case["dv"]
    # slopes halving over the heads, from fast forgetting to a memory of hundreds of tokens
    slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
    s["log_decay"] = -slope * (1.0 + 0.1 * torch.empty(H, device=dev).uniform_(0.0, 1.0, generator=gen))
    if case["op"] == "step":
        N = case["N"]
        s["q"], s["k"] = unit(N, H, dk, dtype=dt), unit(N, H, dk, dtype=dt)
        s["v"] = normal(N, H, dv, dtype=dt)
        rows = N + N // 4 if case["slots"] else N
        s["state"] = normal(rows, H, dk, dv, std=0.5)
        if case["slots"]:
            s["slots"] = _slots(N, rows, seed, dev)
        return s
    B, T = case["B"], case["T"]
    s["q"], s["k"] = unit(B, T, H, dk, dtype=dt), unit(B, T, H, dk, dtype=dt)
    s["v"] = normal(B, T, H, dv, dtype=dt)
    if case["packed"]:
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["lengths"] = lens
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    else:
        s["lengths"] = [T] * B
        s["cu_seqlens"] = None
    N = len(s["lengths"])
    if case["op"] == "prefill" and case["slots"]:
        s["state"] = normal(N + 3, H, dk, dv, std=0.5)
        s["slots"] = _slots(N, N + 3, seed, dev)
    else:
        s["state"] = normal(N, H, dk, dv, std=0.5)
    if case["op"] == "grad":
        s["d_o"] = normal(B, T, H, dv, dtype=dt)
        s["dfinal"] = normal(N, H, dk, dv)
    return s


def _slots(n, rows, seed, dev):
    """A shuffled row for each sequence; every seventh sequence is padding (-1)."""
    perm = list(range(rows))
    random.Random(int(seed)).shuffle(perm)
    return torch.tensor([-1 if i % 7 == 6 else perm[i] for i in range(n)], dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gated_delta_rule_85_b200 as kda

    c = s["case"]
    if c["op"] == "step":
        if c["slots"]:
            o = kda.la_recurrent_step_slots(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["slots"])
        else:
            o = kda.la_recurrent_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"])
        return dict(o=o, state=s["state"])
    if c["op"] == "prefill":
        if c["slots"]:
            o = kda.la_chunk_forward_slots(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["slots"],
                                           s["cu_seqlens"])
            return dict(o=o, state=s["state"])
        o, fs = kda.la_chunk_forward(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["cu_seqlens"])
        return dict(o=o, state=fs)
    if c["op"] == "grad":
        return kda.la_chunk_backward(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], s["state"], s["dfinal"],
                                     s["cu_seqlens"])
    if c["op"] == "norm":
        y, mean, rstd = kda.group_norm(s["x"], c["G"], s["weight"], s["bias"], s["gate"], eps=EPS,
                                       activation=c["act"])
        return dict(y=y, mean=mean, rstd=rstd)
    return kda.group_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], c["G"], s["weight"], s["bias"], s["gate"],
                                   activation=c["act"])


def _powers(log_decay, exponents):
    """exp(log_decay_h * e): [H, *exponents.shape] in fp32, the angle in 64 bits."""
    e = exponents.to(torch.float64)
    return torch.exp(log_decay.to(torch.float64).reshape(-1, *[1] * e.dim()) * e).to(torch.float32)


def _plain_step(s):
    c = s["case"]
    pool = s["state"]
    g = torch.exp(s["log_decay"]).reshape(1, -1, 1, 1)
    q, k, v = (s[x].to(torch.float32) for x in "qkv")
    if not c["slots"]:
        pool.mul_(g).add_(k.unsqueeze(-1) * v.unsqueeze(-2))
        return dict(o=(q.unsqueeze(-2) @ pool).squeeze(-2).to(s["q"].dtype), state=pool)
    # padding rows work on a spare row of zeros; their results are dropped
    live = (s["slots"] >= 0).reshape(-1, 1, 1)
    idx = s["slots"].to(torch.int64)
    spare = torch.cat([pool, torch.zeros_like(pool[:1])])
    at = torch.where(idx >= 0, idx, spare.shape[0] - 1)
    S = spare[at] * g + k.unsqueeze(-1) * v.unsqueeze(-2)
    o = torch.where(live, (q.unsqueeze(-2) @ S).squeeze(-2), torch.zeros_like(v)).to(s["q"].dtype)
    spare[at] = S
    pool.copy_(spare[:-1])
    return dict(o=o, state=pool)


class _Padded:
    """Packed or dense tokens [B, T, H, d] as [N, H, chunks, CHUNK, d] in fp32, zeros behind each sequence."""

    def __init__(self, s):
        q = s["q"]
        self.B, self.T, self.H = q.shape[:3]
        dev = q.device
        if s["cu_seqlens"] is None:
            start = torch.arange(self.B, device=dev) * self.T
            self.len = torch.full((self.B,), self.T, device=dev)
        else:
            cu = s["cu_seqlens"].to(torch.int64)
            start, self.len = cu[:-1], cu[1:] - cu[:-1]
        self.N = start.shape[0]
        self.nc = max(1, -(-max(s["lengths"]) // CHUNK))
        pos = torch.arange(self.nc * CHUNK, device=dev)
        self.live = pos.reshape(1, -1) < self.len.reshape(-1, 1)
        self.at = torch.where(self.live, start.reshape(-1, 1) + pos.reshape(1, -1), 0)
        self.pos = pos

    def chunks(self, x):
        d = x.shape[-1]
        y = x.reshape(-1, self.H, d).to(torch.float32)[self.at]
        y = torch.where(self.live.reshape(self.N, -1, 1, 1), y, torch.zeros_like(y))
        return y.reshape(self.N, self.nc, CHUNK, self.H, d).permute(0, 3, 1, 2, 4)

    def tokens(self, y, like):
        d = y.shape[-1]
        y = y.permute(0, 2, 3, 1, 4).reshape(self.N, -1, self.H, d)
        out = torch.zeros(self.B * self.T, self.H, d, dtype=torch.float32, device=y.device)
        out[self.at[self.live]] = y[self.live]
        return out.reshape(self.B, self.T, self.H, d).to(like.dtype)


def _lower(log_decay, n, first):
    """[H, n, n]: exp(log_decay * (i - j - first)) where i - j >= first, zero elsewhere."""
    i = torch.arange(n, device=log_decay.device)
    e = i.reshape(-1, 1) - i.reshape(1, -1) - first
    return torch.where(e >= 0, _powers(log_decay, e.clamp_min(0)), torch.zeros((), device=log_decay.device))


def _start_states(p, k, v, log_decay, S0):
    """The state before each chunk, [N, H, chunks, dk, dv]."""
    i = torch.arange(CHUNK, device=k.device)
    U = (k * _powers(log_decay, CHUNK - 1 - i).reshape(1, p.H, 1, CHUNK, 1)).transpose(-1, -2) @ v
    M = _lower(log_decay * CHUNK, p.nc, 1)
    dk, dv = U.shape[-2:]
    S = (M @ U.reshape(p.N, p.H, p.nc, dk * dv)).reshape(p.N, p.H, p.nc, dk, dv)
    n = torch.arange(p.nc, device=k.device) * CHUNK
    return S + _powers(log_decay, n).reshape(1, p.H, p.nc, 1, 1) * S0.unsqueeze(2)


def _plain_prefill(s):
    c, lg = s["case"], s["log_decay"]
    p = _Padded(s)
    if c["slots"]:
        idx = s["slots"].to(torch.int64)
        S0 = torch.where((idx >= 0).reshape(-1, 1, 1, 1), s["state"][idx.clamp_min(0)], torch.zeros((), device=lg.device))
    else:
        S0 = s["state"]
    q, k, v = p.chunks(s["q"]), p.chunks(s["k"]), p.chunks(s["v"])
    i = torch.arange(CHUNK, device=lg.device)
    S = _start_states(p, k, v, lg, S0)
    o = ((q @ k.transpose(-1, -2)) * _lower(lg, CHUNK, 0).reshape(1, p.H, 1, CHUNK, CHUNK)) @ v
    o = o + _powers(lg, i + 1).reshape(1, p.H, 1, CHUNK, 1) * (q @ S)
    # every token's weight in its sequence's last state (the exponent is clamped behind the end, where k is zero)
    w = _powers(lg, (p.len.reshape(-1, 1) - 1 - p.pos.reshape(1, -1)).clamp_min(0)).permute(1, 0, 2)
    flat = lambda x: x.reshape(p.N, p.H, p.nc * CHUNK, x.shape[-1])  # noqa: E731
    last = (flat(k) * w.unsqueeze(-1)).transpose(-1, -2) @ flat(v)
    last = last + _powers(lg, p.len).permute(1, 0).reshape(p.N, p.H, 1, 1) * S0
    o = p.tokens(o, s["v"])
    if not c["slots"]:
        return dict(o=o, state=last)
    live = idx >= 0
    s["state"][idx[live]] = last[live]
    return dict(o=o, state=s["state"])


def _plain_grad(s):
    lg = s["log_decay"]
    p = _Padded(s)
    q, k, v, do = (p.chunks(s[x]) for x in ("q", "k", "v", "d_o"))
    i = torch.arange(CHUNK, device=lg.device)
    S = _start_states(p, k, v, lg, s["state"])
    D = _lower(lg, CHUNK, 0).reshape(1, p.H, 1, CHUNK, CHUNK)
    P, dP = (q @ k.transpose(-1, -2)) * D, (do @ v.transpose(-1, -2)) * D
    up = _powers(lg, i + 1).reshape(1, p.H, 1, CHUNK, 1)
    # X: the adjoint of the state behind each chunk, as its last token meets it; padded
    # rows of q and do are zero, and the last state's gradient enters behind each sequence's end
    A = (q * up).transpose(-1, -2) @ do
    M = _lower(lg * CHUNK, p.nc, 1).transpose(-1, -2)
    dk, dv = A.shape[-2:]
    X = (M @ A.reshape(p.N, p.H, p.nc, dk * dv)).reshape(p.N, p.H, p.nc, dk, dv)
    end = (torch.arange(1, p.nc + 1, device=lg.device) * CHUNK).reshape(1, -1)
    last = _powers(lg, (p.len.reshape(-1, 1) - end).clamp_min(0)).permute(1, 0, 2)
    inside = (p.len.reshape(-1, 1) > end).reshape(p.N, 1, p.nc, 1, 1)
    dS = s["dfinal"].unsqueeze(2)
    X = X + torch.where(inside, last.unsqueeze(-1).unsqueeze(-1) * dS, torch.zeros((), device=lg.device))
    down = _powers(lg, CHUNK - 1 - i).reshape(1, p.H, 1, CHUNK, 1)
    # the chunk that holds a sequence's end gets the last state's gradient token by token
    left = p.len.reshape(-1, 1) - 1 - p.pos.reshape(1, -1)
    here = ((left >= 0) & (left < CHUNK) & (p.pos.reshape(1, -1) // CHUNK == (p.len.reshape(-1, 1) - 1) // CHUNK))
    tail = torch.where(here.unsqueeze(0), _powers(lg, left.clamp_min(0)), torch.zeros((), device=lg.device))
    tail = tail.permute(1, 0, 2).reshape(p.N, p.H, p.nc, CHUNK, 1)
    dq = dP @ k + up * (do @ S.transpose(-1, -2))
    dk_ = dP.transpose(-1, -2) @ q + down * (v @ X.transpose(-1, -2)) + tail * (v @ dS.transpose(-1, -2))
    dv_ = P.transpose(-1, -2) @ do + down * (k @ X) + tail * (k @ dS)
    w = _powers(lg, p.pos + 1).reshape(1, p.H, -1, 1)
    flat = lambda x: x.reshape(p.N, p.H, p.nc * CHUNK, x.shape[-1])  # noqa: E731
    dS0 = (flat(q) * w).transpose(-1, -2) @ flat(do)
    dS0 = dS0 + _powers(lg, p.len).permute(1, 0).reshape(p.N, p.H, 1, 1) * s["dfinal"]
    return dict(dq=p.tokens(dq, s["q"]), dk=p.tokens(dk_, s["k"]), dv=p.tokens(dv_, s["v"]), dinit_state=dS0)


def _grouped(x, G):
    """[N, L, G, channels of a group]"""
    return x.reshape(x.shape[0], -1, G, x.shape[-1] // G)


def _statistics(x, G):
    """mean and 1 / sqrt(var + eps) of each (sample, group), [N, G]."""
    x = _grouped(x, G)
    n = x.shape[1] * x.shape[3]
    mean = x.sum((1, 3), keepdim=True) / n
    var = (x - mean).square().sum((1, 3), keepdim=True) / n
    return mean.reshape(x.shape[0], G), ((var + EPS) ** -0.5).reshape(x.shape[0], G)


def _act(x, act):
    return x if act == "none" else (1 / (1 + torch.exp(-x))) * (x if act == "silu" else 1)


def _act_slope(x, act):
    if act == "none":
        return torch.ones_like(x)
    p = 1 / (1 + torch.exp(-x))
    return p * (1 + x * (1 - p)) if act == "silu" else p * (1 - p)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].to(torch.float32)
    mean, rstd = _statistics(x, c["G"])
    put = lambda t: t.reshape(x.shape[0], 1, c["G"], 1)  # noqa: E731
    z = ((_grouped(x, c["G"]) - put(mean)) * put(rstd)).reshape(x.shape) * s["weight"] + s["bias"]
    y = _act(z, c["act"]) if s["gate"] is None else z * _act(s["gate"].to(torch.float32), c["act"])
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_grad(s):
    c = s["case"]
    G, dt = c["G"], s["x"].dtype
    x, dy = s["x"].to(torch.float32), s["dy"].to(torch.float32)
    put = lambda t: t.reshape(x.shape[0], 1, G, 1)  # noqa: E731
    xhat = ((_grouped(x, G) - put(s["mean"])) * put(s["rstd"])).reshape(x.shape)
    z = xhat * s["weight"] + s["bias"]
    out = {}
    if s["gate"] is None:
        dz = dy * _act_slope(z, c["act"])
    else:
        gate = s["gate"].to(torch.float32)
        dz = dy * _act(gate, c["act"])
        out["dgate"] = (dy * z * _act_slope(gate, c["act"])).to(dt)
    rows = tuple(range(x.dim() - 1))
    out["dweight"], out["dbias"] = (dz * xhat).sum(rows), dz.sum(rows)
    t, h = _grouped(dz * s["weight"], G), _grouped(xhat, G)
    n = t.shape[1] * t.shape[3]
    a, b = t.sum((1, 3), keepdim=True) / n, (t * h).sum((1, 3), keepdim=True) / n
    out["dx"] = ((t - a - h * b) * put(s["rstd"])).reshape(x.shape).to(dt)
    return out


def _run_plain(s):
    return {"step": _plain_step, "prefill": _plain_prefill, "grad": _plain_grad, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad}[s["case"]["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        n = case["N"] * case["L"] * case["C"]
        stats, g = 8 * case["N"] * case["G"], 1 if case["gate"] else 0
        if case["op"] == "norm":
            return dict(bytes=n * es * (2 + g) + 8 * case["C"] + stats, flops=(8 + 5 * g) * n)
        return dict(bytes=n * es * (3 + 2 * g) + 16 * case["C"] + stats, flops=(16 + 10 * g) * n)
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] == "step":
        live = case["N"] - (case["N"] // 7 if case["slots"] else 0)
        return dict(bytes=live * H * 8 * dk * dv + case["N"] * H * es * 2 * (dk + dv), flops=live * H * 5 * dk * dv)
    n, seqs = case["B"] * case["T"] * H, case["packed"] or case["B"]
    if case["op"] == "prefill":
        return dict(bytes=n * es * 2 * (dk + dv) + 8 * seqs * H * dk * dv, flops=4 * n * dk * dv)
    return dict(bytes=n * es * (4 * dk + 3 * dv) + 12 * seqs * H * dk * dv, flops=10 * n * dk * dv)


# ------------------------------------------------------------------ the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "prefill": _exact_prefill, "grad": _exact_grad, "norm": _exact_norm,
            "norm_grad": _exact_norm_grad}[case["op"]](s)


def _exact_step(s):
    g = s["log_decay"].double().exp()[:, None, None]
    N = s["q"].shape[0]
    rows = s["slots"].tolist() if s["case"]["slots"] else list(range(N))
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device=g.device)
    state = s["state"].double()
    for n, r in enumerate(rows):
        if r >= 0:
            state[r] = g * state[r] + torch.einsum("hk,hv->hkv", s["k"][n].double(), s["v"][n].double())
            o[n] = torch.einsum("hkv,hk->hv", state[r], s["q"][n].double())
    return dict(o=o, state=state)


def _spans(s):
    T = s["case"]["T"]
    if s["cu_seqlens"] is None:
        return [(b, 0, T) for b in range(s["case"]["B"])]
    cu = s["cu_seqlens"].tolist()
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def _exact_prefill(s):
    """The token recurrence."""
    g = s["log_decay"].double().exp()[:, None, None]
    rows = s["slots"].tolist() if s["case"]["slots"] else list(range(len(s["lengths"])))
    q, k, v = (s[x].double() for x in "qkv")
    o = torch.zeros_like(v)
    state = s["state"].double()
    for n, (b, t0, t1) in enumerate(_spans(s)):
        S = state[rows[n]].clone() if rows[n] >= 0 else torch.zeros_like(state[0])
        for t in range(t0, t1):
            S.mul_(g).add_(k[b, t][:, :, None] * v[b, t][:, None, :])
            o[b, t] = torch.bmm(q[b, t][:, None, :], S)[:, 0]
        if rows[n] >= 0:
            state[rows[n]] = S
    return dict(o=o, state=state)


def _exact_grad(s):
    """Reverse mode through the token recurrence."""
    g = s["log_decay"].double().exp()[:, None, None]
    q, k, v, do = (s[x].double() for x in ("q", "k", "v", "d_o"))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dS0 = s["dfinal"].double()
    for n, (b, t0, t1) in enumerate(_spans(s)):
        S = s["state"][n].double()
        for t in range(t0, t1):
            S = g * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            dq[b, t] = torch.bmm(S, do[b, t][:, :, None])[:, :, 0]
        A = dS0[n].clone()
        for t in reversed(range(t0, t1)):
            A.add_(q[b, t][:, :, None] * do[b, t][:, None, :])
            dk[b, t] = torch.bmm(A, v[b, t][:, :, None])[:, :, 0]
            dv[b, t] = torch.bmm(k[b, t][:, None, :], A)[:, 0]
            A.mul_(g)
        dS0[n] = A
    return dict(dq=dq, dk=dk, dv=dv, dinit_state=dS0)


def _exact_forward_norm(x, gate, weight, bias, G, act):
    h = x.reshape(x.shape[0], -1, G, x.shape[-1] // G)
    mean = h.mean(dim=(1, 3))
    rstd = (h.var(dim=(1, 3), unbiased=False) + EPS).rsqrt()
    z = ((h - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape) * weight + bias
    f = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid}[act]
    return (f(z) if gate is None else z * f(gate)), mean, rstd


def _exact_norm(s):
    c = s["case"]
    gate = None if s["gate"] is None else s["gate"].double()
    y, mean, rstd = _exact_forward_norm(s["x"].double(), gate, s["weight"].double(), s["bias"].double(), c["G"],
                                        c["act"])
    return dict(y=y, mean=mean, rstd=rstd)


def _exact_norm_grad(s):
    """Differentiated by autograd, in 64 bits."""
    c = s["case"]
    names = ["x", "weight", "bias"] + (["gate"] if s["gate"] is not None else [])
    leaf = {n: s[n].double().requires_grad_() for n in names}
    y, _, _ = _exact_forward_norm(leaf["x"], leaf.get("gate"), leaf["weight"], leaf["bias"], c["G"], c["act"])
    y.backward(s["dy"].double())
    return {"d" + n: t.grad for n, t in leaf.items()}
