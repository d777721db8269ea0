"""Linear attention with a decay for each head in float64: the token recurrence and its
reverse mode, token by token, and the element-wise error bounds of the kernels.

Bounds.  With the same sums over absolute values (M of the output), each rounding of an
operand to bf16 is off by at most 2^-8 of its value, so it moves the output by at most
2^-8 of the part of M that it enters.  An output of the bf16 path sees, besides its own
rounding (2^-8 of its value): the decayed score of each pair (parts of M inside a chunk),
the state that a chunk starts from, rounded when it is read, and the decayed key rows
that were summed into it (both: the part of M from earlier chunks).  Together
2^-8 |o| + 2 2^-8 M, and (1 + 2^-8)^2 of that for roundings of rounded values.
fp32 sums of n terms, added in any order, are off by at most n 2^-23 M (a tensor core may
cut instead of rounding: a whole step each time).

Below 2^-126 fp32 has no full precision: a power of the decay there, or a product with it,
may be off by its whole value, less than 2^-126.  Each of the n terms of a sum then moves by
less than 2^-126 times its other factors, here (inputs()) below 2^5: n 2^-121 in all.
"""
import numpy as np
import torch

TINY = 2.0 ** -121   # see above


def to64(x):
    return None if x is None else x.detach().to("cpu", torch.float64).numpy()


def spans(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, log_decay, S0=None, cu=None):
    """o [B, T, H, dv] and the final states [N, H, dk, dv]; tokens outside every sequence stay NaN."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    sp = spans(B, T, cu)
    g = np.exp(log_decay)[:, None, None]
    o = np.full((B, T, H, dv), np.nan)
    S = np.zeros((len(sp), H, dk, dv)) if S0 is None else S0.copy()
    for n, (b, t0, t1) in enumerate(sp):
        for t in range(t0, t1):
            S[n] = g * S[n] + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.einsum("hkv,hk->hv", S[n], q[b, t])
    return o, S


def backward(q, k, v, log_decay, do, S0=None, dS=None, cu=None):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    sp = spans(B, T, cu)
    g = np.exp(log_decay)[:, None, None]
    dq, dkk, dvv = (np.full(x.shape, np.nan) for x in (q, k, v))
    A = np.zeros((len(sp), H, dk, dv)) if dS is None else dS.copy()
    for n, (b, t0, t1) in enumerate(sp):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[n].copy()
        for t in range(t0, t1):
            S = g * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            dq[b, t] = np.einsum("hkv,hv->hk", S, do[b, t])
        for t in reversed(range(t0, t1)):
            A[n] += q[b, t][:, :, None] * do[b, t][:, None, :]
            dkk[b, t] = np.einsum("hkv,hv->hk", A[n], v[b, t])
            dvv[b, t] = np.einsum("hkv,hk->hv", A[n], k[b, t])
            A[n] *= g
    return dict(dq=dq, dk=dkk, dv=dvv, dinit_state=A)


def bound(value, M, dtype, terms):
    """Element-wise bound of an output in the input dtype."""
    if dtype == torch.bfloat16:
        h = 2.0 ** -8
        return h * np.abs(value) + 2 * h * (1 + h) ** 2 * M + terms * (2.0 ** -23 * M + TINY)
    return terms * (2.0 ** -23 * M + TINY) + 2.0 ** -24 * np.abs(value)


def state_bound(M, terms):
    """Element-wise bound of a state: fp32 for either dtype."""
    return terms * (2.0 ** -23 * M + TINY)


def check(got, want, lim, what):
    got = to64(got)
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all(), f"{what}: not finite"
    over = np.abs(got - want)[live] - lim[live]
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond its bound (bound there {lim[live][over.argmax()]:.3e})"


def inputs(B, T, H, dk, dv, dtype, seed=0, N=None, slopes=None, device="cuda"):
    """q, k, v, d_o in dtype; states; log_decay from fast forgetting to none at all."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape).normal_(0.0, std, generator=gen)

    N = B if N is None else N
    if slopes is None:
        slopes = [2.0 ** -(8.0 * (h + 1) / H) for h in range(H)]
    d = dict(q=normal(B, T, H, dk, std=dk ** -0.5).to(dtype), k=normal(B, T, H, dk, std=dk ** -0.5).to(dtype),
             v=normal(B, T, H, dv).to(dtype), d_o=normal(B, T, H, dv).to(dtype), S0=normal(N, H, dk, dv),
             dS=normal(N, H, dk, dv), log_decay=-torch.tensor(slopes, dtype=torch.float32))
    return {n: t.to(device) for n, t in d.items()}


def reference(d, cu=None, with_S0=True):
    """(o, S) and their absolute sums."""
    a = [to64(d[x]) for x in ("q", "k", "v", "log_decay")]
    S0 = to64(d["S0"]) if with_S0 else None
    want = forward(*a, S0, cu)
    M = forward(*(np.abs(x) for x in a[:3]), a[3], None if S0 is None else np.abs(S0), cu)
    return want, M


def reference_backward(d, cu=None, with_S0=True, with_dS=True):
    a = {x: to64(d[x]) for x in ("q", "k", "v", "log_decay", "d_o")}
    S0 = to64(d["S0"]) if with_S0 else None
    dS = to64(d["dS"]) if with_dS else None
    run = lambda f: backward(f(a["q"]), f(a["k"]), f(a["v"]), a["log_decay"], f(a["d_o"]),  # noqa: E731
                             None if S0 is None else f(S0), None if dS is None else f(dS), cu)
    return run(lambda x: x), run(np.abs)
