"""The norm-wise limits of la_precision.py on the CPU: a chunked form with the kernels' own
roundings stays below them, and forms with a planted mistake do not."""
import numpy as np
import pytest
import torch

import la_model as lm
import la_precision as lp

BF16 = torch.bfloat16


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(BF16).to(torch.float64).numpy()


def _keep(x, bits):
    """x with `bits` bits of mantissa."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, bits)), e - bits)


def _terms(x, n):
    """What n bf16 terms hold of fp32 numbers, each rounded from what is left."""
    x, out = np.asarray(x, np.float32), np.zeros(x.shape)
    for _ in range(n):
        term = _bf16(x)
        out += term
        x = x - term.astype(np.float32)
    return out


def _chunked(q, k, v, lg, S0, C=128, score=_bf16, state=_bf16, terms=3, carry=lambda x: x, drop=0):
    """The kernels' chunked form; `drop`: pairs that many tokens apart are left out."""
    B, T, H, dk = q.shape
    o, last = np.zeros(v.shape), np.zeros(S0.shape)
    for b in range(B):
        for h in range(H):
            g, S = np.exp(lg[h]), S0[b, h].copy()
            for t in range(0, T, C):
                a, c, d = q[b, t:t + C, h], k[b, t:t + C, h], v[b, t:t + C, h]
                n = len(a)
                i = np.arange(n)
                apart = i[:, None] - i[None, :]
                D = np.where((apart >= 0) & ((apart != drop) | (drop == 0)), g ** np.maximum(apart, 0), 0.0)
                o[b, t:t + C, h] = score((a @ c.T) * D) @ d + (g ** (i + 1))[:, None] * (a @ state(S))
                w = (g ** (n - 1 - i)).astype(np.float32)[:, None]
                S = carry(g ** n * S + _terms(w * c.astype(np.float32), terms).T @ d)
            last[b, h] = S
    return _bf16(o), last


def _case(T, H=4, d=128, seed=1):
    x = lm.inputs(1, T, H, d, d, BF16, seed=seed, device="cpu")
    (o, S), _ = lm.reference(x)
    return [lm.to64(x[n]) for n in ("q", "k", "v", "log_decay", "S0")], o, S


@pytest.mark.parametrize("T,d", [(61, 64), (200, 128), (700, 128)])
def test_the_kernels_roundings_stay_below(T, d):
    a, o, S = _case(T, d=d)
    got, last = _chunked(*a)
    assert not lp.over(got, o, lp.out_limit(BF16, T, d), 2)
    assert not lp.over(last, S, lp.state_limit(BF16, T, d), 1)


def _wrong(name, a):
    q, k, v, lg, S0 = a
    if name == "rates off by 1 %":
        return _chunked(q, k, v, lg * 1.01, S0)
    if name == "operands of 6 bits":
        return _chunked(_keep(q, 6), _keep(k, 6), _keep(v, 6), lg, S0)
    if name == "state carried in bf16":
        return _chunked(*a, carry=_bf16)
    if name == "pairs three tokens apart dropped":
        return _chunked(*a, drop=3)
    return _chunked(*a, terms=2)


@pytest.mark.parametrize("T", [200, 700])
@pytest.mark.parametrize("name", ["rates off by 1 %", "operands of 6 bits", "pairs three tokens apart dropped"])
def test_wrong_outputs_are_seen(name, T):
    a, o, _ = _case(T)
    got, _ = _wrong(name, a)
    assert lp.over(got, o, lp.out_limit(BF16, T, 128), 2)


@pytest.mark.parametrize("T", [200, 700])
@pytest.mark.parametrize("name", ["rates off by 1 %", "state carried in bf16", "weighted rows of two terms"])
def test_wrong_states_are_seen(name, T):
    a, _, S = _case(T)
    _, last = _wrong(name, a)
    assert lp.over(last, S, lp.state_limit(BF16, T, 128), 1)
    # and fp32 states of the CUDA-core path are held as closely
    assert lp.over(last, S, lp.state_limit(torch.float32, T, 128), 1)
