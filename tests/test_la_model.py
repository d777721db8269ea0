"""The float64 model that the linear-attention kernels are tested against (CPU): closed
forms, the chunked regrouping, and its gradients against central differences."""
import numpy as np
import pytest

import la_model as lm


def _draw(B, T, H, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, T, H, dk)), r.standard_normal((B, T, H, dk)), r.standard_normal((B, T, H, dv)),
            -np.abs(r.standard_normal(H)), r.standard_normal((B, H, dk, dv)))


def test_no_decay_is_the_masked_product():
    q, k, v, _, _ = _draw(2, 9, 3, 4, 5)
    o, S = lm.forward(q, k, v, np.zeros(3))
    s = np.einsum("bihd,bjhd->bhij", q, k) * np.tril(np.ones((9, 9)))
    np.testing.assert_allclose(o, np.einsum("bhij,bjhd->bihd", s, v), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, np.einsum("bthk,bthv->bhkv", k, v), rtol=1e-12, atol=1e-12)


def test_total_decay_keeps_only_the_token_itself():
    q, k, v, _, S0 = _draw(1, 7, 2, 3, 4)
    o, _ = lm.forward(q, k, v, np.full(2, -np.inf), S0)
    np.testing.assert_allclose(o, np.einsum("bthd,bthd->bth", q, k)[..., None] * v, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("C", [1, 4, 5, 32])
def test_chunked_form(C):
    q, k, v, lg, S0 = _draw(1, 13, 2, 3, 4, seed=C)
    o, S = lm.forward(q, k, v, lg, S0)
    for h in range(2):
        g, X, got = np.exp(lg[h]), S0[0, h].copy(), []
        for t in range(0, 13, C):
            a, b, c = (x[0, t:t + C, h] for x in (q, k, v))
            n = len(a)
            i = np.arange(n)
            D = np.tril(g ** np.maximum(i[:, None] - i[None, :], 0))
            got.append(g ** (i + 1)[:, None] * (a @ X) + ((a @ b.T) * D) @ c)
            X = g ** n * X + (b * g ** (n - 1 - i)[:, None]).T @ c
        np.testing.assert_allclose(np.concatenate(got), o[0, :, h], rtol=1e-10, atol=1e-10)
        np.testing.assert_allclose(X, S[0, h], rtol=1e-10, atol=1e-10)


def test_packed_is_separate_runs():
    q, k, v, lg, _ = _draw(1, 12, 2, 3, 4)
    cu = [0, 5, 5, 6, 12]
    o, S = lm.forward(q, k, v, lg, None, cu)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        o1, S1 = lm.forward(q[:, a:b], k[:, a:b], v[:, a:b], lg)
        np.testing.assert_allclose(o[:, a:b], o1)
        np.testing.assert_allclose(S[n], S1[0])


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
def test_gradients_are_differences(cu):
    q, k, v, lg, S0 = _draw(1, 5, 2, 3, 2, seed=4)
    N = 1 if cu is None else len(cu) - 1
    r = np.random.default_rng(9)
    S0 = r.standard_normal((N, 2, 3, 2))
    do, dS = r.standard_normal(v.shape), r.standard_normal(S0.shape)

    def loss(q, k, v, S0):
        o, S = lm.forward(q, k, v, lg, S0, cu)
        return float((o * do).sum() + (S * dS).sum())

    g = lm.backward(q, k, v, lg, do, S0, dS, cu)
    args = dict(dq=q, dk=k, dv=v, dinit_state=S0)
    for name, x in args.items():
        for i in np.ndindex(x.shape):
            keep, h = x[i], 1e-5
            x[i] = keep + h
            up = loss(q, k, v, S0)
            x[i] = keep - h
            down = loss(q, k, v, S0)
            x[i] = keep
            assert abs((up - down) / (2 * h) - g[name][i]) < 1e-7 * max(1.0, abs(g[name][i])), (name, i)
