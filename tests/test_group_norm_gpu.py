"""Group norm with an activation, channels last, against float64 (GPU).

Bounds.  A mean or variance of n values is a sum of sequences of at most n / 32 + 40
roundings (partial sums of 256 threads or more, joined), each 2^-24 of a sum no larger than
that of the absolute values; with the subtraction, the products and the activation's own
error (below 2^-20: a slope of at most 1.1 on an exponential good to 2^-21) an element of z
is held to K = 2^-20 + (n / 32 + 40) 2^-24 of |w| rstd (|x| + max |x| of the group) + |b|.
An output in bf16 adds half a step of its own, 2^-8 of its value.  Sums over samples and
positions are held to their number of terms / 32 + 64 roundings of the sum of absolute values."""
import numpy as np
import pytest
import torch

import gated_delta_rule_85_b200 as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
ACT = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid}


def _model(x, G, w, b, gate, act):
    h = x.reshape(x.shape[0], -1, G, x.shape[-1] // G)
    mean = h.mean(dim=(1, 3))
    rstd = (h.var(dim=(1, 3), unbiased=False) + EPS).rsqrt()
    xhat = ((h - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    z = xhat
    if w is not None:
        z = z * w
    if b is not None:
        z = z + b
    return (ACT[act](z) if gate is None else z * ACT[act](gate)), mean, rstd, xhat


def _inputs(shape, dtype, seed, gate=True, affine=True, mean=0.3, std=1.0):
    gen = torch.Generator().manual_seed(seed)

    def normal(*s, m=0.0, sd=1.0):
        return torch.empty(s).normal_(m, sd, generator=gen).cuda()

    C = shape[-1]
    return dict(x=normal(*shape, m=mean, sd=std).to(dtype), dy=normal(*shape).to(dtype),
                gate=normal(*shape).to(dtype) if gate else None,
                w=normal(C, m=1.0, sd=0.2) if affine else None, b=normal(C, sd=0.2) if affine else None)


def _check(d, G, act, dtype):
    x, C = d["x"], d["x"].shape[-1]
    N, n = x.shape[0], x.numel() // x.shape[0] // G
    up = lambda t: None if t is None else t.double()  # noqa: E731
    leaf = {k: up(t).requires_grad_() for k, t in d.items() if k != "dy" and t is not None}
    y, mean, rstd, xhat = _model(leaf["x"], G, leaf.get("w"), leaf.get("b"), leaf.get("gate"), act)
    y.backward(up(d["dy"]))
    got_y, got_m, got_r = kda.group_norm(x, G, d["w"], d["b"], d["gate"], eps=EPS, activation=act)
    got = kda.group_norm_backward(d["dy"], x, got_m, got_r, G, d["w"], d["b"], d["gate"], activation=act)
    torch.cuda.synchronize()
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    K = 2.0 ** -20 + (n / 32 + 40) * 2.0 ** -24
    with torch.no_grad():
        g = lambda t: t.reshape(N, -1, G, C // G)  # noqa: E731
        spread = lambda t: t.reshape(N, 1, G, 1).expand(g(x).shape).reshape(x.shape)  # noqa: E731
        x64 = x.double()
        big = g(x64).abs().amax(dim=(1, 3))
        one = torch.ones(C, dtype=torch.float64, device="cuda")
        w = one if d["w"] is None else up(d["w"])
        b = 0 * one if d["b"] is None else up(d["b"])
        assert ((got_m.double() - mean).abs() <= K * big).all()
        # rstd: relative error of the variance, whose absolute error is K of the mean square around the mean
        # (moments are centred before they are squared) plus that of the mean's error
        assert ((got_r.double() - rstd).abs() <= rstd * (4 * K + (K * big * rstd) ** 2)).all()
        # an element of xhat: the mean's error and the rstd's relative one
        dh = K * 5 * spread(rstd) * (x64.abs() + spread(big)) + 2.0 ** -23
        dz = dh * w.abs() + 2.0 ** -22 * (xhat * w).abs() + 2.0 ** -23 * b.abs()
        slope = 1.1
        ga = None if d["gate"] is None else ACT[act](up(d["gate"]))
        lim = half * y.abs() + (dz * slope if ga is None else dz * ga.abs() + 2.0 ** -20 * y.abs()) + 2.0 ** -20 * y.abs()
        assert ((got_y.double() - y).abs() <= lim).all(), "y"
        dy = up(d["dy"]).abs()
        z = xhat * w + b
        # dz of the gradient: the slope's own slope is at most 0.5
        e_dz = dy * (0.5 * dz + 2.0 ** -20 * slope) if ga is None else dy * 2.0 ** -20 * ga.abs()
        a_dz = dy * slope if ga is None else dy * ga.abs()
        rows = tuple(range(x.dim() - 1))
        m = N * n // (C // G)
        S = (m / 32 + 64) * 2.0 ** -24
        if d["w"] is not None:
            lw = (e_dz * xhat.abs() + a_dz * dh).sum(rows) + S * (a_dz * xhat.abs()).sum(rows)
            lb = e_dz.sum(rows) + S * a_dz.sum(rows)
            assert ((got["dweight"].double() - leaf["w"].grad).abs() <= lw).all(), "dweight"
            assert ((got["dbias"].double() - leaf["b"].grad).abs() <= lb).all(), "dbias"
        else:
            assert "dweight" not in got and "dbias" not in got
        if ga is not None:
            lg = half * leaf["gate"].grad.abs() + dy * slope * (dz + z.abs() * 2.0 ** -19)
            assert ((got["dgate"].double() - leaf["gate"].grad).abs() <= lg).all(), "dgate"
        t, et = a_dz * w.abs(), e_dz * w.abs()
        mean_g = lambda v: spread(g(v).mean(dim=(1, 3)))  # noqa: E731
        h = xhat.abs()
        inner = t + mean_g(t) + h * mean_g(t * h)
        e_in = et + mean_g(et) + h * mean_g(et * h + t * dh) + dh * mean_g(t * h) + 2 * K * inner
        lx = half * leaf["x"].grad.abs() + spread(rstd) * (e_in + 5 * K * inner)
        assert ((got["dx"].double() - leaf["x"].grad).abs() <= lx).all(), "dx"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act,gate", [("none", False), ("silu", False), ("sigmoid", False), ("silu", True),
                                      ("sigmoid", True), ("none", True)])
@pytest.mark.parametrize("shape,G", [
    ((1, 64), 1), ((5, 3 * 128), 3), ((37, 8 * 64), 8), ((700, 2 * 128), 2),      # heads as groups
    ((3, 6 * 24), 6), ((9, 5 * 200), 5), ((4, 1000), 1), ((2, 7 * 13), 7),        # other widths, odd ones
    ((2, 33, 40), 4), ((1, 1000, 320), 32), ((3, 5, 7, 30), 3), ((2, 129, 96), 1),  # positions
])
def test_matches_float64(dtype, act, gate, shape, G):
    _check(_inputs(shape, dtype, seed=sum(shape), gate=gate), G, act, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,G", [((6, 4 * 128), 4), ((2, 300, 72), 8), ((1, 2, 64), 64), ((2, 4000, 10), 2),
                                     ((3, 2, 5000), 5), ((2, 3, 2600), 1)])
def test_without_affine(dtype, shape, G):
    _check(_inputs(shape, dtype, seed=3, gate=False, affine=False), G, "silu", dtype)


@pytest.mark.parametrize("shape,G", [((8, 4 * 64), 4), ((2, 700, 64), 4)])
def test_large_mean(shape, G):
    """A mean of 1000 standard deviations: squares that are summed uncentred would cancel."""
    _check(_inputs(shape, F32, seed=5, gate=False, mean=1000.0), G, "none", F32)
    d = _inputs(shape, F32, seed=6, gate=False)
    d["x"].view(-1)[0] = 1e4   # one outlier in the first place
    _check(d, G, "none", F32)


@pytest.mark.parametrize("shape,G", [((4, 2 * 128), 2), ((2, 50, 48), 6), ((1, 1, 3), 3)])
def test_constant_groups(shape, G):
    """No variance at all: xhat is 0 and rstd is eps^-1/2."""
    x = torch.full(shape, 2.5, device="cuda")
    b = torch.linspace(-1, 1, shape[-1], device="cuda")
    y, mean, rstd = kda.group_norm(x, G, None, b, activation="none")
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand(shape)) and (mean == 2.5).all()
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=2 ** -21, atol=0)


def test_no_samples():
    x = torch.empty(0, 5, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda")
    y, mean, rstd = kda.group_norm(x, 4, w, w)
    assert y.shape == x.shape and mean.shape == (0, 4)
    g = kda.group_norm_backward(x, x, mean, rstd, 4, w, w)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_bad_samples_stay_alone():
    d = _inputs((5, 60, 48), F32, seed=2)
    run = lambda: kda.group_norm(d["x"], 6, d["w"], d["b"], d["gate"])[0]  # noqa: E731
    a = run()
    d["x"][3] = float("nan")
    d["x"][1, :, :8] = float("inf")
    b = run()
    torch.cuda.synchronize()
    assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]]) and torch.equal(a[1, :, 8:], b[1, :, 8:])
    assert b[3].isnan().all()


def test_repeats_streams_and_graphs():
    d = _inputs((3, 400, 320), BF16, seed=1)
    side = torch.cuda.Stream()

    def call():
        y, m, r = kda.group_norm(d["x"], 32, d["w"], d["b"], d["gate"])
        return y, kda.group_norm_backward(d["dy"], d["x"], m, r, 32, d["w"], d["b"], d["gate"])

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y1, g1 = call()
    y2, g2 = call()
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and all(torch.equal(g1[k], g2[k]) for k in g1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = call()
    d["x"].normal_()
    d["dy"].normal_()
    graph.replay()
    y4, g4 = call()
    torch.cuda.synchronize()
    assert torch.equal(y3, y4) and all(torch.equal(g3[k], g4[k]) for k in g3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_behind_the_attention(dtype):
    """A layer as it is used: prefill, the norm over its heads with a gate, and both backwards."""
    B, T, H, dk, dv = 2, 130, 4, 64, 128
    gen = torch.Generator().manual_seed(3)
    normal = lambda *s, sd=1.0: torch.empty(s).normal_(0, sd, generator=gen).cuda()  # noqa: E731
    q, k = normal(B, T, H, dk, sd=dk ** -0.5).to(dtype), normal(B, T, H, dk, sd=dk ** -0.5).to(dtype)
    v, gate, dy = normal(B, T, H, dv).to(dtype), normal(B * T, H * dv).to(dtype), normal(B * T, H * dv).to(dtype)
    lg = -torch.tensor([0.4, 0.1, 0.03, 0.004], device="cuda")
    w, b = 1 + normal(H * dv, sd=0.1), normal(H * dv, sd=0.1)
    o, _ = kda.la_chunk_forward(q, k, v, lg, final_state=False)
    flat = o.view(B * T, H * dv)
    y, m, r = kda.group_norm(flat, H, w, b, gate)
    g = kda.group_norm_backward(dy, flat, m, r, H, w, b, gate)
    ga = kda.la_chunk_backward(q, k, v, lg, g["dx"].view_as(v), dinit_state=False)
    torch.cuda.synchronize()
    leaf = {n: t.double().requires_grad_() for n, t in dict(q=q, k=k, v=v, gate=gate, w=w, b=b).items()}
    i = torch.arange(T, device="cuda")
    D = torch.tril(torch.exp(lg.double().reshape(H, 1, 1) * (i[:, None] - i[None, :]).clamp_min(0)))
    s = torch.einsum("bihd,bjhd->bhij", leaf["q"], leaf["k"]) * D
    o64 = torch.einsum("bhij,bjhd->bihd", s, leaf["v"]).reshape(B * T, H * dv)
    y64 = _model(o64, H, leaf["w"], leaf["b"], leaf["gate"], "silu")[0]
    y64.backward(dy.double())
    # bf16: three roundings in a row (operands, o, the norm's own); gradients pass twice as many
    tol = 2.0 ** -6 if dtype == BF16 else 2.0 ** -16
    got = dict(y=(y, y64), gate=(g["dgate"], leaf["gate"].grad), w=(g["dweight"], leaf["w"].grad),
               b=(g["dbias"], leaf["b"].grad), q=(ga["dq"], leaf["q"].grad), k=(ga["dk"], leaf["k"].grad),
               v=(ga["dv"], leaf["v"].grad))
    for n, (x, ref) in got.items():
        rel = float((x.detach().double() - ref.detach()).norm() / ref.detach().norm())
        assert rel <= tol, (n, rel)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,G", [
    ((2, 1021, 640), 32), ((3, 4096, 320), 32), ((1, 9000, 24), 3), ((300, 3, 64), 4),   # one cluster of one to eight CTAs
    ((40, 2, 32), 32), ((1, 17, 2048), 1), ((2, 5, 2048), 2), ((1, 7, 4096), 1),            # widest rows, single-element groups
    ((1, 30000, 64), 1), ((2, 200, 1000), 8), ((1, 2500, 1030), 5),                         # beyond a cluster, odd widths
])
@pytest.mark.parametrize("gate", [False, True])
def test_forms_over_positions(dtype, shape, G, gate):
    _check(_inputs(shape, dtype, seed=sum(shape), gate=gate), G, "silu", dtype)


@pytest.mark.parametrize("shape,G", [((2 ** 17 + 5, 128 * 128), 128), ((2 ** 19 + 3, 16, 256), 32), ((1, 2 ** 23 + 64, 256), 32),
                                     ((2, 2 ** 22 + 64, 260), 5)],
                         ids=["rows", "clusters", "positions", "odd_positions"])
def test_elements_beyond_32_bits(shape, G):
    """More than 2^31 elements.  x is +-1 in turn, so every mean is 0 and every variance 1, and an element
    of the result is one of two values.  A thread's sums of ones are exact; the joins of at most 512 parts
    round once each, which holds a mean and a variance to 2^-14."""
    C = shape[-1]
    sign = torch.ones(C, dtype=BF16, device="cuda")
    sign[1::2] = -1
    x = sign.expand(shape).contiguous()
    y = torch.full_like(x, 7.0)
    w, b = torch.full((C,), 1.5, device="cuda"), torch.full((C,), 0.25, device="cuda")
    _, mean, rstd = kda.group_norm(x, G, w, b, activation="none", eps=EPS, y=y)
    z = (1 + EPS) ** -0.5 * 1.5 * sign.double() + 0.25
    assert (mean.abs() <= 2.0 ** -14).all() and ((rstd.double() - (1 + EPS) ** -0.5).abs() <= 2.0 ** -14).all()
    flat = y.view(-1, C)
    for part in (flat[:64], flat[-64:], flat[flat.shape[0] // 2 - 32:][:64]):
        assert ((part.double() - z).abs() <= 2.0 ** -8 * z.abs() + 1.5 * 2.0 ** -13).all()
    assert (y < 2).all()
    # dy = x: the projection takes all of dx but w rstd eps / (1 + eps); its three terms are each at most
    # 1.5 and carry the roundings of a group's sums
    g = kda.group_norm_backward(x, x, mean, rstd, G, w, b, activation="none", out={"dx": y.fill_(7.0)})
    M = x.numel() // C
    n = M // shape[0] * (C // G)
    lim = 3 * 1.5 * ((n / 32 + 64) * 2.0 ** -24 + 2.0 ** -13) + 2 * 1.5 * EPS
    assert (y.abs() <= lim).all()
    want = M * (1 + EPS) ** -0.5
    assert ((g["dweight"].double() - want).abs() <= want * ((M / 32 + 64) * 2.0 ** -24 + 2.0 ** -13)).all()
    assert ((g["dbias"].double() - M * sign.double()).abs() <= M * (M / 32 + 64) * 2.0 ** -24).all()
    del x, y, g, flat
    torch.cuda.empty_cache()
