"""Group norm with an activation: calls at the edges of what is documented (GPU)."""
import threading

import pytest
import torch

import gated_delta_rule_85_b200 as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _tensors(shape, G, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.empty(s).normal_(generator=gen).cuda()  # noqa: E731
    x, dy = normal(*shape).to(dtype), normal(*shape).to(dtype)
    stats = torch.empty(2, shape[0], G, device="cuda")
    return dict(x=x, dy=dy, y=torch.empty_like(x), dx=torch.empty_like(x), mean=stats[0], rstd=stats[1],
                ws=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))


def test_host_threads_with_tiles_of_different_sizes():
    """Two host threads use one kernel, each with the shared memory that its sizes need."""
    lib = kda.load_library()
    work = [(_tensors(s, G, BF16, seed=i), s, G) for i, (s, G) in enumerate([((1, 2, 64), 64), ((1, 4096, 320), 32)])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    errors = []
    start = threading.Barrier(len(work))

    def loop(t, shape, G, stream):
        p = {k: v.data_ptr() for k, v in t.items()}
        n = (shape[0], shape[1], shape[2], G)
        start.wait()
        for _ in range(3000):
            rc = lib.kda_group_norm_forward(p["x"], None, None, None, p["y"], p["mean"], p["rstd"], *n, 1e-5, 1, 0, p["ws"],
                                            1 << 22, stream)
            if rc == 0:
                rc = lib.kda_group_norm_backward(p["dy"], p["x"], p["mean"], p["rstd"], None, None, None, p["dx"], None, None,
                                                 None, *n, 1, 0, p["ws"], 1 << 22, stream)
            if rc:
                errors.append((shape, rc, lib.kda_last_error()))
                return

    threads = [threading.Thread(target=loop, args=(*w, s.cuda_stream)) for w, s in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for t, shape, G in work:
        y, mean, rstd = kda.group_norm(t["x"], G)
        g = kda.group_norm_backward(t["dy"], t["x"], mean, rstd, G)
        assert torch.equal(y, t["y"]) and torch.equal(mean, t["mean"]) and torch.equal(g["dx"], t["dx"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,G", [((2, 1, 5003), 5003), ((1, 37, 5001), 1667), ((3, 2, 4099), 4099), ((2, 3, 3015), 3),
                                     ((1, 21, 6007), 1), ((2, 50, 2304), 768), ((1, 3, 513), 27), ((1, 600, 1), 1)])
def test_partial_sums_of_many_channel_blocks(dtype, shape, G):
    """Groups inside one block of channels, across a border and over many blocks, in a workspace of exactly
    the size that is asked for, with what lies behind it unchanged."""
    N, L, C = shape
    t = _tensors(shape, G, dtype, seed=C)
    got = []
    for backward in (False, True):
        need = kda.group_norm_workspace_size(N, L, C, G, dtype, backward=backward)
        room = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
        ws = room[:need] if need else None
        if not backward:
            y, mean, rstd = kda.group_norm(t["x"], G, activation="none", workspace=ws)
            got.append(y)
        else:
            w = torch.ones(C, device="cuda")
            g = kda.group_norm_backward(t["dy"], t["x"], mean, rstd, G, w, w * 0, activation="none", workspace=ws)
        torch.cuda.synchronize()
        assert (room[need:] == 171).all()
    x = t["x"].double().requires_grad_()
    h = x.reshape(N, L, G, C // G)
    m, v = h.mean(dim=(1, 3), keepdim=True), h.var(dim=(1, 3), unbiased=False, keepdim=True)
    want = ((h - m) * (v + 1e-5).rsqrt()).reshape(shape)
    want.backward(t["dy"].double())
    # fp32 sums of n values around a mean of 0, in the root mean square; a group of one or two values may be
    # divided by a deviation far below the values (or by eps), which multiplies the mean's error
    n = L * C // G
    scale = 1 + float(((v + 1e-5).rsqrt() * h.abs().amax(dim=(1, 3), keepdim=True)).max().detach())
    tol = scale * 2.0 ** -24 * (n + 32) ** 0.5 * 8 + (2.0 ** -8 if dtype == BF16 else 0)
    size = float(want.detach().norm()) + 2.0 ** -10
    assert float((y.double() - want.detach()).norm()) <= tol * size
    assert float((g["dx"].double() - x.grad).norm()) <= tol * scale * (float(x.grad.norm()) + 2.0 ** -10 * float(t["dy"].double().norm()))
    assert float((mean.double() - m.detach().view(N, G)).abs().max()) <= 2.0 ** -24 * (n + 32) * float(h.detach().abs().max())
    xhat = want.detach()
    dw, db = (t["dy"].double() * xhat).sum((0, 1)), t["dy"].double().sum((0, 1))
    assert float((g["dweight"].double() - dw).norm()) <= 2 * tol * (float(dw.norm()) + 2.0 ** -10 * float(t["dy"].double().norm()))
    assert float((g["dbias"].double() - db).norm()) <= 2.0 ** -22 * (N * L + 32) ** 0.5 * float(t["dy"].double().norm())


@pytest.mark.parametrize("shape,G", [((5, 4 * 128), 4), ((2, 70, 48), 6), ((2, 7 * 13), 7)])
@pytest.mark.parametrize("gate", [False, True])
def test_either_way(monkeypatch, shape, G, gate):
    """The compiled short way and the Python way give the same bits and make the same refusals."""
    t = _tensors(shape, G, BF16, seed=9)
    C = shape[-1]
    w, b = torch.linspace(0.5, 1.5, C, device="cuda"), torch.linspace(-1, 1, C, device="cuda")
    ga = t["dy"].flip(0).contiguous() if gate else None
    odd = torch.empty(t["x"].numel() + 1, dtype=BF16, device="cuda")[1:].view(shape)
    got = []
    for long_way in (False, True):
        if long_way:
            monkeypatch.setattr(kda, "_fast", kda._LongWay())
        y, mean, rstd = kda.group_norm(t["x"], G, w, b, ga, eps=1e-4)
        g = kda.group_norm_backward(t["dy"], t["x"], mean, rstd, G, w, b, ga)
        plain = kda.group_norm(t["x"], G, activation="none")
        got.append((y, mean, rstd, *(g[k] for k in sorted(g)), *plain))
        given = torch.full_like(t["x"], 7.0)
        assert kda.group_norm(t["x"], G, w, b, ga, eps=1e-4, y=given)[0] is given and torch.equal(given, y)
        with pytest.raises(kda.KDAError, match="aligned"):
            kda.group_norm(odd, G)
        with pytest.raises(ValueError, match="eps"):
            kda.group_norm(t["x"], G, eps=-1.0)
        with pytest.raises(ValueError, match="activation"):
            kda.group_norm(t["x"], G, activation="relu")
        with pytest.raises(ValueError, match="groups"):
            kda.group_norm(t["x"], C + 1)
        with pytest.raises(ValueError, match="weight must be"):
            kda.group_norm(t["x"], G, w.double())
        with pytest.raises(ValueError, match="is on cpu"):
            kda.group_norm_backward(t["dy"], t["x"], mean.cpu(), rstd, G)
        with pytest.raises(ValueError, match="dy is required"):
            kda.group_norm_backward(None, t["x"], mean, rstd, G)
        with pytest.raises(TypeError):
            kda.group_norm(t["x"].half(), G)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
