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
