"""The limits of norm_precision.py on the CPU: fp32 arithmetic stays below them, planted mistakes do not."""
import pytest
import torch

import norm_precision as np_


def _fp32(d, G, lose=0, part=0):
    """y in fp32 arithmetic; `lose` positions are left out of the mean, or the mean is of `part` values too many."""
    x = d["x"].reshape(d["x"].shape[0], -1, G, d["x"].shape[-1] // G)
    L, D = x.shape[1], x.shape[3]
    mean = x[:, : L - lose].sum((1, 3)) / ((L - lose) * D + part)
    c = x - mean[:, None, :, None]
    rstd = (c.square().sum((1, 3)) / (L * D) + np_.EPS).rsqrt()
    return (c * rstd[:, None, :, None]).reshape(d["x"].shape) * d["w"] + d["b"], mean


@pytest.mark.parametrize("shape,G", [((2, 700, 64), 4), ((64, 512), 4)])
def test_limits(shape, G):
    d = np_.inputs(shape, torch.float32, 1, False, device="cpu")
    want = np_.model(d["x"], d["dy"], G, d["w"], d["b"], None, "none")["y"]
    assert np_.rms(_fp32(d, G)[0], want) <= np_.limit(torch.float32)
    assert np_.rms(_fp32(d, G, part=1)[0], want) > np_.limit(torch.float32)
    if len(shape) == 3:
        assert np_.rms(_fp32(d, G, lose=8)[0], want) > np_.limit(torch.float32)


def test_large_mean_limit():
    d = np_.inputs((2, 700, 64), torch.float32, 2, False, mean=1000.0, device="cpu")
    want = np_.model(d["x"], d["dy"], 4, d["w"], d["b"], None, "none")
    assert float((_fp32(d, 4)[1].double() - want["mean"]).abs().max()) <= 2.0 ** -10
    assert float((_fp32(d, 4, lose=8)[1].double() - want["mean"]).abs().max()) > 2.0 ** -10
