"""Group norm with an activation: errors in the root mean square against norm_precision.py (GPU)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda
import norm_precision as np_

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act,gate", [("silu", False), ("silu", True), ("sigmoid", True), ("none", False)])
@pytest.mark.parametrize("shape,G", [
    ((700, 4 * 128), 4), ((300, 6 * 24), 6), ((64, 5 * 200), 5), ((50, 7 * 13), 7),       # one position: rows, odd widths
    ((2, 700, 64), 4), ((1, 1021, 640), 32), ((3, 512, 320), 32),                          # clusters
    ((1, 30000, 64), 1), ((2, 600, 1000), 8), ((1, 2500, 1030), 5), ((8, 1500, 320), 32),  # over positions
])
def test_every_output(dtype, act, gate, shape, G):
    d = np_.inputs(shape, dtype, sum(shape), gate)
    want = np_.model(d["x"], d["dy"], G, d["w"], d["b"], d["gate"], act)
    y, mean, rstd = kda.group_norm(d["x"], G, d["w"], d["b"], d["gate"], activation=act)
    g = kda.group_norm_backward(d["dy"], d["x"], mean, rstd, G, d["w"], d["b"], d["gate"], activation=act)
    torch.cuda.synchronize()
    m = d["x"].numel() // shape[-1]
    for name, got in dict(y=y, **g).items():
        lim = np_.limit(F32, m) if name in ("dweight", "dbias") else np_.limit(dtype)
        if dtype == BF16 and name in ("dweight", "dbias"):
            lim += 2.0 ** -16   # the hardware's exponential and reciprocal: a few 2^-22 of terms that are summed
        assert np_.rms(got, want[name]) <= lim, name
    assert float((mean.double() - want["mean"]).abs().max()) <= 2.0 ** -20
    assert np_.rms(rstd, want["rstd"]) <= 2.0 ** -20


@pytest.mark.parametrize("shape,G", [((64, 4 * 64), 4), ((2, 700, 64), 4), ((1, 30000, 64), 1), ((2, 600, 1000), 8)])
def test_large_mean(shape, G):
    """A mean of 1000 deviations."""
    d = np_.inputs(shape, F32, 3, False, mean=1000.0)
    want = np_.model(d["x"], d["dy"], G, d["w"], d["b"], None, "none")
    y, mean, rstd = kda.group_norm(d["x"], G, d["w"], d["b"], activation="none")
    torch.cuda.synchronize()
    assert float((mean.double() - want["mean"]).abs().max()) <= 2.0 ** -10
    assert np_.rms(rstd, want["rstd"]) <= 2.0 ** -18
    assert np_.rms(y, want["y"]) <= 2.0 ** -10 + np_.limit(F32)
