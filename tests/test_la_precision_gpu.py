"""Linear attention with a decay for each head: the error of each head's outputs, states and
gradients in the norm, against the limits of la_precision.py (GPU)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda
import la_model as lm
import la_precision as lp

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 61, 8, 64, 64), (2, 200, 4, 128, 128), (1, 700, 5, 128, 128), (1, 513, 3, 64, 128), (1, 700, 3, 128, 64)]


def _prefill(d, o, S, dtype, cu=None, T=None):
    (o_ref, S_ref), _ = lm.reference(d, cu)
    T = d["q"].shape[1] if T is None else T
    dim = max(d["q"].shape[3], d["v"].shape[3])
    assert not lp.over(o, o_ref, lp.out_limit(dtype, T, dim), 2)
    assert not lp.over(S, S_ref, lp.state_limit(dtype, T, dim), 1)


def _grads(d, g, dtype, cu=None, T=None):
    want, _ = lm.reference_backward(d, cu)
    T = d["q"].shape[1] if T is None else T
    dim = max(d["q"].shape[3], d["v"].shape[3])
    for x in ("dq", "dk", "dv"):
        assert not lp.over(g[x], want[x], lp.out_limit(dtype, T, dim), 2), x
    assert not lp.over(g["dinit_state"], want["dinit_state"], lp.state_limit(dtype, T, dim), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,dk,dv", SHAPES)
def test_prefill_and_gradients(dtype, B, T, H, dk, dv):
    d = lm.inputs(B, T, H, dk, dv, dtype, seed=T + dv)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = kda.la_chunk_forward(*a, d["S0"])
    g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
    torch.cuda.synchronize()
    _prefill(d, o, S, dtype)
    _grads(d, g, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed(dtype):
    """The limits are those of the longest sequence."""
    cu = [0, 300, 301, 301, 430, 1100]
    d = lm.inputs(1, cu[-1], 3, 128, 128, dtype, seed=2, N=5)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, S = kda.la_chunk_forward(*a, d["S0"], cu_t)
    g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"], cu_t)
    torch.cuda.synchronize()
    _prefill(d, o, S, dtype, cu, 670)
    _grads(d, g, dtype, cu, 670)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_memory(dtype):
    """Heads that hardly forget: the sum of absolute products is a hundred times the output."""
    d = lm.inputs(1, 2000, 3, 128, 128, dtype, seed=3, slopes=[1e-5, 1e-3, 0.02])
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = kda.la_chunk_forward(*a, d["S0"])
    g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
    torch.cuda.synchronize()
    _prefill(d, o, S, dtype)
    _grads(d, g, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step(dtype):
    """One rounding of o, in the root mean square at the most half a step / sqrt(3)."""
    d = lm.inputs(16, 1, 4, 128, 64, dtype, seed=4)
    (o_ref, S_ref), _ = lm.reference(d)
    S = d["S0"].clone()
    o = kda.la_recurrent_step(*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"], S)
    torch.cuda.synchronize()
    limit = 1.1 * 2.0 ** -8 / 3 ** 0.5 if dtype == BF16 else lp.out_limit(F32, 1, 128)
    assert not lp.over(o.unsqueeze(1), o_ref, limit, 2)
    assert not lp.over(S, S_ref, lp.state_limit(F32, 1, 128), 1)
