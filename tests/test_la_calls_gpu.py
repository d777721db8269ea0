"""Linear attention with a decay for each head: calls at the edges of what is documented (GPU)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda
import la_model as lm
import la_precision as lp

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [40, 300])
def test_lowest_rates(dtype, T):
    """The lowest fp32 number, minus infinity and one between: nothing is remembered, and o_t = (q_t . k_t) v_t."""
    d = lm.inputs(1, T, 4, 64, 128, dtype, seed=T)
    d["log_decay"].copy_(torch.tensor([torch.finfo(F32).min, float("-inf"), -2.4e38, -1e30]))
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = kda.la_chunk_forward(*a, d["S0"])
    g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
    pool = d["S0"].clone()
    one = kda.la_recurrent_step(*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"], pool)
    torch.cuda.synchronize()
    (o_ref, S_ref), _ = lm.reference(d)
    want, _ = lm.reference_backward(d)
    assert not lp.over(o, o_ref, lp.out_limit(dtype, T, 128), 2)
    assert not lp.over(S, S_ref, lp.state_limit(dtype, T, 128), 1)
    for x in ("dq", "dk", "dv"):
        assert not lp.over(g[x], want[x], lp.out_limit(dtype, T, 128), 2), x
    assert (g["dinit_state"] == 0).all()
    assert not lp.over(one.unsqueeze(1), o_ref[:, :1], lp.out_limit(dtype, 1, 128), 2)
    assert torch.equal(pool[0], d["k"][0, 0].float().unsqueeze(-1) * d["v"][0, 0].float().unsqueeze(-2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [60, 300])
def test_bad_slot_of_a_sequence_without_tokens(dtype, T):
    """It is flagged like any other, whether a call's sequences are cut between CTAs or not."""
    d = lm.inputs(1, T, 2, 64, 64, dtype, seed=T, N=3)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    cu = torch.tensor([0, T - 1, T - 1, T], dtype=torch.int32, device="cuda")
    pool = torch.randn(4, 2, 64, 64, device="cuda")
    before = pool.clone()
    good = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    o = kda.la_chunk_forward_slots(*a, pool, good, cu)
    after = pool.clone()
    assert kda.device_status() == 0
    for bad in (4, -2):
        pool.copy_(before)
        o2 = kda.la_chunk_forward_slots(*a, pool, torch.tensor([2, bad, 0], dtype=torch.int32, device="cuda"), cu)
        assert kda.device_status() == kda.DEV_BAD_SLOT
        assert torch.equal(o, o2) and torch.equal(pool, after)
    assert kda.device_status() == 0
