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


def test_step_by_either_way(monkeypatch):
    """The compiled short way and the Python way give the same bits and make the same refusals."""
    d = lm.inputs(3, 1, 2, 64, 128, BF16, seed=6)
    a = (*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"])
    slots = torch.tensor([4, -1, 2], dtype=torch.int32, device="cuda")
    pool = torch.randn(5, 2, 64, 128, device="cuda")
    odd = torch.empty(a[0].numel() + 1, dtype=BF16, device="cuda")[1:].view_as(a[0])
    got = []
    for long_way in (False, True):
        if long_way:
            monkeypatch.setattr(kda, "_fast", kda._LongWay())
        S, P = d["S0"].clone(), pool.clone()
        o, given = torch.empty_like(a[2]), torch.full_like(a[2], 7.0)
        got.append((kda.la_recurrent_step(*a, S), S.clone(), kda.la_recurrent_step_slots(*a, P, slots), P))
        assert kda.la_recurrent_step(*a, S, given) is given and kda.la_recurrent_step_slots(*a, P, slots, o) is o
        with pytest.raises(kda.KDAError, match="aligned"):
            kda.la_recurrent_step(odd, *a[1:], S)
        with pytest.raises(kda.KDAError, match="num_slots|state_pool"):
            kda.la_recurrent_step_slots(*a, P[:0], slots)
        with pytest.raises(ValueError, match="slots must be"):
            kda.la_recurrent_step_slots(*a, P, slots[:2])
        with pytest.raises(ValueError, match="state must be"):
            kda.la_recurrent_step(*a, S[:2])
        with pytest.raises(ValueError, match="contiguous"):
            kda.la_recurrent_step(*a, S.transpose(2, 3).contiguous().transpose(2, 3))
        with pytest.raises(ValueError, match="is on cpu"):
            kda.la_recurrent_step(*a[:3], a[3].cpu(), S)
        with pytest.raises(ValueError, match="slots is required"):
            kda.la_recurrent_step_slots(*a, P, None)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert kda.device_status() == 0


@pytest.mark.parametrize("cu", [None, [0, 90, 90, 170]])
def test_prefill_by_either_way(monkeypatch, cu):
    B, T, N = (2, 170, 2) if cu is None else (1, 170, 3)
    d = lm.inputs(B, T, 2, 64, 64, BF16, seed=7, N=N)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, -1, 0][:N], dtype=torch.int32, device="cuda")
    got = []
    for long_way in (False, True):
        if long_way:
            monkeypatch.setattr(kda, "_fast", kda._LongWay())
        pool = torch.cat([d["S0"], d["S0"]])
        o, S = kda.la_chunk_forward(*a, d["S0"], cu_t)
        g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"], cu_t)
        got.append((o, S, kda.la_chunk_forward_slots(*a, pool, slots, cu_t), pool, *g.values()))
        assert kda.la_chunk_backward(*a, d["d_o"], dinit_state=False)["dinit_state"] is None if cu is None else True
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
