"""Linear attention with a decay for each head against its float64 model (GPU): prefill,
slots, decode, gradients; element-wise bounds derived in la_model.py."""
import numpy as np
import pytest
import torch

import gated_delta_rule_85_b200 as kda
import la_model as lm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _terms(T, d):
    return T + d + 32


def _check_prefill(d, o, S, dtype, cu=None, with_S0=True):
    (o_ref, S_ref), (Mo, MS) = lm.reference(d, cu, with_S0)
    n = _terms(d["q"].shape[1], max(d["q"].shape[3], d["v"].shape[3]))
    lm.check(o, o_ref, lm.bound(o_ref, Mo, dtype, n), "o")
    if S is not None:
        lm.check(S, S_ref, lm.state_bound(MS, n), "final state")
    assert kda.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,dk,dv", [
    (1, 1, 1, 64, 64), (1, 1, 3, 128, 128), (2, 63, 2, 64, 128), (1, 64, 2, 128, 64), (2, 65, 3, 128, 128),
    (1, 127, 2, 64, 64), (1, 128, 1, 128, 128), (3, 129, 2, 64, 128), (1, 700, 5, 128, 128), (2, 513, 3, 128, 64),
    (5, 200, 7, 64, 64),
])
def test_prefill(dtype, B, T, H, dk, dv):
    d = lm.inputs(B, T, H, dk, dv, dtype, seed=T + dk)
    o, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], d["S0"])
    torch.cuda.synchronize()
    _check_prefill(d, o, S, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_without_states(dtype):
    d = lm.inputs(2, 150, 2, 64, 128, dtype, seed=3)
    o, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], final_state=False)
    torch.cuda.synchronize()
    assert S is None
    _check_prefill(d, o, None, dtype, with_S0=False)
    # the outputs do not depend on whether the final state is asked for
    o2, S2 = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"])
    assert torch.equal(o, o2)
    _check_prefill(d, o2, S2, dtype, with_S0=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("slopes", [[0.0, 0.0], [100.0, 5.0], [0.7, 88.0], [1e-5, 0.05]],
                         ids=["none", "total", "strong", "weak"])
def test_decay_range(dtype, slopes):
    """From rates that forget nothing to rates whose powers leave fp32 within a chunk."""
    d = lm.inputs(1, 300, 2, 128, 64, dtype, seed=11, slopes=slopes)
    o, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], d["S0"])
    _check_prefill(d, o, S, dtype)
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"])
    _check_grads(d, g, dtype)


@pytest.mark.parametrize("dtype,T", [(BF16, 300), (F32, 150)])
@pytest.mark.parametrize("slotted", [False, True])
def test_dense_batches_of_whole_sequences(dtype, T, slotted):
    """More sequences than SMs, each of several chunks: spans of one and of two whole ones."""
    B, H = 10, 20
    d = lm.inputs(B, T, H, 64, 64, dtype, seed=T)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    if slotted:
        pool = torch.cat([d["S0"].flip(0), torch.zeros_like(d["S0"][:1])])
        slots = torch.arange(B - 1, -1, -1, dtype=torch.int32, device="cuda")
        o = kda.la_chunk_forward_slots(*a, pool, slots)
        S = pool[:B].flip(0)
    else:
        o, S = kda.la_chunk_forward(*a, d["S0"])
        g = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
        _check_grads(d, g, dtype)
    _check_prefill(d, o, S, dtype)


CUS = [[0, 70, 70, 199, 200, 264], [0, 0, 0, 5], [0, 1], [0, 128, 256, 384], [0, 300, 301, 301, 301, 650, 651],
       [0] + list(range(1, 41)) + [400]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", CUS, ids=[f"{len(c) - 1}seq_{c[-1]}" for c in CUS])
@pytest.mark.parametrize("H", [1, 3])
def test_packed(dtype, cu, H):
    N = len(cu) - 1
    d = lm.inputs(1, cu[-1], H, 64, 128, dtype, seed=N, N=N)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], d["S0"], cu_t)
    torch.cuda.synchronize()
    _check_prefill(d, o, S, dtype, cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_the_last_sequence_stay(dtype):
    cu, T = [0, 40, 150], 200
    d = lm.inputs(1, T, 2, 64, 64, dtype, seed=5, N=2)
    for x in ("q", "k", "v", "d_o"):
        d[x][:, 150:] = float("nan")   # nobody's rows: neither read into a result nor written
    o = torch.full_like(d["v"], 7.0)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    _, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], d["S0"], cu_t, o=o)
    out = {x: torch.full_like(d[y], 7.0) for x, y in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"], cu_t, out=out)
    torch.cuda.synchronize()
    for t in (o, g["dq"], g["dk"], g["dv"]):
        assert (t[:, 150:] == 7.0).all()
    e = {x: (t[:, :150] if x in ("q", "k", "v", "d_o") else t) for x, t in d.items()}
    _check_prefill(e, o[:, :150], S, dtype, cu)
    _check_grads(e, {x: (t[:, :150] if x != "dinit_state" else t) for x, t in g.items()}, dtype, cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_neighbours_do_not_leak(dtype):
    """A sequence whose tokens and state are NaN or infinite leaves the others' results alone."""
    cu = [0, 30, 95, 170, 330]
    d = lm.inputs(1, 330, 2, 128, 64, dtype, seed=8, N=4)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    args = lambda: (d["q"], d["k"], d["v"], d["log_decay"])  # noqa: E731
    o1, S1 = kda.la_chunk_forward(*args(), d["S0"], cu_t)
    g1 = kda.la_chunk_backward(*args(), d["d_o"], d["S0"], d["dS"], cu_t)
    for x in ("q", "k", "v", "d_o"):
        d[x][:, 30:60] = float("nan")
        d[x][:, 60:95] = float("inf")
    d["S0"][1] = float("nan")
    d["dS"][1] = float("-inf")
    o2, S2 = kda.la_chunk_forward(*args(), d["S0"], cu_t)
    g2 = kda.la_chunk_backward(*args(), d["d_o"], d["S0"], d["dS"], cu_t)
    torch.cuda.synchronize()
    keep = torch.ones(330, dtype=torch.bool, device="cuda")
    keep[30:95] = False
    assert torch.equal(o1[:, keep], o2[:, keep])
    for x in ("dq", "dk", "dv"):
        assert torch.equal(g1[x][:, keep], g2[x][:, keep]), x
    for n in (0, 2, 3):
        assert torch.equal(S1[n], S2[n])
        assert torch.equal(g1["dinit_state"][n], g2["dinit_state"][n])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [None, [0, 70, 70, 199, 200, 564]])
def test_slots(dtype, cu):
    """From and into pool rows; a row that nobody names, a padding sequence, a bad entry."""
    B, T = (5, 140) if cu is None else (1, cu[-1])
    d = lm.inputs(B, T, 3, 64, 128, dtype, seed=21, N=5)
    pool = torch.randn(9, 3, 64, 128, device="cuda")
    table = [4, 0, -1, 7, 2]
    slots = torch.tensor(table, dtype=torch.int32, device="cuda")
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    before = pool.clone()
    for n, s in enumerate(table):
        d["S0"][n] = pool[s] if s >= 0 else 0
    o = kda.la_chunk_forward_slots(d["q"], d["k"], d["v"], d["log_decay"], pool, slots, cu_t)
    torch.cuda.synchronize()
    S = torch.stack([pool[s] if s >= 0 else torch.zeros_like(pool[0]) for s in table])
    (o_ref, S_ref), (Mo, MS) = lm.reference(d, cu)
    n = _terms(T, 128)
    lm.check(o, o_ref, lm.bound(o_ref, Mo, dtype, n), "o")
    live = [i for i, s in enumerate(table) if s >= 0]
    lm.check(S[live], S_ref[live], lm.state_bound(MS, n)[live], "pool rows")
    for s in (1, 3, 5, 6, 8):
        assert torch.equal(pool[s], before[s])
    assert kda.device_status() == 0
    # an entry outside the pool is flagged and counts as none
    slots[1] = 9
    kda.la_chunk_forward_slots(d["q"], d["k"], d["v"], d["log_decay"], pool, slots, cu_t)
    assert kda.device_status() == kda.DEV_BAD_SLOT
    assert kda.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 60, 300])
def test_bad_slot_is_flagged(dtype, T):
    """Whether a sequence is cut between CTAs or not; its rows are those of a start from zeros."""
    d = lm.inputs(2, T, 2, 64, 64, dtype, seed=T)
    pool = torch.randn(3, 2, 64, 64, device="cuda")
    before = pool.clone()
    d["S0"][0], d["S0"][1] = pool[2], 0
    for bad in (3, -2, 2 ** 31 - 1):
        pool.copy_(before)
        slots = torch.tensor([2, bad], dtype=torch.int32, device="cuda")
        o = kda.la_chunk_forward_slots(d["q"], d["k"], d["v"], d["log_decay"], pool, slots)
        assert kda.device_status() == kda.DEV_BAD_SLOT
        (o_ref, _), (Mo, _) = lm.reference(d)
        lm.check(o, o_ref, lm.bound(o_ref, Mo, dtype, _terms(T, 64)), "o")
        assert torch.equal(pool[:2], before[:2])
        one = kda.la_recurrent_step_slots(*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"], pool, slots)
        assert (one[1] == 0).all()
        assert kda.device_status() == kda.DEV_BAD_SLOT
    assert kda.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_malformed_offsets_stay_in_bounds(dtype):
    """Offsets that fall, leave the tokens or are negative: every access is clamped, rows around
    the tensors stay, and a well-formed call behind is right."""
    T, N = 500, 4
    d = lm.inputs(1, T, 3, 64, 128, dtype, seed=1, N=N)
    big = {x: torch.full((T + 64, *d[y].shape[2:]), 7.0, dtype=dtype, device="cuda")
           for x, y in (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    at = {x: t[32:32 + T].unsqueeze(0) for x, t in big.items()}
    for cu in ([0, 400, 100, 500, 300], [-5, 200, 900, 3, 500], [500, 0, 500, 0, 500], [2 ** 31 - 1, -2 ** 31, 0, 7, 9]):
        cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        a = (d["q"], d["k"], d["v"], d["log_decay"])
        kda.la_chunk_forward(*a, d["S0"], cu_t, o=at["o"])
        kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"], cu_t, out={x: at[x] for x in ("dq", "dk", "dv")})
        torch.cuda.synchronize()
        for x, t in big.items():
            assert (t[:32] == 7.0).all() and (t[32 + T:] == 7.0).all(), x
    assert kda.device_status() == 0
    cu = [0, 100, 100, 300, 500]
    o, S = kda.la_chunk_forward(*a, d["S0"], torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _check_prefill(d, o, S, dtype, cu)


def test_short_way_and_long_way_agree():
    """Calls that the compiled short way leaves to Python (outputs of gradients given, a workspace
    of another type) give the same bits; errors of the C ABI come through either."""
    d = lm.inputs(1, 200, 2, 64, 64, BF16, seed=9)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    g1 = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
    out = {x: torch.empty_like(t) for x, t in g1.items()}
    g2 = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"], out=dict(out))
    for x in g1:
        assert torch.equal(g1[x], g2[x]) and g2[x].data_ptr() == out[x].data_ptr()
    o1, S1 = kda.la_chunk_forward(*a, d["S0"])
    o2, S2 = torch.empty_like(o1), torch.empty_like(S1)
    ws = torch.empty(kda.la_workspace_size(1, 200, 2, 64, 64, 1) // 4 + 64, dtype=torch.float32, device="cuda")
    r = kda.la_chunk_forward(*a, d["S0"], o=o2, final_state=S2, workspace=ws)
    assert r[0] is o2 and r[1] is S2 and torch.equal(o1, o2) and torch.equal(S1, S2)
    with pytest.raises(kda.KDAError, match="workspace"):
        kda.la_chunk_forward(*a, d["S0"], workspace=ws[:16])
    odd = torch.empty(d["q"].numel() + 1, dtype=BF16, device="cuda")[1:].view_as(d["q"])
    with pytest.raises(kda.KDAError, match="aligned"):
        kda.la_chunk_forward(odd, *a[1:], d["S0"])
    with pytest.raises(ValueError, match="contiguous"):
        kda.la_chunk_forward(d["q"].expand(1, 200, 2, 64).transpose(1, 2).contiguous().transpose(1, 2), *a[1:], d["S0"])
    with pytest.raises(ValueError, match="float32"):
        kda.la_chunk_forward(*a, d["S0"].double())
    with pytest.raises(ValueError, match="slots"):
        kda.la_recurrent_step_slots(*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"], d["S0"],
                                    torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="is on cpu"):
        kda.la_chunk_forward(d["q"], d["k"].cpu(), *a[2:], d["S0"])


def _check_grads(d, g, dtype, cu=None, with_S0=True, with_dS=True, dinit=True):
    want, M = lm.reference_backward(d, cu, with_S0, with_dS)
    n = _terms(d["q"].shape[1], max(d["q"].shape[3], d["v"].shape[3]))
    for x in ("dq", "dk", "dv"):
        lm.check(g[x], want[x], lm.bound(want[x], M[x], dtype, n), x)
    if dinit:
        lm.check(g["dinit_state"], want["dinit_state"], lm.state_bound(M["dinit_state"], n), "dinit_state")
    assert kda.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 1, 2, 64, 128), (2, 64, 2, 128, 128), (1, 130, 3, 128, 64),
                                         (3, 200, 2, 64, 64), (1, 700, 3, 64, 128), (1, 385, 2, 128, 128)])
def test_gradients(dtype, B, T, H, dk, dv):
    d = lm.inputs(B, T, H, dk, dv, dtype, seed=T)
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"])
    torch.cuda.synchronize()
    _check_grads(d, g, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", CUS, ids=[f"{len(c) - 1}seq_{c[-1]}" for c in CUS])
def test_packed_gradients(dtype, cu):
    N = len(cu) - 1
    d = lm.inputs(1, cu[-1], 2, 64, 128, dtype, seed=N, N=N)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"], cu_t)
    torch.cuda.synchronize()
    _check_grads(d, g, dtype, cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_without_states(dtype):
    d = lm.inputs(2, 300, 2, 128, 128, dtype, seed=2)
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], dinit_state=False)
    torch.cuda.synchronize()
    assert g["dinit_state"] is None
    _check_grads(d, g, dtype, with_S0=False, with_dS=False, dinit=False)


def test_gradients_are_differences():
    """fp32, through the library's own forward: <d_o, o> + <dS, S> moved along a random direction.
    The function is linear in v and S0 and quadratic in (q, k) together, so a central
    difference has no error of its own for one of them; what is left is fp32 rounding of two
    sums of T H dv + H dk dv products, held here to 2^-23 times the sum of their absolute values."""
    d = lm.inputs(1, 150, 2, 64, 64, F32, seed=6)
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"])
    gen = torch.Generator().manual_seed(1)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dinit_state")):
        step = torch.empty(d[name].shape).normal_(generator=gen).cuda() * 0.5
        side = []
        scale = 0.0
        for sign in (1, -1):
            e = dict(d)
            e[name] = d[name] + sign * step
            o, S = kda.la_chunk_forward(e["q"], e["k"], e["v"], e["log_decay"], e["S0"])
            a, b = o.double() * d["d_o"].double(), S.double() * d["dS"].double()
            side.append(float(a.sum() + b.sum()))
            scale += float(a.abs().sum() + b.abs().sum())
        diff = (side[0] - side[1]) / 2
        want = float((g[key].double() * step.double()).sum())
        scale += float((g[key].double() * step.double()).abs().sum())
        # each o, S and gradient is itself a sum of at most 150 + 64 + 32 terms
        assert abs(diff - want) <= (150 + 64 + 32) * 2.0 ** -23 * scale, name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_step(dtype, dk, dv):
    d = lm.inputs(5, 6, 3, dk, dv, dtype, seed=dk + dv)
    (o_ref, S_ref), (Mo, MS) = lm.reference(d)
    S = d["S0"].clone()
    for t in range(6):
        o = kda.la_recurrent_step(*(d[x][:, t].contiguous() for x in "qkv"), d["log_decay"], S)
        # one rounding of o; fp32 sums of dk products
        lim = (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * np.abs(o_ref[:, t]) + (dk + 16) * 2.0 ** -23 * Mo[:, t]
        lm.check(o, o_ref[:, t], lim, f"o of step {t}")
    lm.check(S, S_ref, lm.state_bound(MS, 32), "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_slots(dtype):
    d = lm.inputs(4, 1, 3, 128, 64, dtype, seed=4)
    pool = torch.randn(6, 3, 128, 64, device="cuda")
    table = [5, -1, 0, 3]
    before = pool.clone()
    for n, s in enumerate(table):
        d["S0"][n] = pool[s] if s >= 0 else 0
    (o_ref, S_ref), (Mo, MS) = lm.reference(d)
    slots = torch.tensor(table, dtype=torch.int32, device="cuda")
    o = kda.la_recurrent_step_slots(*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"], pool, slots)
    torch.cuda.synchronize()
    assert (o[1] == 0).all()
    live = [0, 2, 3]
    lim = (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * np.abs(o_ref) + (128 + 16) * 2.0 ** -23 * Mo
    lm.check(o[live], o_ref[live, 0], lim[live, 0], "o")
    S = torch.stack([pool[table[i]] for i in live])
    lm.check(S, S_ref[live], lm.state_bound(MS, 8)[live], "pool")
    for s in (1, 2, 4):
        assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_in_pieces_then_decode(dtype):
    """One run as a server makes it: a prompt in two calls through its slot, then tokens."""
    d = lm.inputs(1, 210, 2, 128, 128, dtype, seed=13)
    pool = torch.zeros(3, 2, 128, 128, device="cuda")
    pool[1] = d["S0"][0]
    slots = torch.tensor([1], dtype=torch.int32, device="cuda")
    o = [kda.la_chunk_forward_slots(*(d[x][:, a:b].contiguous() for x in "qkv"), d["log_decay"], pool, slots)
         for a, b in ((0, 100), (100, 207))]
    for t in range(207, 210):
        step = kda.la_recurrent_step_slots(*(d[x][:, t].contiguous() for x in "qkv"), d["log_decay"], pool, slots)
        o.append(step.unsqueeze(1))
    torch.cuda.synchronize()
    _check_prefill(d, torch.cat(o, 1), pool[1:2], dtype)


def test_no_tokens():
    q = torch.empty(2, 0, 3, 64, device="cuda", dtype=BF16)
    lg = -torch.rand(3, device="cuda")
    S0 = torch.randn(2, 3, 64, 64, device="cuda")
    o, S = kda.la_chunk_forward(q, q, q, lg, S0)
    assert o.shape == q.shape and torch.equal(S, S0)
    _, S = kda.la_chunk_forward(q, q, q, lg)
    assert (S == 0).all()
    g = kda.la_chunk_backward(q, q, q, lg, q, S0, S0)
    assert torch.equal(g["dinit_state"], S0)
    empty = torch.empty(0, 3, 64, device="cuda", dtype=BF16)
    assert kda.la_recurrent_step(empty, empty, empty, lg, S0[:0]).shape == (0, 3, 64)


def test_repeats_are_equal():
    """The same call twice gives the same bits, and a workspace's old contents do not matter."""
    d = lm.inputs(1, 1500, 6, 128, 128, BF16, seed=1)
    ws = torch.full((kda.la_workspace_size(1, 1500, 6, 128, 128, 1),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((kda.la_backward_workspace_size(1, 1500, 6, 128, 128, 1),), 255, dtype=torch.uint8, device="cuda")
    a = [d[x] for x in ("q", "k", "v", "log_decay")]
    o1, S1 = kda.la_chunk_forward(*a, d["S0"], workspace=ws)
    o2, S2 = kda.la_chunk_forward(*a, d["S0"])
    g1 = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"], workspace=wb)
    g2 = kda.la_chunk_backward(*a, d["d_o"], d["S0"], d["dS"])
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(S1, S2)
    for x in g1:
        assert torch.equal(g1[x], g2[x]), x
    _check_prefill(d, o1, S1, BF16)
    _check_grads(d, g1, BF16)


def test_streams_and_graphs():
    """Two streams at once, and a captured forward, backward and step replayed on new inputs."""
    d1, d2 = (lm.inputs(1, 333, 4, 128, 128, BF16, seed=s) for s in (1, 2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        o2, S2 = kda.la_chunk_forward(d2["q"], d2["k"], d2["v"], d2["log_decay"], d2["S0"])
    o1, S1 = kda.la_chunk_forward(d1["q"], d1["k"], d1["v"], d1["log_decay"], d1["S0"])
    torch.cuda.synchronize()
    _check_prefill(d1, o1, S1, BF16)
    _check_prefill(d2, o2, S2, BF16)
    s = {x: t.clone() for x, t in d1.items()}
    pool = s["S0"].clone()

    def call():
        o, S = kda.la_chunk_forward(s["q"], s["k"], s["v"], s["log_decay"], s["S0"])
        g = kda.la_chunk_backward(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], s["S0"], s["dS"])
        step = kda.la_recurrent_step(s["q"][:, 0].contiguous(), s["k"][:, 0].contiguous(),
                                     s["v"][:, 0].contiguous(), s["log_decay"], pool)
        return o, S, g, step

    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S, g, step = call()
    for d in (d1, d2):
        for x, t in d.items():
            s[x].copy_(t)
        pool.copy_(d["S0"])
        graph.replay()
        torch.cuda.synchronize()
        _check_prefill(d, o, S, BF16)
        _check_grads(d, g, BF16)
        one = {x: (t[:, :1] if x in ("q", "k", "v", "d_o") else t) for x, t in d.items()}
        (o_ref, S_ref), (Mo, MS) = lm.reference(one)
        lm.check(step, o_ref[:, 0], 2.0 ** -8 * np.abs(o_ref[:, 0]) + (128 + 16) * 2.0 ** -23 * Mo[:, 0], "step")
        lm.check(pool, S_ref, lm.state_bound(MS, 8), "stepped state")


@pytest.mark.slow
@pytest.mark.parametrize("T,H", [(8192, 4), (20000, 1)])
def test_long(T, H):
    """Long sequences cut into many spans, a head that hardly forgets among them."""
    slopes = [1e-5, 1e-3, 0.01, 0.3][:H]
    d = lm.inputs(1, T, H, 128, 128, BF16, seed=T, slopes=slopes)
    o, S = kda.la_chunk_forward(d["q"], d["k"], d["v"], d["log_decay"], d["S0"])
    torch.cuda.synchronize()
    _check_prefill(d, o, S, BF16)
    g = kda.la_chunk_backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["S0"], d["dS"])
    torch.cuda.synchronize()
    _check_grads(d, g, BF16)


def _some_heads(d, heads):
    """The inputs of these heads alone."""
    axis = {"S0": 1, "dS": 1, "log_decay": 0}
    return {x: t.index_select(axis.get(x, 2), torch.tensor(heads, device="cuda")) for x, t in d.items()}


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_elements_beyond_32_bits(dtype):
    """A last sequence whose elements all lie behind 2^31 others (zeros), and every state but the first."""
    H, tail, heads = 128, 150, [0, 125, 127]
    first = 2 ** 31 // (H * 128)
    d = lm.inputs(1, tail, H, 128, 128, dtype, seed=21, N=2)
    big = {x: torch.zeros(1, first + tail, H, 128, dtype=dtype, device="cuda") for x in ("q", "k", "v", "d_o")}
    for x, t in big.items():
        t[:, first:] = d[x]
    d["S0"][0], d["dS"][0] = 0, 0
    cu = torch.tensor([0, first, first + tail], dtype=torch.int32, device="cuda")
    o, S = kda.la_chunk_forward(big["q"], big["k"], big["v"], d["log_decay"], d["S0"], cu)
    g = kda.la_chunk_backward(big["q"], big["k"], big["v"], d["log_decay"], big["d_o"], d["S0"], d["dS"], cu)
    torch.cuda.synchronize()
    assert not S[0].any() and not g["dinit_state"][0].any() and not o[:, :first].any()
    small = _some_heads({**d, "S0": d["S0"][1:], "dS": d["dS"][1:]}, heads)
    _check_prefill(small, o[:, first:, heads], S[1:, heads], dtype)
    got = {x: g[x][:, first:, heads] for x in ("dq", "dk", "dv")}
    _check_grads(small, {**got, "dinit_state": g["dinit_state"][1:, heads]}, dtype)
    del big, o, g
    torch.cuda.empty_cache()


def test_pool_beyond_32_bits():
    """Slots behind 2^31 floats of the pool give what the first ones do."""
    H = 128
    rows = 2 ** 31 // (H * 128 * 128) + 2
    d = lm.inputs(2, 150, H, 128, 128, BF16, seed=22)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    one = (*(d[x][:, 0].contiguous() for x in "qkv"), d["log_decay"])
    pool = torch.zeros(rows, H, 128, 128, device="cuda")
    got = []
    for table in ([0, 1], [rows - 1, rows - 2]):
        slots = torch.tensor(table, dtype=torch.int32, device="cuda")
        pool[table] = d["S0"]
        o = kda.la_chunk_forward_slots(*a, pool, slots)
        after = pool[table]
        step = kda.la_recurrent_step_slots(*one, pool, slots)
        got.append((o, after, step, pool[table]))
        pool[table] = 0
        assert kda.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert not pool.any()
    del pool
    torch.cuda.empty_cache()
