"""Refusals of the linear-attention and group-norm calls: the C ABI (host checks, nothing is
launched) and the Python binding (CPU)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, WORKSPACE = 0, -1, -2, -3, -4, -5
A = [0x10000 * (i + 1) for i in range(16)]   # aligned addresses that nothing dereferences
WS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_85_b200.build import build
    build()
    return kda.load_library()


def prefill(lib, **over):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], s0=A[4], o=A[5], fs=A[6], cu=None, B=1, T=256, H=2, dk=128, dv=128, N=1,
             dtype=0, ws=A[7], wsb=WS)
    a.update(over)
    return lib.kda_la_chunk_forward(*(a[x] for x in ("q", "k", "v", "g", "s0", "o", "fs", "cu", "B", "T", "H", "dk",
                                                     "dv", "N", "dtype", "ws", "wsb")), None)


PREFILL_BAD = [
    (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(o=None), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(N=2), INVALID), (dict(cu=A[8], B=2, N=2), INVALID), (dict(cu=A[8], N=0), INVALID),
    (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(B=65536, N=65536), UNSUPPORTED), (dict(H=70000), UNSUPPORTED), (dict(B=60000, N=60000, T=60000), UNSUPPORTED),
    (dict(k=A[1] + 8), MISALIGNED), (dict(fs=A[6] + 4), MISALIGNED), (dict(g=A[3] + 2), MISALIGNED),
    (dict(cu=A[8] + 2), MISALIGNED), (dict(ws=A[7] + 64), MISALIGNED), (dict(ws=None), WORKSPACE),
    (dict(wsb=1000), WORKSPACE),
]


@pytest.mark.parametrize("over,code", PREFILL_BAD)
def test_prefill_rejects(lib, over, code):
    assert prefill(lib, **over) == code
    assert lib.kda_last_error().decode() != ""


def slots(lib, **over):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], pool=A[4], slots=A[5], o=A[6], cu=None, B=1, T=256, H=2, dk=128, dv=128,
             N=1, ns=4, dtype=0, ws=A[7], wsb=WS)
    a.update(over)
    return lib.kda_la_chunk_forward_slots(*(a[x] for x in ("q", "k", "v", "g", "pool", "slots", "o", "cu", "B", "T",
                                                           "H", "dk", "dv", "N", "ns", "dtype", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [(dict(pool=None), INVALID), (dict(slots=None), INVALID), (dict(ns=0), INVALID),
                                       (dict(slots=A[5] + 1), MISALIGNED), (dict(pool=A[4] + 4), MISALIGNED),
                                       (dict(dk=32), UNSUPPORTED), (dict(ws=None), WORKSPACE)])
def test_slots_rejects(lib, over, code):
    assert slots(lib, **over) == code


def test_slots_workspace_holds_the_states(lib):
    f = lib.kda_la_chunk_forward_workspace_size
    assert f(4, 300, 8, 64, 128, 4, 0, 1) == f(4, 300, 8, 64, 128, 4, 0, 0) + 4 * 8 * 64 * 128 * 4
    # one chunk a sequence: nothing is carried from CTA to CTA
    assert f(4, 128, 8, 64, 128, 4, 0, 1) == 0 and f(4, 64, 8, 64, 128, 4, 1, 1) == 0 < f(4, 65, 8, 64, 128, 4, 1, 0)
    assert f(1, 1 << 20, 32, 128, 128, 1, 0, 0) == f(1, 256, 32, 128, 128, 1, 0, 0)   # not a function of T
    assert f(1, 0, 8, 64, 64, 1, 0, 0) == 0 and f(1, 64, 8, 96, 64, 1, 0, 0) == 0


def backward(lib, **over):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], s0=A[4], do=A[5], ds=A[6], dq=A[7], dkk=A[8], dvv=A[9], di=A[10], cu=None,
             B=1, T=256, H=2, dk=128, dv=128, N=1, dtype=0, ws=A[11], wsb=WS)
    a.update(over)
    return lib.kda_la_chunk_backward(*(a[x] for x in ("q", "k", "v", "g", "s0", "do", "ds", "dq", "dkk", "dvv", "di",
                                                      "cu", "B", "T", "H", "dk", "dv", "N", "dtype", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [(dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dkk=None), INVALID),
                                       (dict(dvv=None), INVALID), (dict(dvv=A[9] + 2), MISALIGNED),
                                       (dict(di=A[10] + 8), MISALIGNED), (dict(ds=A[6] + 4), MISALIGNED),
                                       (dict(dv=72), UNSUPPORTED), (dict(wsb=64), WORKSPACE)])
def test_backward_rejects(lib, over, code):
    assert backward(lib, **over) == code


def step(lib, **over):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], s=A[4], o=A[5], N=4, H=2, dk=128, dv=128, dtype=0)
    a.update(over)
    return lib.kda_la_recurrent_step(*(a[x] for x in ("q", "k", "v", "g", "s", "o", "N", "H", "dk", "dv", "dtype")),
                                     None)


@pytest.mark.parametrize("over,code", [(dict(s=None), INVALID), (dict(N=-1), INVALID), (dict(dk=32), UNSUPPORTED),
                                       (dict(dtype=9), UNSUPPORTED), (dict(s=A[4] + 4), MISALIGNED),
                                       (dict(g=A[3] + 1), MISALIGNED), (dict(N=1 << 20, H=1 << 12), UNSUPPORTED)])
def test_step_rejects(lib, over, code):
    assert step(lib, **over) == code


def test_step_slots_rejects(lib):
    f = lib.kda_la_recurrent_step_slots
    assert f(A[0], A[1], A[2], A[3], A[4], None, A[5], 4, 2, 64, 64, 8, 0, None) == INVALID
    assert f(A[0], A[1], A[2], A[3], A[4], A[6], A[5], 4, 2, 64, 64, 0, 0, None) == INVALID
    assert f(A[0], A[1], A[2], A[3], A[4], A[6] + 2, A[5], 4, 2, 64, 64, 8, 0, None) == MISALIGNED
    assert f(None, None, None, None, None, None, None, 0, 2, 64, 64, 8, 0, None) == OK


def norm(lib, **over):
    a = dict(x=A[0], w=A[1], b=A[2], gate=A[3], y=A[4], m=A[5], r=A[6], N=8, L=100000, C=64, G=4, eps=1e-5, act=1, dtype=0,
             ws=A[7], wsb=WS)
    a.update(over)
    return lib.kda_group_norm_forward(*(a[x] for x in ("x", "w", "b", "gate", "y", "m", "r", "N", "L", "C", "G", "eps",
                                                       "act", "dtype", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(m=None), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID),
    (dict(L=0), INVALID), (dict(N=-1), INVALID), (dict(act=3), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(C=1 << 25, G=1), UNSUPPORTED),
    (dict(N=1 << 40), UNSUPPORTED), (dict(x=A[0] + 2), MISALIGNED), (dict(gate=A[3] + 8), MISALIGNED),
    (dict(w=A[1] + 2), MISALIGNED), (dict(r=A[6] + 1), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
    (dict(N=0, x=None, y=None), OK),
])
def test_norm_rejects(lib, over, code):
    assert norm(lib, **over) == code


def norm_back(lib, **over):
    a = dict(dy=A[0], x=A[1], m=A[2], r=A[3], w=A[4], b=A[5], gate=A[6], dx=A[7], dg=A[8], dw=A[9], db=A[10], N=8, L=100000,
             C=64, G=4, act=1, dtype=0, ws=A[11], wsb=WS)
    a.update(over)
    return lib.kda_group_norm_backward(*(a[x] for x in ("dy", "x", "m", "r", "w", "b", "gate", "dx", "dg", "dw", "db",
                                                        "N", "L", "C", "G", "act", "dtype", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [(dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dg=None), INVALID),
                                       (dict(r=None), INVALID), (dict(dg=A[8] + 4), MISALIGNED),
                                       (dict(dw=A[9] + 2), MISALIGNED), (dict(ws=None), WORKSPACE)])
def test_norm_backward_rejects(lib, over, code):
    assert norm_back(lib, **over) == code


def test_python_refuses_host_tensors_and_shapes(lib):
    q = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    lg = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.la_chunk_forward(q, q, q, lg)
    with pytest.raises(ValueError, match="log_decay"):
        kda.la_chunk_forward(q, q, q, torch.zeros(3))
    with pytest.raises(ValueError, match="log_decay"):
        kda.la_chunk_forward(q, q, q, torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="k must be"):
        kda.la_chunk_forward(q, q[:, :4], q, lg)
    with pytest.raises(ValueError, match="v must be"):
        kda.la_chunk_forward(q, q, q.float(), lg)
    with pytest.raises(TypeError):
        kda.la_chunk_forward(q.half(), q.half(), q.half(), lg)
    with pytest.raises(ValueError, match="init_state"):
        kda.la_chunk_forward(q, q, q, lg, torch.zeros(2, 2, 64, 64))
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.la_chunk_forward(q, q, q, lg, None, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots"):
        kda.la_chunk_forward_slots(q, q, q, lg, torch.zeros(4, 2, 64, 64), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="d_o"):
        kda.la_chunk_backward(q, q, q, lg, q[:, :3])
    with pytest.raises(ValueError, match="state"):
        kda.la_recurrent_step(q[:, 0], q[:, 0], q[:, 0], lg, torch.zeros(1, 2, 64, 128))
    x = torch.zeros(4, 6, 30)
    with pytest.raises(ValueError, match="groups"):
        kda.group_norm(x, 7)
    with pytest.raises(ValueError, match="activation"):
        kda.group_norm(x, 3, activation="relu")
    with pytest.raises(ValueError, match="eps"):
        kda.group_norm(x, 3, eps=0.0)
    with pytest.raises(ValueError, match="weight"):
        kda.group_norm(x, 3, torch.zeros(6))
    with pytest.raises(ValueError, match="gate"):
        kda.group_norm(x, 3, gate=torch.zeros(4, 6, 15))
    with pytest.raises(ValueError, match="CUDA"):
        kda.group_norm(x, 3)
    with pytest.raises(ValueError, match="position"):
        kda.group_norm(torch.zeros(4, 0, 30), 3)
    with pytest.raises(ValueError, match="mean"):
        kda.group_norm_backward(x, x, torch.zeros(4, 2), torch.zeros(4, 3), 3)
