"""What a refusal of the linear-attention calls names (C ABI; host checks, nothing is launched)."""
import pytest

import test_la_abi as abi
from test_la_abi import A, lib  # noqa: F401  (the fixture)


@pytest.mark.parametrize("call,over,names,others", [
    (abi.prefill, dict(g=None), ["log_decay"], ["beta", "log_alpha"]),
    (abi.prefill, dict(g=A[3] + 2), ["log_decay is not 4-byte"], []),
    (abi.prefill, dict(s0=A[4] + 4), ["init_state is not 16-byte"], []),
    (abi.prefill, dict(fs=A[6] + 4), ["final_state is not 16-byte"], []),
    (abi.slots, dict(o=None), ["log_decay and o"], ["beta"]),
    (abi.slots, dict(pool=A[4] + 4), ["state_pool is not 16-byte"], ["init_state"]),
    (abi.backward, dict(do=None), ["d_o"], ["beta", "log_alpha"]),
    (abi.backward, dict(do=A[5] + 2), ["d_o is not 16-byte"], []),
    (abi.backward, dict(ds=A[6] + 4), ["dfinal_state is not 16-byte"], []),
    (abi.step, dict(g=None), ["log_decay", "state"], ["beta", "log_alpha"]),
    (abi.step, dict(g=A[3] + 1), ["log_decay is not 4-byte"], []),
    (abi.step, dict(s=A[4] + 4), ["state is not 16-byte"], []),
])
def test_message_names_the_argument(lib, call, over, names, others):  # noqa: F811
    assert call(lib, **over) != 0
    text = lib.kda_last_error().decode()
    assert all(n in text for n in names) and not any(n in text for n in others), text


def test_pool_step_names_the_pool(lib):  # noqa: F811
    f = lib.kda_la_recurrent_step_slots
    assert f(A[0], A[1], A[2], None, A[4], A[6], A[5], 4, 2, 64, 64, 8, 0, None) != 0
    text = lib.kda_last_error().decode()
    assert "log_decay" in text and "state_pool" in text and "beta" not in text


def test_delta_rule_names_stay(lib):  # noqa: F811
    f = lib.kda_recurrent_step
    assert f(A[0], A[1], A[2], None, A[4], A[5], A[6], 4, 2, 64, 64, 0, None) != 0
    assert "log_alpha, beta, state and o are required" in lib.kda_last_error().decode()
    assert f(A[0], A[1], A[2], A[3] + 4, A[4], A[5], A[6], 4, 2, 64, 64, 0, None) != 0
    assert "log_alpha is not 16-byte aligned" in lib.kda_last_error().decode()


@pytest.mark.parametrize("B,T,H,N", [(1, 300, 70000, 1), (65536, 300, 4, 65536), (60000, 60000, 4, 60000)])
def test_sizes_that_are_refused_need_nothing(lib, B, T, H, N):  # noqa: F811
    """A caller that allocates first gets the refusal, not an allocation that cannot be had."""
    for slots in (0, 1):
        assert lib.kda_la_chunk_forward_workspace_size(B, T, H, 128, 128, N, 0, slots) == 0
    assert lib.kda_la_chunk_backward_workspace_size(B, T, H, 128, 128, N, 0) == 0
    assert abi.prefill(lib, B=B, T=T, H=H, N=N, ws=None, wsb=0) == abi.UNSUPPORTED
    assert abi.slots(lib, B=B, T=T, H=H, N=N, ws=None, wsb=0) == abi.UNSUPPORTED
    assert abi.backward(lib, B=B, T=T, H=H, N=N, ws=None, wsb=0) == abi.UNSUPPORTED
