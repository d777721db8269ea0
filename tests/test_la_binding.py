"""The Python binding of linear attention and group norm: what it does without a GPU."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda

Q = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
ONE = Q[:, 0].contiguous()
LG, STATE, SLOTS = torch.zeros(2), torch.zeros(1, 2, 64, 64), torch.zeros(1, dtype=torch.int32)
X, STAT = torch.zeros(4, 6, 30), torch.zeros(4, 3)
CALLS = {
    "la_chunk_forward": ((Q, Q, Q, LG), ["q", "k", "v", "log_decay"]),
    "la_chunk_forward_slots": ((Q, Q, Q, LG, STATE, SLOTS), ["q", "k", "v", "log_decay", "state_pool", "slots"]),
    "la_chunk_backward": ((Q, Q, Q, LG, Q), ["q", "k", "v", "log_decay", "d_o"]),
    "la_recurrent_step": ((ONE, ONE, ONE, LG, STATE), ["q", "k", "v", "log_decay", "state"]),
    "la_recurrent_step_slots": ((ONE, ONE, ONE, LG, STATE, SLOTS), ["q", "k", "v", "log_decay", "state_pool", "slots"]),
    "group_norm": ((X, 3), ["x"]),
    "group_norm_backward": ((X, X, STAT, STAT, 3), ["dy", "x", "mean", "rstd"]),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_delta_rule_85_b200.build import build
    build()


@pytest.mark.parametrize("call", CALLS)
def test_required_tensors_are_named(call):
    args, names = CALLS[call]
    with pytest.raises(ValueError, match="CUDA"):   # all given: refused for where they are
        getattr(kda, call)(*args)
    for i, name in enumerate(names):
        for other in (None, 1.0):
            bad = list(args)
            bad[i] = other
            with pytest.raises(ValueError, match=f"{name} is required"):
                getattr(kda, call)(*bad)
