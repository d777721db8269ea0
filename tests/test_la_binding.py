"""The Python binding of linear attention and group norm: what it does without a GPU."""
import os

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


@pytest.mark.parametrize("case", ["missing", "another torch", "no library"])
def test_calls_go_on_without_the_short_way(case, monkeypatch, tmp_path):
    kda.load_library()
    monkeypatch.setattr(kda, "_fast", None)
    if case == "another torch":
        monkeypatch.setattr(torch, "__version__", "0.0")
    else:
        monkeypatch.setattr(kda, "_HERE", str(tmp_path))
    if case == "no library":
        (tmp_path / "_kda_fast.so").write_bytes(b"not a library")
    with pytest.warns(UserWarning, match="_kda_fast.so"):
        with pytest.raises(ValueError, match="CUDA"):
            kda.la_chunk_forward(Q, Q, Q, LG)
    for call, (args, _) in CALLS.items():   # no second warning, and every call by its Python way
        with pytest.raises(ValueError, match="CUDA"):
            getattr(kda, call)(*args)


def test_short_way_is_built_again_for_another_torch(monkeypatch):
    from gated_delta_rule_85_b200 import build

    sources = [os.path.join(build.HERE, "csrc", "kda_fast.cpp")]
    assert not build._fast_stale(sources)
    assert kda._load_fast().built_for == build._built_for()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    assert build._fast_stale(sources)
