"""Sizes that a C int does not hold are refused by the binding of the serving operators (truncated,
a call would work on the first rows, layers or pages and report nothing). Shapes only: the
tensors have no storage, and the checks that need a GPU are stood in for."""

import pytest
import torch

import gated_delta_rule_144_b200 as kda

BIG = (1 << 32) + 5


@pytest.fixture(autouse=True)
def shapes_only(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise AssertionError("reached the library: " + name)

    monkeypatch.setattr(kda, "_dev", lambda t, *_: t)
    monkeypatch.setattr(kda, "lib", lambda: Library())


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


F, I = torch.float32, torch.int32


@pytest.mark.parametrize("call", [
    lambda: kda.linear_fwd(t(1, BIG, 1, 1), t(1, BIG, 1, 1), t(1, BIG, 1, 1), t(1, BIG, 1, dtype=F)),
    lambda: kda.linear_fwd(t(1, 4, 1, 1), t(1, 4, 1, 1), t(1, 4, 1, 1), t(1, 4, 1, dtype=F),
                           cu_seqlens=t(BIG, dtype=I)),
    lambda: kda.linear_decode(t(BIG, 1, 8), t(BIG, 1, 8), t(BIG, 2, 8), t(2, dtype=F),
                              t(BIG, 2, 8, 8, dtype=F)),
    lambda: kda.linear_decode(t(1, 1, 8), t(1, 1, 8), t(1, BIG, 8), t(BIG, dtype=F),
                              t(1, BIG, 8, 8, dtype=F)),
    lambda: kda.decode_tree(*[t(BIG, 1, 1, 128)] * 3, t(BIG, 1, 1, 128, dtype=F), t(BIG, 1, 1),
                            t(BIG, 1, dtype=I), t(BIG, 1, 128, 128, dtype=F)),
    lambda: kda.commit_path(*[t(1, BIG, 1, 128)] * 2, t(1, BIG, 1, 128, dtype=F), t(1, BIG, 1),
                            t(1, 2, dtype=I), t(1, 1, 128, 128, dtype=F)),
    lambda: kda.commit_path(*[t(1, 4, 1, 128)] * 2, t(1, 4, 1, 128, dtype=F), t(1, 4, 1),
                            t(1, BIG, dtype=I), t(1, 1, 128, 128, dtype=F)),
    lambda: kda.state_copy(t(BIG, 4, dtype=F), t(2, dtype=I), t(2, dtype=I)),
    lambda: kda.state_copy(t(1 << 20, 1 << 13, 2, 4, dtype=F), t(2, dtype=I), t(2, dtype=I),
                           page_dim=2),
    lambda: kda.state_copy(t(4, 4, dtype=F), t(BIG, dtype=I), t(BIG, dtype=I)),
])
def test_refused(call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()
