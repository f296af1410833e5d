"""Packed prompts of linear attention leave the same bits at every launch, and the oracle's values:
each block of the chunk kernel looks its document up in shared memory before its copies start."""

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import TOL_BF16, TOL_F32, host, rel_l2, require_cuda
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("docs", [2, 100, 128])
def test_packed_launches_repeat_themselves(docs):
    require_cuda()
    r = np.random.default_rng(docs)
    lens = [int(x) for x in r.integers(40, 300, size=docs)]
    g = torch.Generator().manual_seed(docs)
    T, H, Hk = sum(lens), 4, 2
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(n(1, T, Hk, 128)).bfloat16().to(DEV) for _ in range(2))
    v = n(1, T, H, 64).bfloat16().to(DEV)
    gate = -torch.nn.functional.softplus(n(1, T, H) - 2).to(DEV)
    h0 = (0.05 * n(docs, H, 128, 64)).to(DEV)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=DEV)
    first = kda.linear_fwd(q, k, v, gate, h0=h0, cu_seqlens=cu)
    ro, rh = linear_attention(host(q), host(k), host(v), host(gate), host(h0), cu.cpu().numpy())
    assert rel_l2(host(first[0]), ro) <= TOL_BF16 and rel_l2(host(first[1]), rh) <= TOL_F32
    for _ in range(30):
        o, hT = kda.linear_fwd(q, k, v, gate, h0=h0, cu_seqlens=cu)
        assert torch.equal(o, first[0]) and torch.equal(hT, first[1])
    assert kda.get_device_error() == 0
