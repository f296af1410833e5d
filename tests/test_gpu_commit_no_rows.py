"""Commits without rows: an empty path leaves its state, and one that names a row is reported."""

import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import require_cuda

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_paths_into_no_rows(dtype):
    require_cuda()
    S = torch.randn(3, 2, 128, 128, device=DEV)
    before = S.clone()
    k = torch.empty(3, 0, 2, 128, device=DEV, dtype=dtype)
    for path, code in (([[-1, 4], [-1, -1], [-3, 0]], 0), ([[-1, 4], [0, -1], [-1, -1]], 7)):
        p = torch.tensor(path, dtype=torch.int32, device=DEV)
        kda.commit_path(k, k, k.float(), k[..., 0].contiguous(), p, S)
        assert kda.get_device_error() == code, path
        assert torch.equal(S, before)
    kda.commit_path(k, k, k.float(), k[..., 0].contiguous(), p[:, :0].contiguous(), S)
    assert kda.get_device_error() == 0 and torch.equal(S, before)
