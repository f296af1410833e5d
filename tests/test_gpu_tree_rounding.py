"""What the one tf32 product of bf16 trees loses: each factor is rounded to tf32, to nearest, so it
is off by at most 2^-11 of its value to either side, and the output by a half step (2^-8) more."""

import math

import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import require_cuda

pytestmark = pytest.mark.gpu
DEV, D = "cuda", 128


@pytest.fixture(autouse=True)
def _gpu():
    require_cuda()
    yield
    torch.cuda.synchronize()


def one_hot(N, T, H):
    """Rows [N, T, H, 128] with a single 1, in a channel of its own for each unit."""
    x = torch.zeros(N, T, H, D, device=DEV, dtype=torch.bfloat16)
    c = (torch.arange(N * H, device=DEV) * 37 % D).view(N, 1, H, 1).expand(N, T, H, 1)
    return x.scatter_(3, c, 1.0), c


@pytest.mark.parametrize("N,H", [(2, 3), (20, 8)])   # two blocks per unit, and one
def test_state_factor(N, H):
    """o = one element of S, all other terms zero."""
    q, c = one_hot(N, 1, H)
    zero = torch.zeros_like(q)
    g = torch.Generator().manual_seed(N)
    S = torch.randn(N, H, D, D, generator=g).to(DEV)
    S[..., ::2] = 1 + 2.0 ** -8 + 2.0 ** -10 - 2.0 ** -23   # just below a tf32 value, above a bf16 tie
    o = kda.decode_tree(q, zero, zero, zero.float(), zero[..., 0].contiguous(),
                        torch.full((N, 1), -1, dtype=torch.int32, device=DEV), S)
    assert kda.get_device_error() == 0
    ref = S.gather(2, c[:, 0, :, :, None].expand(N, H, 1, D))[:, :, 0].double()
    off = ((o[:, 0].double() - ref) / ref).abs().max().item()
    assert off <= (1 + 2.0 ** -11) * (1 + 2.0 ** -8) - 1


def test_quotient_factor():
    """A child's read-out of its parent's write: (q d_1) (k / d_0) u_0 with d_1 = d_0, so only the
    roundings of d_0 and 1 / d_0 are left. Over n units their mean is that of n independent errors
    of at most 2^-11 to either side, evenly spread: a standard deviation of 2^-11 sqrt(2 / 3 / n) (two
    factors), and the outputs' own, 2^-8 / sqrt(3 / (128 n)) at most. Six of both: 8e-5 (a factor cut
    off instead of rounded is off by 3.5e-4 on average)."""
    N, H = 64, 32
    n = N * H
    x, c = one_hot(N, 2, H)
    q, k = x.clone(), x
    q[:, 0] = 0
    k[:, 1] = 0
    g = torch.Generator().manual_seed(0)
    gate = torch.zeros(N, 2, H, D, device=DEV)
    gate[:, 0] = (-3 * torch.rand(N, H, 1, generator=g)).to(DEV)
    v = torch.randn(N, 2, H, D, generator=g).bfloat16().to(DEV)
    beta = torch.sigmoid(torch.randn(N, 2, H, generator=g)).bfloat16().to(DEV)
    S = torch.zeros(N, H, D, D, device=DEV)
    parents = torch.tensor([[-1, 0]] * N, dtype=torch.int32, device=DEV)
    o = kda.decode_tree(q, k, v, gate, beta, parents, S)
    assert kda.get_device_error() == 0
    ref = beta[:, 0, :, None].double() * v[:, 0].double()
    off = ((o[:, 1].double() - ref) / ref)[ref != 0]
    assert off.abs().max().item() <= (1 + 2.0 ** -11) ** 2 * (1 + 2.0 ** -8) * (1 + 2.0 ** -20) - 1
    bound = 6 * (2.0 ** -11 * math.sqrt(2 / 3 / n) + 2.0 ** -8 / math.sqrt(3 * 128 * n))
    assert abs(off.mean().item()) <= bound
