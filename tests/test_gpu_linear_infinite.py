"""An infinite value of v in linear attention with odd key widths: the walk's state has no rows
behind dk, so nothing there turns an infinite output into NaN."""

import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import require_cuda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows(B, T, H, dk, dv, dtype):
    g = torch.Generator().manual_seed(dk)
    u = lambda *s: torch.rand(s, generator=g) + 0.1  # noqa: E731
    x = dict(q=u(B, T, H, dk).to(dtype), k=u(B, T, H, dk).to(dtype), v=u(B, T, H, dv).to(dtype),
             log_g=-0.02 * u(B, T, H), h0=u(B, H, dk, dv))
    return {a: b.to(DEV) for a, b in x.items()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T,dk,dv", [(5, 20, 8), (70, 20, 7), (400, 33, 8), (300, 100, 12),
                                     (50, 129, 16), (90, 7, 64)])   # (none for the tensor-core kernel)
def test_infinite_value(T, dk, dv, dtype, sign):
    """All of q and k are positive: the outputs of the column from its token on, and its last
    states, are that infinity; the rest is as without it (two orders of the same sums: up to 400
    tokens with two roundings of 2^-24 each, 4.8e-5, and one step of a bf16 output)."""
    require_cuda()
    x = rows(1, T, 2, dk, dv, dtype)
    ro, rh = kda.linear_fwd(**x)
    t, c = T // 2, 3
    x["v"][0, t, 1, c] = sign * float("inf")
    o, hT = kda.linear_fwd(**x)
    S = x["h0"].clone()
    od = kda.linear_decode(x["q"], x["k"], x["v"], x["log_g"], S)
    for out, last in ((o, hT), (od, S)):
        assert (out[0, t:, 1, c] == sign * float("inf")).all()
        assert (last[0, 1, :, c] == sign * float("inf")).all()
        keep, kept = torch.ones_like(o, dtype=torch.bool), torch.ones_like(hT, dtype=torch.bool)
        keep[0, t:, 1, c] = False
        kept[0, 1, :, c] = False
        torch.testing.assert_close(out[keep], ro[keep], rtol=2 ** -7 if dtype == torch.bfloat16 else 4.8e-5, atol=1e-5)
        torch.testing.assert_close(last[kept], rh[kept], rtol=4.8e-5, atol=1e-6)
    assert kda.get_device_error() == 0
