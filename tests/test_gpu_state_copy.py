"""Pages of a pool of states: copies are exact, and what no pair names keeps its bits."""

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import require_cuda

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    require_cuda()
    yield
    torch.cuda.synchronize()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def copied(S, src, dst, dim):
    out, old = S.clone(), S
    for a, b in zip(src, dst):
        if b >= 0:
            out.select(dim, b).copy_(old.select(dim, a) if a >= 0 else torch.zeros_like(
                old.select(dim, b)))
    return out


@pytest.mark.parametrize("shape,dim", [((9, 2, 128, 128), 0), ((3, 9, 1, 64, 64), 1),
                                       ((9, 4), 0), ((2, 9, 3, 7, 4), 1), ((9, 8191, 4), 0)])
def test_copy_fork_clear(shape, dim):
    S = torch.randn(shape, device=DEV)
    for src, dst in (([0], [3]), ([2] * 5, [0, 1, 3, 8, 4]), ([-1, 5, -1], [0, 6, 8]),
                     ([4, 1, 7], [-1, -1, 0]), ([3, 3], [3, 2]), ([], [])):
        ref = copied(S, src, dst, dim)
        if src == [3, 3]:   # a page onto itself while another reads it: left out, with an error
            kda.state_copy(S, ints(src), ints(dst), page_dim=dim)
            assert kda.get_device_error() == 7
            continue
        kda.state_copy(S, ints(src), ints(dst), page_dim=dim)
        assert kda.get_device_error() == 0
        assert torch.equal(S, ref)


def test_conflicts_and_ranges_are_left_out():
    for src, dst, good in (([0, 1], [5, 5], []), ([0, 5], [5, 6], []), ([0, 1, 2], [9, 3, 4], [1, 2]),
                           ([9, 1], [3, 4], [1]), ([-2, 1], [3, 4], [1]), ([0, 1], [-2, 4], [1]),
                           ([-1, 3, 6], [3, 7, 8], [2]), ([0, 1], [1, 0], [])):
        S = torch.randn(9, 1000, device=DEV)
        ref = copied(S, [src[i] for i in good], [dst[i] for i in good], 0)
        kda.state_copy(S, ints(src), ints(dst))
        assert kda.get_device_error() == 7, (src, dst)
        assert torch.equal(S, ref), (src, dst)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8, torch.float64])
def test_other_types(dtype):
    S = torch.randint(0, 100, (5, 3, 16), device=DEV).to(dtype)
    ref = copied(S, [1, -1], [0, 4], 0)
    kda.state_copy(S, ints([1, -1]), ints([0, 4]))
    assert torch.equal(S, ref)


def test_offsets_beyond_32_bits():
    """Pages behind the first 4 GiB."""
    S = torch.zeros(36, 1 << 25, device=DEV)            # 128 MiB pages, 4.5 GiB
    S[35] = torch.arange(1 << 25, device=DEV)
    kda.state_copy(S, ints([35, 35]), ints([0, 34]))
    assert torch.equal(S[0], S[35]) and torch.equal(S[34], S[35]) and not S[33].any()


def test_compaction_then_decode():
    """A pool compacted by the plan decodes as the sequences did in their old places."""
    r = np.random.default_rng(0)
    P, H = 12, 2
    S = 0.1 * torch.randn(P, H, 128, 128, device=DEV)
    live = r.random(P) < 0.6
    old = S.clone()
    src, dst, where = kda.plan_compaction(live)
    kda.state_copy(S, ints(src), ints(dst))
    n = int(live.sum())
    x = [torch.randn(n, H, 128, device=DEV) for _ in range(3)]
    g = -torch.rand(n, H, device=DEV)
    keep = torch.tensor([p for p in range(P) if live[p]], device=DEV)
    at = torch.tensor([where[p] for p in range(P) if live[p]], device=DEV)
    ref_S = old[keep].contiguous()
    ref = kda.linear_decode(*x, g, ref_S)
    back = torch.argsort(at)           # row i of the compacted pool is live page keep[back[i]]
    got_S = S[:n]
    got = kda.linear_decode(*[t[back].contiguous() for t in x], g[back].contiguous(), got_S)
    assert torch.equal(got, ref[back]) and torch.equal(got_S, ref_S[back])
    assert kda.get_device_error() == 0


def test_capture():
    S = torch.randn(6, 256, device=DEV)
    src, dst = ints([0, 0, 0]), ints([3, -1, 4])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.state_copy(S, src, dst)
    src.copy_(ints([1, -1, 2]))
    dst.copy_(ints([5, 0, -1]))
    ref = copied(S, [1, -1], [5, 0], 0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, ref)


def test_refusals():
    S = torch.zeros(4, 3, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.state_copy(S, ints([0]), ints([1]))          # 12-byte pages
    S = torch.zeros(4, 8, device=DEV)
    with pytest.raises(TypeError):
        kda.state_copy(S, ints([0]).long(), ints([1]))
    with pytest.raises(ValueError):
        kda.state_copy(S, ints([0]), ints([1, 2]))
    with pytest.raises(ValueError):
        kda.state_copy(S.t(), ints([0]), ints([1]))
    with pytest.raises(ValueError):
        kda.state_copy(S, ints([0]), ints([1]), page_dim=2)
    with pytest.raises(kda.KdaError):
        kda.state_copy(S, S.view(-1).view(torch.int32)[:1], ints([1]))
