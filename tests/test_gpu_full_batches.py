"""The forms that full batches run, against the float64 oracles: trees with one block per state,
commits whose blocks take several states one after another, and packed prompts of more documents
than a block reads the offsets of.

Tolerances (relative L2), as for the small batches: 5e-3 for bf16 outputs, 1e-5 for fp32 ones and
for states.
"""

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
import oracle
from kda_testutil import TOL_BF16, TOL_F32, host, rel_l2, require_cuda
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_cuda()
    yield
    torch.cuda.synchronize()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def make(N, T, H, dtype, seed, mu=0.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(n(N, T, H, 128)).to(DT[dtype]), k=unit(n(N, T, H, 128)).to(DT[dtype]),
             v=n(N, T, H, 128).to(DT[dtype]),
             log_g=-torch.nn.functional.softplus(n(N, T, H, 128) + mu),
             beta=torch.sigmoid(n(N, T, H)).to(DT[dtype]), S=0.05 * n(N, H, 128, 128))
    return {a: b.to(DEV) for a, b in x.items()}


class Walk:
    """The oracle along rows of one sequence."""

    def __init__(self, x):
        self.x = {a: host(x[a]) for a in ("q", "k", "v", "log_g", "beta", "S")}

    def __call__(self, n, rows):
        f = lambda a: self.x[a][n:n + 1, rows]  # noqa: E731
        return oracle.kda_fwd(f("q"), f("k"), f("v"), f("log_g"), f("beta"),
                              h0=self.x["S"][n:n + 1])


def leaves_first_paths(row):
    """Paths from the root that together pass every node, each as long as it can be."""
    parents = {int(p) for p in row}
    for i in range(len(row)):
        if row[i] != -2 and i not in parents:
            up = []
            j = i
            while j >= 0:
                up.append(j)
                j = int(row[j])
            yield up[::-1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("steep", [False, True])
@pytest.mark.parametrize("T", [1, 7, 16, 17, 32, 33, 64])
def test_trees(T, steep, dtype):
    """Sequences of all sizes, one without nodes, one rejected; with `steep` every other tree has
    gates that clear the state."""
    N, H = 40, 2
    assert 2 * N * H > sms()
    x = make(N, T, H, dtype, seed=T, mu=2.0 if steep else 0.0)
    r = np.random.default_rng(T)
    parents = np.full((N, T), -2, np.int32)
    for n in range(N):
        m = T if n % 3 == 0 else int(r.integers(1, T + 1))
        for i in range(m):
            parents[n, i] = max(-1, i - int(r.integers(1, 5)))
        if steep and n % 2:
            x["log_g"][n, int(r.integers(0, m)), :, ::5] = -float("inf")
    parents[5] = -2
    parents[6, 0] = 0
    before = torch.randn(N, T, H, 128, device=DEV).to(DT[dtype])
    S0 = x["S"].clone()
    p = torch.tensor(parents, device=DEV)
    args = (x["q"], x["k"], x["v"], x["log_g"], x["beta"], p, x["S"])
    o = kda.decode_tree(*args, o=before.clone())
    assert kda.get_device_error() == 7
    walk, got = Walk(x), host(o)
    ref, seen = got.astype(np.float64), np.zeros((N, T), dtype=bool)
    for n in range(N):
        if n == 6:
            continue
        for path in leaves_first_paths(parents[n]):
            ref[n, path] = walk(n, path)[0][0]
            seen[n, path] = True
    there = parents != -2
    there[6] = False
    assert (seen == there).all()
    assert rel_l2(got[there], ref[there]) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    for n in range(N):   # each by itself: a wrong one is not hidden by the rest
        if there[n].any():
            assert rel_l2(got[n, there[n]], ref[n, there[n]]) <= (
                TOL_BF16 if dtype == "bf16" else TOL_F32), n
    gone = torch.tensor(~there, device=DEV)
    assert torch.equal(o[gone], before[gone]) and torch.equal(x["S"], S0)
    new = kda.decode_tree(*args)
    assert kda.get_device_error() == 7
    assert torch.equal(new[~gone], o[~gone]) and not new[gone].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H", [(1300, 1), (80, 16)])
def test_commits(N, H, dtype):
    """Every block takes four states or more, with paths of none to twelve rows between paths that
    are empty or leave the rows."""
    T, A = 9, 12
    assert N * H >= 4 * 2 * sms()
    x = make(N, T, H, dtype, seed=N)
    r = np.random.default_rng(N)
    path = np.full((N, A), -1, np.int32)
    rows = []
    for n in range(N):
        m = int(r.choice([0, 0, 1, 3, 4, 5, 7, 8, 9, 12]))
        rows.append([int(i) for i in r.integers(0, T, size=m)])
        path[n, :m] = rows[n]
        if m and n % 7 == 3:
            path[n, int(r.integers(0, m))] = T + int(r.integers(0, 3))
            rows[n] = []
    bad = any(len(a) == 0 and (b >= T).any() for a, b in zip(rows, path))
    before = x["S"].clone()
    kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], torch.tensor(path, device=DEV), x["S"])
    assert bad and kda.get_device_error() == 7
    after = x["S"]
    x["S"] = before
    walk, got = Walk(x), host(after)
    for n in range(N):
        if rows[n]:
            for h, ref in enumerate(walk(n, rows[n])[1][0]):
                assert rel_l2(got[n, h], ref) <= TOL_F32, (n, h, rows[n])
        else:
            assert torch.equal(after[n], before[n]), n


def many_documents():
    r = np.random.default_rng(0)
    lens = r.integers(0, 95, size=1100)
    lens[[3, 500, 501, 1099]] = 300, 128, 129, 0
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    T, H, Hk, dk, dv = int(lens.sum()), 2, 1, 64, 64
    assert T > 32 * len(lens)     # (below, a walk takes them)
    x = dict(q=unit(n(1, T, Hk, dk)).bfloat16(), k=unit(n(1, T, Hk, dk)).bfloat16(),
             v=n(1, T, H, dv).bfloat16(), log_g=-torch.nn.functional.softplus(n(1, T, H) - 2),
             h0=0.05 * n(len(lens), H, dk, dv))
    return {a: b.to(DEV) for a, b in x.items()}, np.cumsum([0] + lens.tolist())


def test_more_documents_than_a_block_reads():
    x, cu = many_documents()
    o, hT = kda.linear_fwd(**x, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert kda.get_device_error() == 0
    ro, rh = linear_attention(*(host(x[a]) for a in ("q", "k", "v", "log_g", "h0")), cu)
    assert rel_l2(host(o), ro) <= TOL_BF16 and rel_l2(host(hT), rh) <= TOL_F32
    for n in (0, 3, 500, 501, 1098, 1099):
        assert rel_l2(host(hT[n]), rh[n]) <= TOL_F32


def test_more_documents_with_malformed_offsets():
    x, cu = many_documents()
    T = int(cu[-1])
    for at, value in ((0, 1), (1100, T - 1), (700, int(cu[701]) + 1), (700, -4), (700, T + 9),
                      (1100, T + 1)):
        bad = cu.copy()
        bad[at] = value
        kda.linear_fwd(**x, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device=DEV))
        assert kda.get_device_error() == 5, (at, value)
    assert kda.get_device_error() == 0
