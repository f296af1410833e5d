"""Trees of drafted tokens and the commit of their accepted path, against the float64 oracle run
along every node's own path.

Tolerances (relative L2): fp32 outputs 1e-5 (split products lose 2^-21 per factor, sums are fp32);
bf16 outputs 5e-3 (one rounding, at most 2^-8 of a value, and tf32 factors, 2^-11 each).
"""

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
import oracle
from kda_testutil import TOL_BF16, TOL_F32, host, rel_l2, require_cuda

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_cuda()
    yield
    torch.cuda.synchronize()


def make(N, T, H, dtype="bf16", seed=0, mu=0.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(n(N, T, H, 128)).to(DT[dtype]), k=unit(n(N, T, H, 128)).to(DT[dtype]),
             v=n(N, T, H, 128).to(DT[dtype]),
             log_g=-torch.nn.functional.softplus(n(N, T, H, 128) + mu),
             beta=torch.sigmoid(n(N, T, H)).to(DT[dtype]), S=0.05 * n(N, H, 128, 128))
    return {a: b.to(DEV) for a, b in x.items()}


def random_parents(N, T, seed, kind="mixed"):
    r = np.random.default_rng(seed)
    p = np.full((N, T), -2, dtype=np.int32)
    for n in range(N):
        m = T if n % 2 == 0 else int(r.integers(0, T + 1))
        for i in range(m):
            p[n, i] = (i - 1 if kind == "chain" else -1 if kind == "star"
                       else max(-1, i - int(r.integers(1, 6))))
        if kind == "holes" and T > 2:   # absent nodes between present ones
            p[n, 1] = -2
            p[n][p[n] == 1] = -1
    return p


def path_of(row, i):
    up = []
    while i >= 0:
        up.append(i)
        i = int(row[i])
    return up[::-1]


def walk(x, n, rows):
    """Oracle along rows of sequence n: (read-outs, final state)."""
    f = lambda t: host(t[n:n + 1, rows])  # noqa: E731
    return oracle.kda_fwd(f(x["q"]), f(x["k"]), f(x["v"]), f(x["log_g"]), f(x["beta"]),
                          h0=host(x["S"][n:n + 1]))


def check_tree(x, parents, o, before):
    S0 = x["S"].clone()
    got, ref = host(o), np.zeros(tuple(o.shape))
    for n, row in enumerate(parents):
        for i, p in enumerate(row):
            if p == -2:
                assert torch.equal(o[n, i], before[n, i])   # left as it was
                ref[n, i] = got[n, i]
            else:
                ref[n, i] = walk(x, n, path_of(row, i))[0][0, -1]
    assert torch.equal(x["S"], S0)
    assert rel_l2(got, ref) <= (TOL_BF16 if o.dtype == torch.bfloat16 else TOL_F32)
    assert kda.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["mixed", "chain", "star", "holes"])
@pytest.mark.parametrize("N,T,H", [(1, 1, 1), (3, 5, 2), (2, 16, 1), (2, 17, 2), (1, 40, 1),
                                   (1, 64, 2)])
def test_tree(N, T, H, kind, dtype):
    x = make(N, T, H, dtype, seed=T)
    parents = random_parents(N, T, T, kind)
    before = torch.randn(N, T, H, 128, device=DEV).to(DT[dtype])
    o = before.clone()
    r = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"],
                        torch.tensor(parents, device=DEV), x["S"], o=o)
    assert r is o
    check_tree(x, parents, o, before)


@pytest.mark.parametrize("T", [1, 5, 16, 30, 61])
def test_tree_keeps_fp32(T):
    """fp32 rows, 1.3e-6: a tensor-core accumulation cuts a sum off at 2^-23 of its size, half of that
    on average, and running sums are about two thirds of the last one. A pair's coefficient is two
    sums of 24 steps: 24 x 2^-24 x 2/3 = 9.5e-7 of the output. The products with S take 48 steps,
    1.9e-6 of a part that is a tenth of the output here (S is scaled down); v must not pass
    through those sums. The split factors leave 2^-22 of the same terms."""
    x = make(3, T, 2, "f32", seed=77)
    x["S"] *= 0.1
    parents = random_parents(3, T, 78)
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"],
                        torch.tensor(parents, device=DEV), x["S"])
    assert kda.get_device_error() == 0
    there = parents != -2
    ref = np.zeros(tuple(o.shape))
    for n, i in np.argwhere(there):
        ref[n, i] = walk(x, n, path_of(parents[n], i))[0][0, -1]
    assert rel_l2(host(o)[there], ref[there]) <= 1.3e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,H", [(3, 5, 2), (3, 40, 1), (40, 18, 4)])
def test_tree_without_nodes(N, T, H, dtype):
    """Absent nodes and rejected sequences: zeros in a new output, untouched rows in a given one."""
    x = make(N, T, H, dtype, seed=31)
    parents = random_parents(N, T, 32, "holes")
    parents[-1] = 0                                     # rejected: node 0 its own parent
    parents[1, :] = -2
    p = torch.tensor(parents, device=DEV)
    given = torch.full_like(x["q"], 7.0)
    kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"], p, x["S"], o=given)
    assert kda.get_device_error() == 7
    poison = torch.full_like(given, float("nan"))       # what a new output is likely to find there
    torch.cuda.synchronize()
    del poison
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"], p, x["S"])
    assert kda.get_device_error() == 7
    there = p != -2
    there[-1] = False
    assert torch.equal(o[there], given[there])
    assert not o[~there].any() and (given[~there] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_steep_gates(dtype):
    x = make(2, 20, 2, dtype, seed=1)
    x["log_g"][0, 3] = -float("inf")
    x["log_g"][1, :, :, ::3] = -200.0
    x["log_g"][:, 7] = 0.0
    parents = random_parents(2, 20, 3)
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"],
                        torch.tensor(parents, device=DEV), x["S"])
    # the oracle's exp(-inf) is 0, as the kernel's
    check_tree(x, parents, o, torch.zeros_like(o))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_branches_do_not_leak(bad, dtype):
    """Non-finite values of one branch stay in it; those of absent nodes reach nothing."""
    x = make(1, 18, 2, dtype, seed=2)
    parents = np.array([[-1, 0, 0, 1, 2, 3, 4, -1, 7, 2, 9, 8, 5, -1, 13, 14, -2, -2]], np.int32)
    P = torch.tensor(parents, device=DEV)
    args = lambda: (x["q"], x["k"], x["v"], x["log_g"], x["beta"], P, x["S"])  # noqa: E731
    ref = kda.decode_tree(*args())
    for t in ("q", "k", "v", "beta", "log_g"):
        x[t][:, 16:] = bad
    x["v"][:, 2, 0, 5] = bad          # one column of node 2 and what is below it
    x["k"][:, 13] = bad
    o = kda.decode_tree(*args())
    under2 = [i for i in range(16) if 2 in path_of(parents[0], i)]
    under13 = [13, 14, 15]
    for i in range(18):
        if i in under13:
            assert not torch.isfinite(o[0, i]).any()
            continue
        same = torch.ones(2, 128, dtype=torch.bool, device=DEV)
        if i in under2:
            same[0, 5] = False
            assert not torch.isfinite(o[0, i, 0, 5])
        assert torch.equal(o[0, i][same], ref[0, i][same])
    assert kda.get_device_error() == 0


def test_tree_bad_parents():
    x = make(3, 4, 2)
    for bad in ([0, 0, 1, 2], [-1, 1, 0, 0], [-1, 0, 5, 1], [-3, -1, -1, -1], [-2, 0, -1, -1],
                [-1, 2, -1, -1]):
        parents = np.array([[-1, 0, 1, 1], bad, [-1, -1, 0, 2]], np.int32)
        before = torch.full((3, 4, 2, 128), 7.0, device=DEV, dtype=torch.bfloat16)
        o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"],
                            torch.tensor(parents, device=DEV), x["S"], o=before.clone())
        assert kda.get_device_error() == 7, bad
        assert torch.equal(o[1], before[1])
        for n in (0, 2):
            ref = np.stack([walk(x, n, path_of(parents[n], i))[0][0, -1] for i in range(4)])
            assert rel_l2(host(o[n]), ref) <= TOL_BF16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,H,A", [(1, 1, 1, 1), (4, 9, 2, 3), (5, 16, 1, 6), (2, 40, 2, 35),
                                     (3, 6, 3, 17)])
def test_commit(N, T, H, A, dtype):
    x = make(N, T, H, dtype, seed=A)
    r = np.random.default_rng(A)
    path = np.full((N, A), -1, np.int32)
    for n in range(N):
        m = A if n == 0 else int(r.integers(0, A + 1))
        path[n, :m] = r.integers(0, T, size=m)      # any rows, also the same one again
        if m + 1 < A:
            path[n, m + 1] = 0                      # behind the end: not part of the path
    before = x["S"].clone()
    kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], torch.tensor(path, device=DEV), x["S"])
    assert kda.get_device_error() == 0
    after, x["S"] = x["S"], before
    for n in range(N):
        rows = []
        for i in path[n]:
            if i < 0:
                break
            rows.append(int(i))
        if rows:
            assert rel_l2(host(after[n]), walk(x, n, rows)[1][0]) <= TOL_F32
        else:
            assert torch.equal(after[n], before[n])


def test_commit_bad_rows():
    x = make(3, 5, 2)
    path = torch.tensor([[0, 1, -1], [2, 5, 0], [4, -7, 9]], dtype=torch.int32, device=DEV)
    before = x["S"].clone()
    kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], path, x["S"])
    assert kda.get_device_error() == 7
    after, x["S"] = x["S"], before
    assert torch.equal(after[1], before[1])
    assert rel_l2(host(after[0]), walk(x, 0, [0, 1])[1][0]) <= TOL_F32
    assert rel_l2(host(after[2]), walk(x, 2, [4])[1][0]) <= TOL_F32


def test_draft_verify_commit_follows_decode():
    """A tree of drafts whose accepted path is then decoded step by step gives the same read-outs
    and states."""
    N, T, H = 4, 12, 2
    x = make(N, T, H, "f32", seed=8)
    parents = random_parents(N, T, 1)
    parents[:, :] = parents[0]
    P = torch.tensor(parents, device=DEV)
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"], P, x["S"])
    rows = path_of(parents[0], T - 1)
    S = x["S"].clone()
    for i in rows:
        c = [x[a][:, i].contiguous() for a in ("q", "k", "v", "log_g", "beta")]
        step = kda.decode_step(*c, S)
        assert rel_l2(host(o[:, i]), host(step)) <= TOL_F32
    kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"],
                    torch.tensor([rows] * N, dtype=torch.int32, device=DEV), x["S"])
    assert rel_l2(host(x["S"]), host(S)) <= TOL_F32


def test_other_stream_and_capture():
    x = make(3, 10, 2, seed=4)
    parents = random_parents(3, 10, 2)
    P = torch.tensor(parents, device=DEV)
    a = (x["q"], x["k"], x["v"], x["log_g"], x["beta"], P, x["S"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = kda.decode_tree(*a, stream=side)
    side.synchronize()
    check_tree(x, parents, o, torch.zeros_like(o))
    path = torch.tensor([[0, 1], [-1, 0], [0, -1]], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    S = x["S"].clone()
    with torch.cuda.graph(graph):
        kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], path, S)
        oc = kda.decode_tree(*a[:-1], S)
    graph.replay()
    torch.cuda.synchronize()
    S1 = x["S"].clone()
    kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], path, S1)
    assert torch.equal(S, S1) and torch.equal(oc, kda.decode_tree(*a[:-1], S1))


def test_refusals():
    x = make(2, 4, 2)
    P = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    ok = dict(q=x["q"], k=x["k"], v=x["v"], log_g=x["log_g"], beta=x["beta"], parents=P, S=x["S"])
    for change, err in (({"parents": P.long()}, TypeError), ({"parents": P[:, :3]}, ValueError),
                        ({"S": x["S"].half()}, TypeError), ({"S": x["S"][:1]}, ValueError),
                        ({"q": x["q"].float()}, TypeError), ({"beta": x["beta"].float()}, TypeError),
                        ({"k": x["k"][..., :64].contiguous()}, ValueError),
                        ({"v": x["v"].transpose(1, 2)}, ValueError),
                        ({"log_g": x["log_g"].cpu()}, ValueError)):
        with pytest.raises(err):
            kda.decode_tree(**{**ok, **change})
    with pytest.raises(kda.KdaError):
        kda.decode_tree(**ok, o=x["v"])
    y = make(1, 65, 1)
    with pytest.raises(kda.KdaError):
        kda.decode_tree(y["q"], y["k"], y["v"], y["log_g"], y["beta"],
                        torch.full((1, 65), -1, dtype=torch.int32, device=DEV), y["S"])
    with pytest.raises(ValueError):
        kda.commit_path(x["k"], x["v"], x["log_g"], x["beta"], P[:1], x["S"])
    assert kda.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [7, 30, 64])
@pytest.mark.parametrize("gate", [-3.0, -30.0, -90.0])
def test_tree_chains_near_the_range(T, gate, dtype):
    """Paths whose gate products approach and pass what a float's range holds."""
    x = make(1, T, 2, dtype, seed=T)
    x["log_g"][:, ::4] = gate
    parents = random_parents(1, T, 5, "chain")
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_g"], x["beta"],
                        torch.tensor(parents, device=DEV), x["S"])
    check_tree(x, parents, o, torch.zeros_like(o))
