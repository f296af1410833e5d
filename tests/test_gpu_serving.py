"""The serving operators run together, as an engine uses them, against the float64 oracles.

A pool [layers, pages, H, 128, 128] holds the states of a KDA layer (0) and of a linear-attention
layer (1). Prompts fill pages, a page is forked, drafted trees are read and their accepted paths
committed, single tokens follow, a sequence retires and the pool is compacted, and decoding goes on
over the moved pages. Every sequence's outputs and last states must be those of its tokens in order.

Tolerances (relative L2): as for the operators by themselves, 5e-3 for bf16 outputs; 1e-5 for the
linear states and for KDA states that only the per-token kernels touched (the prompt runs per token).
"""

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
from kda_testutil import TOL_BF16, TOL_F32, host, oracle_fwd, rel_l2, require_cuda
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV, H, D = "cuda", 4, 128
LENS = [37, 1, 200]                       # prompts
FORK = ([0, 2, 0], [3, 4, 5])             # page 0 -> 3 and 5, page 2 -> 4
PARENTS = [-1, 0, 0, 1, 1, 2, -1, 6, 7, -2]
PATHS = [[0, 1, 3], [6, 7, 8], [0, 2, 5], [0, 1, 4], [0, 1, 3], [6, 7, 8]]
LIVE = [1, 0, 1, 0, 1, 1, 0, 0]           # after the single tokens: pages 1 and 3 retire


@pytest.fixture(autouse=True)
def _gpu():
    require_cuda()
    yield
    torch.cuda.synchronize()


def rows(lead, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(n(*lead, H, D)), k=unit(n(*lead, H, D)), v=n(*lead, H, D),
             beta=torch.sigmoid(n(*lead, H)))
    x = {a: b.to(torch.bfloat16) for a, b in x.items()}
    x["log_g"] = -torch.nn.functional.softplus(n(*lead, H, D))
    x["gate"] = -torch.nn.functional.softplus(n(*lead, H) - 2)   # the linear layer's, per head
    return {a: b.to(DEV) for a, b in x.items()}


class Engine:
    """Inputs of one run, and its steps. Outputs land in `out`: name -> (KDA, linear)."""

    def __init__(self):
        self.prompt = rows((1, sum(LENS)), 1)
        self.cu = torch.tensor(np.cumsum([0] + LENS), dtype=torch.int32, device=DEV)
        n = len(PATHS)
        self.tree = rows((n, len(PARENTS)), 2)
        self.token, self.after = rows((n,), 3), rows((sum(LIVE),), 4)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        self.parents, self.path = i32([PARENTS] * n), i32([p + [-1] for p in PATHS])
        self.fork = [i32(x) for x in FORK]
        src, dst, self.where = kda.plan_compaction(LIVE)
        self.moves = i32(src + [-1, -1]), i32(dst + [len(LIVE) - 1, -1])   # and clear the last page
        idx = torch.tensor(PATHS, device=DEV)
        self.accepted = {a: torch.stack([b[i, idx[i]] for i in range(n)]).contiguous()
                         for a, b in self.tree.items()}
        self.pool = torch.full((2, len(LIVE), H, D, D), float("nan"), device=DEV)
        self.out = {}

    @staticmethod
    def kda_args(x):
        return [x[a] for a in ("q", "k", "v", "log_g", "beta")]

    @staticmethod
    def lin_args(x):
        return [x[a] for a in ("q", "k", "v", "gate")]

    def prefill(self):
        n = len(LENS)
        a, _ = kda.fwd(*self.kda_args(self.prompt), cu_seqlens=self.cu, hT=self.pool[0, :n],
                       chunk_size=kda.CHUNK_PER_TOKEN)
        b, _ = kda.linear_fwd(*self.lin_args(self.prompt), cu_seqlens=self.cu, hT=self.pool[1, :n])
        self.out["prompt"] = a, b

    def serve(self):
        pool, n, m = self.pool, len(PATHS), sum(LIVE)
        kda.state_copy(pool, *self.fork, page_dim=1)
        a = kda.decode_tree(*self.kda_args(self.tree), self.parents, pool[0, :n])
        kda.commit_path(*self.kda_args(self.tree)[1:], self.path, pool[0, :n])
        b = kda.linear_decode(*self.lin_args(self.accepted), pool[1, :n])
        self.out["tree"] = a, b
        a = kda.decode_step(*self.kda_args(self.token), pool[0, :n])
        b = kda.linear_decode(*self.lin_args(self.token), pool[1, :n])
        self.out["token"] = a, b
        kda.state_copy(pool, *self.moves, page_dim=1)
        a = kda.decode_step(*self.kda_args(self.after), pool[0, :m])
        b = kda.linear_decode(*self.lin_args(self.after), pool[1, :m])
        self.out["after"] = a, b

    def tokens(self, i, path):
        """Sequence i's tokens in order, its path's included: prompt, path, token, after."""
        src = dict(zip(FORK[1], FORK[0])).get(i, i)
        t0 = sum(LENS[:src])
        pieces = {a: [b[0, t0:t0 + LENS[src]], self.tree[a][i, path], self.token[a][i:i + 1]]
                  for a, b in self.prompt.items()}
        if LIVE[i]:
            w = self.where[i]
            for a, b in self.after.items():
                pieces[a].append(b[w:w + 1])
        return {a: torch.cat(b)[None] for a, b in pieces.items()}, LENS[src]


def reference(x):
    return (*oracle_fwd({a: x[a] for a in ("q", "k", "v", "log_g", "beta")}),
            *linear_attention(*(host(x[a]) for a in ("q", "k", "v", "gate"))))


def test_prompt_fork_tree_commit_decode_compact():
    e = Engine()
    e.prefill()
    e.serve()
    assert kda.get_device_error() == 0
    out = {k: [host(t) for t in v] for k, v in e.out.items()}
    for i, path in enumerate(PATHS):
        x, prompt = e.tokens(i, path)
        ko, kS, lo, lS = reference(x)
        end = prompt + len(path)
        if i < len(LENS):
            at = slice(sum(LENS[:i]), sum(LENS[:i + 1]))
            assert rel_l2(out["prompt"][0][0, at], ko[0, :prompt]) <= TOL_BF16
            assert rel_l2(out["prompt"][1][0, at], lo[0, :prompt]) <= TOL_BF16
        assert rel_l2(out["tree"][0][i, path], ko[0, prompt:end]) <= TOL_BF16
        assert rel_l2(out["tree"][1][i], lo[0, prompt:end]) <= TOL_BF16
        assert rel_l2(out["token"][0][i], ko[0, end]) <= TOL_BF16
        assert rel_l2(out["token"][1][i], lo[0, end]) <= TOL_BF16
        if LIVE[i]:
            w = e.where[i]
            assert rel_l2(out["after"][0][w], ko[0, end + 1]) <= TOL_BF16
            assert rel_l2(out["after"][1][w], lo[0, end + 1]) <= TOL_BF16
            assert rel_l2(host(e.pool[0, w]), kS[0]) <= TOL_F32
            assert rel_l2(host(e.pool[1, w]), lS[0]) <= TOL_F32
    assert not e.pool[:, -1].any()   # the cleared page
    rest = out["tree"][0][:, PARENTS.index(-2)]
    assert not rest.any()            # no node: zeros


def test_the_same_steps_captured_and_replayed():
    e = Engine()
    e.prefill()
    e.pool[:, len(LENS):] = 0
    start = e.pool.clone()
    e.serve()
    want = {k: [t.clone() for t in v] for k, v in e.out.items()}, e.pool.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    e.pool.copy_(start)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        e.serve()
    for _ in range(3):
        e.pool.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert kda.get_device_error() == 0
        assert torch.equal(e.pool, want[1])
        for name, pair in e.out.items():
            if name != "prompt":
                assert all(torch.equal(a, b) for a, b in zip(pair, want[0][name])), name


def test_two_engines_at_once():
    """Two runs interleaved on two streams leave what each leaves by itself."""
    alone = Engine()
    alone.prefill()
    alone.serve()
    torch.cuda.synchronize()
    streams, engines = [torch.cuda.Stream() for _ in range(2)], [Engine() for _ in range(2)]
    torch.cuda.synchronize()
    for step in ("prefill", "serve"):
        for s, e in zip(streams, engines):
            with torch.cuda.stream(s):
                getattr(e, step)()
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    m = sum(LIVE)
    for e in engines:
        assert torch.equal(e.pool[:, :m], alone.pool[:, :m])
        for name, pair in e.out.items():
            assert all(torch.equal(a, b) for a, b in zip(pair, alone.out[name])), name
