"""Linear attention with a decay for each head on the GPU, against the float64 oracle.

Tolerances (relative L2). fp32 outputs (hT, S, and o of fp32 inputs): 1e-5; their terms are fp32
products whose roundings (2^-24 each) stay below 1e-6 together. bf16 o: 5e-3; it is rounded once
(at most 2^-8 of a value, 1.7e-3 root mean square), and the tensor-core kernel rounds the decayed
scores and the state that a chunk reads, each as much again, on disjoint parts of the sum.
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_144_b200 as kda
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


def make(B, T, H, Hk, dk, dv, dtype="bf16", gate="token", N=None, mu=-2.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    lead = (B, T, H) if gate == "token" else (H,)
    x = dict(q=unit(n(B, T, Hk, dk)).to(DT[dtype]), k=unit(n(B, T, Hk, dk)).to(DT[dtype]),
             v=n(B, T, H, dv).to(DT[dtype]),
             log_g=-torch.nn.functional.softplus(n(*lead) + mu),
             h0=0.05 * n(B if N is None else N, H, dk, dv))
    return {a: b.to(DEV) for a, b in x.items()}


def cu_of(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV)


def check(x, o, hT, cu=None, h0=True):
    ro, rh = linear_attention(host(x["q"]), host(x["k"]), host(x["v"]), host(x["log_g"]),
                              host(x["h0"]) if h0 else None,
                              None if cu is None else cu.cpu().numpy())
    assert kda.get_device_error() == 0
    assert o.dtype == x["q"].dtype and hT.dtype == torch.float32
    assert rel_l2(host(o), ro) <= (TOL_BF16 if o.dtype == torch.bfloat16 else TOL_F32)
    assert rel_l2(host(hT), rh) <= TOL_F32


SHAPES = [  # B, T, H, Hk, dk, dv
    (1, 1, 1, 1, 128, 128), (2, 1, 3, 1, 128, 64), (1, 63, 2, 2, 128, 128),
    (2, 127, 2, 1, 128, 128), (1, 128, 4, 2, 128, 64), (2, 129, 2, 2, 128, 128),
    (1, 257, 6, 3, 64, 64), (2, 300, 2, 2, 64, 128), (1, 1100, 2, 1, 128, 128),
    (1, 333, 1, 1, 32, 32), (1, 200, 3, 3, 96, 40), (1, 150, 2, 1, 128, 192),
    (1, 140, 1, 1, 128, 256), (1, 70, 2, 2, 256, 256), (1, 70, 2, 1, 20, 7), (1, 33, 1, 1, 1, 1),
    (1, 2500, 1, 1, 8, 8), (3, 640, 1, 1, 128, 24),
]


@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_prefill(shape, dtype, gate):
    x = make(*shape, dtype=dtype, gate=gate, seed=sum(shape))
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"])
    check(x, o, hT)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0, 0, 130, 1, 128, 0], [700, 3, 0, 400, 129],
                                  [64] * 7, [2, 1200]], ids=str)
def test_packed(lens, dtype):
    x = make(1, sum(lens), 4, 2, 128, 64, dtype=dtype, N=len(lens), seed=len(lens))
    cu = cu_of(lens)
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], cu_seqlens=cu)
    check(x, o, hT, cu)
    o2, h2 = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], cu_seqlens=cu,
                            output_final_state=False)
    assert h2 is None
    assert rel_l2(host(o2), linear_attention(
        host(x["q"]), host(x["k"]), host(x["v"]), host(x["log_g"]), None,
        cu.cpu().numpy())[0]) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    x = make(2, 0, 2, 1, 128, 64, dtype=dtype)
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"])
    assert o.numel() == 0 and torch.equal(hT, x["h0"])
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"])
    assert not hT.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["reset", "steep", "none"])
def test_gates(mode, dtype):
    """Gates that clear the state (-inf, and far below what a float's exponential holds) in
    the middle of a chunk, and gates of one."""
    x = make(1, 400, 2, 2, 128, 64, dtype=dtype, seed=5)
    g = x["log_g"]
    if mode == "reset":
        g[:, 37] = -float("inf")
        g[:, 200:203, 0] = -float("inf")
    elif mode == "steep":
        g[:, 10:60] = -300.0
        g[:, 140, 1] = -3.0e38
    else:
        g.zero_()
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], g, h0=x["h0"])
    check(x, o, hT)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_documents_do_not_leak(dtype, bad):
    """Infinities and NaN of one document stay out of its neighbours in the same chunk."""
    lens = [70, 90, 130]
    x = make(1, sum(lens), 2, 1, 128, 64, dtype=dtype, N=3, seed=9)
    cu = cu_of(lens)
    ref, href = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], cu_seqlens=cu)
    for t in ("q", "k", "v"):
        x[t][:, 70:160] = bad
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], cu_seqlens=cu)
    for a, b in ((0, 70), (160, 290)):
        assert torch.equal(o[:, a:b], ref[:, a:b])
    assert torch.equal(hT[0], href[0]) and torch.equal(hT[2], href[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,spots", [   # (token, column); column None: the whole row
    (300, [(200, 3)]), (300, [(128, None), (290, None)]), (300, [(255, None)]), (100, [(99, 0)]),
    (700, [(600, 1), (300, 2), (690, 71), (0, 5)]), (9000, [(5003, 7), (8999, None)]),
    (9000, [(1000, None)]),
], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_bad_values_reach_no_earlier_token(T, spots, bad, dtype):
    """An infinity or NaN in v spoils its column from its token on, and nothing else."""
    x = make(1, T, 2, 1, 128, 72, dtype, seed=7)
    ro, _ = linear_attention(*(host(x[n]) for n in ("q", "k", "v", "log_g", "h0")))
    first = np.full(72, T)
    for t, c in spots:
        cols = slice(None) if c is None else c
        x["v"][0, t, 1, cols] = bad
        first[cols] = np.minimum(first[cols], t)
    o, hT = kda.linear_fwd(**x)
    assert kda.get_device_error() == 0
    o, hT = host(o), host(hT)
    clean = np.ones_like(o, dtype=bool)
    clean[0, :, 1] = np.arange(T)[:, None] < first
    assert rel_l2(o[clean], ro[clean]) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    for c in np.nonzero(first < T)[0]:   # the rows that are computed again, by themselves
        rows = slice(first[c] // 128 * 128, first[c])
        if rows.stop - rows.start > 8:
            assert rel_l2(o[0, rows, 1, c], ro[0, rows, 1, c]) <= (
                TOL_BF16 if dtype == "bf16" else TOL_F32)
    assert not np.isfinite(o[~clean]).any()
    assert np.isfinite(hT[0, 0]).all()
    assert (np.isfinite(hT[0, 1]).all(0) == (first == T)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,t", [(300, 200), (300, 128), (700, 130), (9000, 5003)])
@pytest.mark.parametrize("name", ["q", "k", "log_g"])
def test_bad_rows_reach_no_earlier_token(name, T, t, dtype):
    """A NaN in a row of q spoils that row's output, in k or a gate those from its token on."""
    x = make(1, T, 2, 2, 128, 64, dtype, seed=8)
    ro, _ = linear_attention(*(host(x[n]) for n in ("q", "k", "v", "log_g", "h0")))
    x[name][(0, t, 1) + ((5,) if name != "log_g" else ())] = float("nan")
    o, _ = kda.linear_fwd(**x)
    assert kda.get_device_error() == 0
    o = host(o)
    clean = np.ones_like(o, dtype=bool)
    clean[0, t:t + 1 if name == "q" else T, 1] = False
    assert rel_l2(o[clean], ro[clean]) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    assert not np.isfinite(o[~clean]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,H,Hk,dk,dv", [(1, 1, 1, 1, 128, 128), (5, 1, 4, 2, 128, 64),
                                            (3, 4, 2, 2, 128, 128), (2, 9, 3, 1, 64, 128),
                                            (2, 1, 2, 2, 32, 96), (1, 3, 1, 1, 256, 256),
                                            (3, 2, 2, 1, 20, 7), (300, 1, 2, 2, 128, 128),
                                            (2, 1, 2, 2, 64, 64), (1, 70, 2, 1, 128, 128)])
def test_decode(N, T, H, Hk, dk, dv, dtype):
    for gate in ("token", "head"):
        x = make(N, T, H, Hk, dk, dv, dtype=dtype, gate=gate, seed=N + T)
        S = x["h0"].clone()
        o = kda.linear_decode(x["q"], x["k"], x["v"], x["log_g"], S)
        check(x, o, S)
        if T == 1:   # the single-token form of the arguments
            S1 = x["h0"].clone()
            g = x["log_g"] if gate == "head" else x["log_g"][:, 0]
            o1 = kda.linear_decode(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], g, S1)
            assert o1.shape == (N, H, dv) and torch.equal(o1, o[:, 0]) and torch.equal(S1, S)


def test_prefill_then_decode_is_one_prefill():
    x = make(2, 140, 4, 2, 128, 128, seed=3)
    q, k, v, g = (x[a] for a in ("q", "k", "v", "log_g"))
    cut = lambda a, b: [t[:, a:b].contiguous() for t in (q, k, v, g)]  # noqa: E731
    o, S = kda.linear_fwd(*cut(0, 130), h0=x["h0"])
    parts = [o] + [kda.linear_decode(*cut(t, t + 5), S) for t in (130, 135)]
    check(x, torch.cat(parts, 1), S)


def test_other_stream_and_capture():
    """On a side stream, and captured into a graph whose replay sees new inputs in place."""
    x = make(1, 700, 2, 2, 128, 128, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], stream=side)
    side.synchronize()
    check(x, o, hT)
    S = x["h0"].clone()
    one = [x[a][:, :1].contiguous() for a in ("q", "k", "v", "log_g")]
    graph = torch.cuda.CUDAGraph()
    kda.linear_decode(*one, S.clone())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        oc, hc = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"])
        od = kda.linear_decode(*one, S)
    y = make(1, 700, 2, 2, 128, 128, seed=2)
    for a in x:
        x[a].copy_(y[a])
    S.copy_(x["h0"])
    for t, a in zip(one, ("q", "k", "v", "log_g")):
        t.copy_(x[a][:, :1])
    graph.replay()
    torch.cuda.synchronize()
    check(x, oc, hc)
    x1 = {a: t[:, :1] for a, t in x.items() if a != "h0"} | {"h0": x["h0"]}
    check(x1, od, S)


def test_bad_offsets_are_reported():
    x = make(1, 600, 2, 2, 128, 64, N=3)
    for cu in ([0, 200, 100, 600], [0, 200, 400, 599], [1, 200, 400, 600], [0, 900, 400, 600],
               [0, -5, 400, 600]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], cu_seqlens=c)
        assert kda.get_device_error() == 5, cu
    assert kda.get_device_error() == 0


def test_refusals():
    x = make(2, 8, 4, 2, 64, 32)
    q, k, v, g, h0 = (x[a] for a in ("q", "k", "v", "log_g", "h0"))
    with pytest.raises(ValueError):
        kda.linear_fwd(q[0], k, v, g)
    with pytest.raises(ValueError):
        kda.linear_fwd(q.transpose(1, 2), k, v, g)
    with pytest.raises(TypeError):
        kda.linear_fwd(q.half(), k.half(), v.half(), g)
    with pytest.raises(TypeError):
        kda.linear_fwd(q, k.float(), v, g)
    with pytest.raises(TypeError):
        kda.linear_fwd(q, k, v, g.double())
    with pytest.raises(ValueError):
        kda.linear_fwd(q, k, v, g[:, :, :2].contiguous())
    with pytest.raises(ValueError):
        kda.linear_fwd(q, k, v, g, h0=h0[:1])
    with pytest.raises(ValueError):
        kda.linear_fwd(q.cpu(), k, v, g)
    cu = cu_of([4, 4])
    with pytest.raises(kda.KdaError):
        kda.linear_fwd(q, k, v, g, cu_seqlens=cu)          # B = 2
    with pytest.raises(kda.KdaError):
        kda.linear_fwd(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous())   # 3 % 2 heads
    with pytest.raises(kda.KdaError):
        kda.linear_fwd(q, k, v, g, h0=h0, hT=h0)
    flat = make(1, 8, 1, 1, 64, 64)
    with pytest.raises(kda.KdaError):
        kda.linear_fwd(flat["q"], flat["k"], flat["v"], flat["log_g"], o=flat["v"])
    big = make(1, 2, 1, 1, 264, 8)
    with pytest.raises(kda.KdaError):
        kda.linear_fwd(big["q"], big["k"], big["v"], big["log_g"])
    with pytest.raises(ValueError):
        kda.linear_decode(q, k, v, g, h0[:1])
    with pytest.raises(ValueError):
        kda.linear_decode(q[:, 0], k[:, 0], v, g, h0)
    assert kda.get_device_error() == 0


@pytest.mark.parametrize("T", [1, 127, 128, 129, 1000, 9000])
def test_long_prompt_single_head(T):
    """Few chains: segments, and their states chained."""
    x = make(1, T, 1, 1, 128, 64, seed=T, mu=-4.0)
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"])
    check(x, o, hT)


@pytest.mark.parametrize("lens", [[3000, 1, 0, 500], [100] * 40, [1] * 1100, [2000, 0, 3, 2500, 700],
                                  [0, 0, 5000], [1632, 1633, 0, 1025, 1, 1024, 2048, 2049, 3265],
                                  [1633] * 5 + [700] * 600], ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_packed_few_heads(lens):
    """Documents longer than an SM's share are cut into segments; very many are taken in order."""
    x = make(1, sum(lens), 1, 1, 32, 64, N=len(lens), seed=len(lens))
    cu = cu_of(lens)
    o, hT = kda.linear_fwd(x["q"], x["k"], x["v"], x["log_g"], h0=x["h0"], cu_seqlens=cu)
    check(x, o, hT, cu)


def test_expired_wait_reports_timeout_and_context_survives():
    """Failure injection: with KDA_DEBUG_STALL_WAIT set, the loader of every chunked CTA waits
    (bounded by a 2M-cycle budget) on a barrier that nothing signals, and every other role runs
    into its own bound. The kernel must report KDA_ERR_TIMEOUT, free TMEM and return; the context
    must stay usable. Runs in a child process: the hooks are read once per process."""
    code = (
        "import torch, gated_delta_rule_144_b200 as kda\n"
        "mk = lambda dt: [torch.randn(1, 600, 2, 128, device='cuda').to(dt) for _ in range(3)]\n"
        "g = -torch.rand(1, 600, 2, device='cuda')\n"
        "kda.linear_fwd(*mk(torch.bfloat16), g)\n"
        "st = kda.get_device_error()\n"
        "kda.linear_fwd(*mk(torch.float32), g)\n"
        "torch.cuda.synchronize()\n"
        "print('STATUS', st, int(kda.get_device_error()))\n")
    env = dict(os.environ, KDA_DEBUG_WAIT_CYCLES="2000000", KDA_DEBUG_STALL_WAIT="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("STATUS")][-1]
    assert line.split()[1:] == ["4", "0"]
