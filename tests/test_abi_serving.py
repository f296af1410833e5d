"""Host-side checks of the linear-attention, draft-tree and page entry points (no GPU needed:
every call here is refused before a launch, so the fake pointers are never read)."""

import ctypes

import numpy as np
import pytest

import gated_delta_rule_144_b200 as kda
from gated_delta_rule_144_b200 import build as kbuild

FAKE = 0x100000
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def P(x):
    return None if x is None else ctypes.c_void_p(x)


def far(i):
    return FAKE + (i << 32)   # fake buffers that do not overlap


def linear(L, h0=None, cu=None, ptr=None, ws=None, ws_bytes=0, **kw):
    d = dict(B=1, T=64, H=4, Hk=2, dk=128, dv=64, num_seqs=1, dtype=kda.KDA_BF16, gate=0)
    d.update(kw)
    p = dict(q=far(0), k=far(1), v=far(2), g=far(3), o=far(4), hT=far(5))
    p.update(ptr or {})
    return L.kda_linear_fwd(ctypes.byref(kda.LinearDesc(**d)), P(p["q"]), P(p["k"]), P(p["v"]),
                            P(p["g"]), P(h0), P(cu), P(p["o"]), P(p["hT"]), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=3), INVALID), (dict(Hk=0), INVALID),
    (dict(B=2), INVALID), (dict(dtype=5), INVALID), (dict(gate=2), INVALID),
    (dict(dk=257), UNSUPPORTED), (dict(dv=300), UNSUPPORTED),
    (dict(B=2, num_seqs=2, cu=far(6)), INVALID), (dict(num_seqs=0, cu=far(6)), INVALID),
    (dict(ptr=dict(q=None)), INVALID), (dict(ptr=dict(g=None)), INVALID),
    (dict(ptr=dict(o=far(4) + 2)), INVALID), (dict(h0=far(6) + 4), INVALID),
    (dict(ptr=dict(o=far(2))), INVALID), (dict(ptr=dict(o=far(0) + 64)), INVALID),
    (dict(h0=far(5)), INVALID),
    (dict(ptr=dict(o=far(3))), INVALID), (dict(ptr=dict(hT=far(1) + 128)), INVALID),
    (dict(ptr=dict(hT=far(4) + 16)), INVALID), (dict(h0=far(6), ptr=dict(o=far(6))), INVALID),
    (dict(T=4096, dtype=0, ws=far(2), ws_bytes=1 << 30), INVALID),
    (dict(T=4096, dtype=0, ws=far(5) - 64, ws_bytes=1 << 30), INVALID),
], ids=str)
def test_linear_fwd_refuses(L, kw, code):
    assert linear(L, **kw) == code
    assert L.kda_last_error()


def test_linear_fwd_needs_its_workspace(L):
    d = dict(B=1, T=4096, H=2, Hk=2, num_seqs=1, dtype=kda.KDA_F32)
    need = kda.linear_fwd_workspace_size(1, 4096, 2, 2, 128, 64, 1, dtype=None)
    assert need > 0
    assert linear(L, **d) == INVALID
    assert linear(L, ws=far(8), ws_bytes=need // 2, **d) == INVALID
    assert linear(L, ws=far(8) + 4, ws_bytes=need, **d) == INVALID


def test_workspace_of_a_rejected_description(L):
    assert kda.linear_fwd_workspace_size(1, 4096, 3, 2, 128, 64, 1) == 0
    assert kda.linear_fwd_workspace_size(1, 0, 2, 2, 128, 64, 1) == 0


def test_linear_decode_refuses(L):
    def call(N=2, T=1, H=2, Hk=1, dk=64, dv=64, dtype=1, gate=0, q=far(0), S=far(3), o=far(4)):
        return L.kda_linear_decode(N, T, H, Hk, dk, dv, dtype, gate, P(q), P(far(1)), P(far(2)),
                                   P(far(6)), P(S), P(o), None)
    assert call(N=-1) == INVALID and call(T=-1) == INVALID and call(Hk=4) == INVALID
    assert call(dk=512) == UNSUPPORTED and call(dtype=9) == INVALID and call(gate=-1) == INVALID
    assert call(q=None) == INVALID and call(S=far(3) + 8) == INVALID
    assert call(S=far(0)) == INVALID and call(o=far(1)) == INVALID and call(S=far(4)) == INVALID
    assert call(S=far(6)) == INVALID and call(o=far(6)) == INVALID
    assert call(N=0, q=None, S=None, o=None) == 0 and call(T=0, q=None) == 0


def test_tree_and_path_refuse(L):
    def tree(N=1, H=2, T=4, dtype=1, q=far(0), par=far(6), o=far(5)):
        return L.kda_decode_tree(N, H, T, dtype, P(q), P(far(1)), P(far(2)), P(far(3)), P(far(4)),
                                 P(par), P(far(7)), P(o), 0, None)
    assert tree(N=-1) == INVALID and tree(H=0) == INVALID and tree(dtype=2) == INVALID
    assert tree(T=65) == UNSUPPORTED and tree(q=None) == INVALID and tree(par=far(6) + 4) == INVALID
    assert tree(o=far(0)) == INVALID and tree(o=far(7) + 65536) == INVALID
    assert tree(N=0, q=None) == 0

    def path(N=1, H=2, T=4, A=2, dtype=1, k=far(1), idx=far(6), S=far(7)):
        return L.kda_commit_path(N, H, T, A, dtype, P(k), P(far(2)), P(far(3)), P(far(4)), P(idx),
                                 P(S), None)
    assert path(A=-1) == INVALID and path(k=None) == INVALID and path(S=far(2)) == INVALID
    assert path(S=far(7) + 4) == INVALID and path(A=0, k=None) == 0


def test_state_copy_refuses(L):
    def copy(pool=far(0), layers=1, pages=4, page=64, src=far(1), dst=far(2), n=2):
        return L.kda_state_copy(P(pool), layers, pages, page, P(src), P(dst), n, None)
    assert copy(pages=-1) == INVALID and copy(page=0) == INVALID and copy(n=-1) == INVALID
    assert copy(page=24) == UNSUPPORTED and copy(pool=None) == INVALID and copy(src=None) == INVALID
    assert copy(dst=far(2) + 4) == INVALID and copy(src=far(0) + 64) == INVALID
    assert copy(n=0, src=None, dst=None) == 0 and copy(layers=0, pool=None) == 0


@pytest.mark.parametrize("live", [[], [1], [0], [0, 1], [1, 0, 1, 0, 0, 1, 1], [0] * 3, [1] * 4])
def test_plan_compaction(live):
    src, dst, where = kda.plan_compaction(live)
    pool = list(range(len(live)))
    assert not set(src) & set(dst) and len(set(dst)) == len(dst)
    for a, b in zip(src, dst):
        pool[b] = a
    n = sum(live)
    assert sorted(pool[:n]) == [p for p, x in enumerate(live) if x]
    assert all((w == -1) != bool(x) for w, x in zip(where, live))
    assert all(pool[w] == p for p, w in enumerate(where) if w >= 0)
    rng = np.random.default_rng(len(live))
    big = rng.random(200) < 0.5
    s, d, w = kda.plan_compaction(big)
    assert len(s) == int((~big[:int(big.sum())]).sum())
