"""Timed cases of the operators that serve a recurrent state.

Five operators work on one kind of data, an fp32 state S [dk, dv] per (sequence, head):

  linear_fwd     linear attention with a scalar decay for each head over whole prompts or packed
                 documents: S <- exp(log_g) S + k v^T, o = S^T q
  linear_decode  the same recurrence for one or a few tokens of many sequences, state in place
  decode_tree    the read-outs of the gated delta rule for every node of a tree of drafted tokens,
                 against a state that stays as it is
  commit_path    the state advanced in place along the accepted path of such a tree
  state_copy     pages of a pool of states copied, forked, compacted and cleared in place

``run`` computes a case in plain torch operations, or, with ``own`` set, by the package's calls.
``exact`` steps the definitions token by token in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Lengths of the package's packed workload (8 documents, 28,937 tokens).
PACKED8 = "6393,3101,965,4774,3267,1950,7056,1431"


def listed():
    return [
        # a short chat prompt on a small model's layer: latency counts
        dict(name="linear-prompt-77", op="linear_fwd", B=1, T=77, H=16, Hk=16, dk=128, dv=128,
             dtype="bf16", gate="token", lens="", h0=False),
        # one ordinary prompt
        dict(name="linear-prompt-4096", op="linear_fwd", B=1, T=4096, H=16, Hk=16, dk=128, dv=128,
             dtype="bf16", gate="token", lens="", h0=False),
        # packed documents, heads of width 64 whose queries and keys are shared by four
        dict(name="linear-packed-8docs", op="linear_fwd", B=1, T=28937, H=32, Hk=8, dk=128, dv=64,
             dtype="bf16", gate="token", lens=PACKED8, h0=True),
        # long context from a carried state, one fixed decay for each head
        dict(name="linear-long-65536", op="linear_fwd", B=2, T=65536, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16", gate="head", lens="", h0=True),
        # one step of a small batch in 32 bits: latency counts
        dict(name="linear-decode-n3", op="linear_decode", N=3, T=1, H=16, Hk=16, dk=128, dv=128,
             dtype="f32", gate="token"),
        # one step of a full serving batch
        dict(name="linear-decode-n256", op="linear_decode", N=256, T=1, H=32, Hk=32, dk=128,
             dv=128, dtype="bf16", gate="token"),
        # one sequence with a wide tree of drafts
        dict(name="tree-n1-t61", op="decode_tree", N=1, T=61, H=32, dtype="bf16"),
        # a batch with ordinary trees
        dict(name="tree-n128-t16", op="decode_tree", N=128, T=16, H=32, dtype="bf16"),
        # the accepted rows of a small batch, in 32 bits
        dict(name="commit-n5-a3", op="commit_path", N=5, T=9, A=3, H=16, dtype="f32"),
        # the accepted rows of a full batch
        dict(name="commit-n256-a6", op="commit_path", N=256, T=16, A=6, H=32, dtype="bf16"),
        # one prompt's state forked to the seven samples drawn from it, in every layer's pool
        dict(name="fork-1-to-7", op="state_copy", layers=4, pages=48, H=16, dk=128, dv=128,
             how="fork", moved=7),
        # a third of a full pool's sequences have ended: the holes are filled from the tail, and
        # the tail's own holes are cleared
        dict(name="compact-256", op="state_copy", layers=2, pages=256, H=32, dk=128, dv=128,
             how="compact", moved=85),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_decode", "decode_tree", "commit_path",
                     "state_copy"])
    H = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
    Hk = rng.choice([h for h in (1, 2, 3, 4, 8, 16, 32) if H % h == 0])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    gate = rng.choice(["token", "token", "head"])
    if op == "linear_fwd":
        dk, dv = rng.choice([(128, 128), (128, 128), (128, 64), (64, 64), (64, 128)])
        most = 32768 if dtype == "bf16" else 4096
        if rng.random() < 0.5:
            lens = [_log_int(rng, 1, most // 8) for _ in range(rng.randint(1, 8))]
            return dict(op=op, B=1, T=sum(lens), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, gate=gate,
                        lens=",".join(map(str, lens)), h0=rng.random() < 0.5)
        B = rng.randint(1, 4)
        return dict(op=op, B=B, T=_log_int(rng, 1, most // B), H=H, Hk=Hk, dk=dk, dv=dv,
                    dtype=dtype, gate=gate, lens="", h0=rng.random() < 0.5)
    if op == "linear_decode":
        dk, dv = rng.choice([(128, 128), (128, 128), (128, 64), (64, 64), (64, 128)])
        return dict(op=op, N=_log_int(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 4, 7]), H=H, Hk=Hk,
                    dk=dk, dv=dv, dtype=dtype, gate=gate)
    if op == "decode_tree":
        N = _log_int(rng, 1, 128)
        return dict(op=op, N=N, T=_log_int(rng, 1, 64 if N <= 16 else 24), H=H, dtype=dtype)
    if op == "commit_path":
        T = _log_int(rng, 1, 64)
        return dict(op=op, N=_log_int(rng, 1, 256), T=T, A=rng.randint(1, min(T, 8)), H=H,
                    dtype=dtype)
    how = rng.choice(["fork", "compact"])
    pages = _log_int(rng, 3, 256)
    return dict(op=op, layers=rng.randint(1, 3), pages=pages, H=H,
                dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), how=how,
                moved=rng.randint(1, pages // 2 if how == "compact" else pages - 1))


# ---------------------------------------------------------------- inputs

def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else None


def _normal(g, *shape, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV)
    return x if std == 1.0 else x.mul_(std)


def _unit(g, dt, *shape):
    x = _normal(g, *shape)
    return x.div_(torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp_min(1e-30)).to(dt)


def _decay(g, mean, *shape):
    return torch.nn.functional.softplus(_normal(g, *shape).add_(mean)).neg_()


def _head_decay(H):
    h = torch.arange(1, H + 1, device=DEV, dtype=torch.float64) / H
    return torch.log1p(-torch.exp2(-1 - 7 * h)).float()


def _trees(rng, N, T):
    """parents [N, T]: -1 for a child of the committed state, -2 for the absent nodes behind a
    smaller tree; most nodes hang on a recent one."""
    p = np.full((N, T), -2, dtype=np.int32)
    for n in range(N):
        m = T if rng.random() < 0.5 else int(rng.integers(1, T + 1))
        back = rng.integers(1, 5, size=T)
        p[n, :m] = np.maximum(np.arange(m) - back[:m], -1)
    return p


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, s = case["op"], {"case": case}
    if op == "state_copy":
        L, P, m = case["layers"], case["pages"], case["moved"]
        s["S"] = _normal(g, L, P, case["H"], case["dk"], case["dv"], std=0.02)
        perm = rng.permutation(P)
        if case["how"] == "fork":
            src, dst = np.full(m, perm[0]), perm[1:m + 1]
        else:
            live = np.ones(P, dtype=bool)
            live[perm[:m]] = False
            n = P - m                                  # the first n pages are full afterwards
            holes, tail = np.flatnonzero(~live[:n]), n + np.flatnonzero(live[n:])
            src = np.concatenate([tail, np.full(m, -1)])
            dst = np.concatenate([holes, np.arange(n, P)])
            # a page that is read by the call is not written by it
            keep = (src >= 0) | ~np.isin(dst, tail)
            src, dst = src[keep], dst[keep]
        s["src"] = torch.tensor(src.astype(np.int32), device=DEV)
        s["dst"] = torch.tensor(dst.astype(np.int32), device=DEV)
        return s
    dt, H = DTYPES[case["dtype"]], case["H"]
    if op == "linear_fwd":
        B, T, Hk, dk, dv = (case[x] for x in ("B", "T", "Hk", "dk", "dv"))
        s["q"], s["k"] = _unit(g, dt, B, T, Hk, dk), _unit(g, dt, B, T, Hk, dk)
        s["v"] = _normal(g, B, T, H, dv).to(dt)
        s["log_g"] = _decay(g, -2.0, B, T, H) if case["gate"] == "token" else _head_decay(H)
        lens = _lens(case)
        N = len(lens) if lens else B
        s["h0"] = _normal(g, N, H, dk, dv, std=0.02) if case["h0"] else None
        s["cu"] = torch.tensor(np.cumsum([0] + lens).astype(np.int32), device=DEV) if lens else None
        return s
    N, T = case["N"], case["T"]
    if op == "linear_decode":
        Hk, dk, dv = case["Hk"], case["dk"], case["dv"]
        s["q"], s["k"] = _unit(g, dt, N, T, Hk, dk), _unit(g, dt, N, T, Hk, dk)
        s["v"] = _normal(g, N, T, H, dv).to(dt)
        s["log_g"] = _decay(g, -2.0, N, T, H) if case["gate"] == "token" else _head_decay(H)
        s["S"] = _normal(g, N, H, dk, dv, std=0.02)
        return s
    d = 128
    s["q"], s["k"] = _unit(g, dt, N, T, H, d), _unit(g, dt, N, T, H, d)
    s["v"] = _normal(g, N, T, H, d).to(dt)
    s["log_g"] = _decay(g, 0.0, N, T, H, d)
    s["beta"] = torch.sigmoid(_normal(g, N, T, H)).to(dt)
    s["S"] = _normal(g, N, H, d, d, std=0.02)
    parents = _trees(rng, N, T)
    if op == "decode_tree":
        s["parents"] = torch.tensor(parents, device=DEV)
        s["o"] = torch.zeros(N, T, H, d, dtype=dt, device=DEV)   # rows of absent nodes stay
        return s
    path = np.full((N, case["A"]), -1, dtype=np.int32)
    for n in range(N):                                 # a path from the root towards some node
        i, up = int(rng.integers(0, max(1, (parents[n] >= -1).sum()))), []
        while i >= 0:
            up.append(i)
            i = int(parents[n, i])
        up = up[::-1][:case["A"]]
        path[n, :len(up)] = up
    s["path"] = torch.tensor(path, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

CHUNK = 128


def _chunked(q, k, v, log_g, h0):
    """q, k [N, L, H, dk], v [N, L, H, dv], log_g [N, L, H], h0 [N, H, dk, dv], fp32, padded with
    zeros to whole chunks: (o [N, L, H, dv], S after the last row)."""
    N, L, H, dk = q.shape
    dv, C = v.shape[3], CHUNK
    n = L // C
    q, k, v = (x.view(N, n, C, H, -1).permute(0, 3, 1, 2, 4) for x in (q, k, v))   # [N,H,n,C,d]
    G = log_g.double().view(N, n, C, H).permute(0, 3, 1, 2).cumsum(-1)              # [N,H,n,C]
    below = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = (G[..., :, None] - G[..., None, :]).masked_fill_(~below, -math.inf).exp_().float()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)).mul_(D), v)
    del D
    end = G[..., -1]                                                                # [N,H,n]
    kv = torch.matmul((k * (end[..., None] - G).exp().float()[..., None]).transpose(-1, -2), v)
    # states at the chunk borders 0 .. n: row 0 of the sum is h0
    E = torch.nn.functional.pad(end.cumsum(-1), (1, 0))                             # [N,H,n+1]
    reach = torch.ones(n + 1, n + 1, dtype=torch.bool, device=q.device).tril()
    W = (E[..., :, None] - E[..., None, :]).masked_fill_(~reach, -math.inf).exp_().float()
    kv = torch.cat([h0.view(N, H, 1, dk * dv), kv.view(N, H, n, dk * dv)], 2)
    S = torch.matmul(W, kv)
    del kv
    o += torch.matmul(q, S[:, :, :n].reshape(N, H, n, dk, dv)) * G.exp().float()[..., None]
    return (o.permute(0, 2, 3, 1, 4).reshape(N, L, H, dv),
            S[:, :, n].reshape(N, H, dk, dv).contiguous())


def _rows(lens, B, T, device):
    """Rows [N, L] of the flat token axis that each sequence takes, padded to whole chunks, and
    which of them are its own."""
    starts = [b * T for b in range(B)] if lens is None else np.cumsum([0] + lens)[:-1].tolist()
    lens = [T] * B if lens is None else lens
    L = max(1, -(-max(lens) // CHUNK)) * CHUNK
    at = torch.arange(L, device=device)
    ln = torch.tensor(lens, device=device)
    st = torch.tensor(starts, device=device)
    real = at[None, :] < ln[:, None]
    return torch.where(real, st[:, None] + at[None, :], 0), real


def _prefill(q, k, v, log_g, h0, lens):
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    idx, real = _rows(lens, B, T, q.device)
    N = idx.shape[0]

    def take(x):
        y = x.reshape(B * T, *x.shape[2:]).float()[idx]
        return y * real.view(*real.shape, *[1] * (y.dim() - 2))

    q, k = take(q), take(k)
    if Hk != H:
        q, k = q.repeat_interleave(H // Hk, 2), k.repeat_interleave(H // Hk, 2)
    g = take(log_g.expand(B, T, H) if log_g.dim() == 1 else log_g)
    h0 = torch.zeros(N, H, dk, dv, device=q.device) if h0 is None else h0
    o, hT = _chunked(q, k, take(v), g, h0)
    flat = torch.empty(B * T, H, dv, device=q.device)
    flat[idx[real]] = o[real]
    return flat.view(B, T, H, dv), hT


def _ancestors(parents):
    """anc [N, T, T]: 1 where j is i or an ancestor of i."""
    N, T = parents.shape
    up = (parents[:, :, None] == torch.arange(T, device=parents.device)).double()
    eye = torch.eye(T, device=parents.device, dtype=torch.float64)
    return (torch.matrix_power(eye + up, T) > 0).float()


def _delta(q, k, v, log_g, beta, S, anc):
    """The gated delta rule over nodes with ancestors anc [N, T, T]: read-outs of every node (q
    None: none), the rows u that each node writes, and each node's cumulative log decay G. All
    [N, H, T, .], fp32."""
    T = k.shape[2]
    eye = torch.eye(T, device=k.device)
    G = torch.matmul(anc[:, None].double(), log_g.double())
    D = (G[:, :, :, None] - G[:, :, None]).masked_fill_(anc[:, None, :, :, None] == 0, -math.inf)
    D = D.exp_().float()                                               # [N, H, i, j, dk]
    eG = G.exp().float()
    A = torch.einsum("nhic,nhijc,nhjc->nhij", k, D, k) * (1 - eye)
    r = beta[..., None] * (v - torch.matmul(k * eG, S))
    u = torch.linalg.solve_triangular(eye + beta[..., None] * A, r, upper=False, unitriangular=True)
    if q is None:
        return None, u, G
    Q = torch.einsum("nhic,nhijc,nhjc->nhij", q, D, k)
    return torch.matmul(q * eG, S) + torch.matmul(Q, u), u, G


def _by_head(x):
    return x.float().transpose(1, 2)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear_fwd":
        o, hT = _prefill(s["q"], s["k"], s["v"], s["log_g"], s["h0"], _lens(c))
        return {"o": o.to(s["q"].dtype), "hT": hT}
    if op == "linear_decode":
        if c["T"] == 1:
            r = c["H"] // c["Hk"]
            q, k = (x[:, 0].float().repeat_interleave(r, 1) for x in (s["q"], s["k"]))
            e = s["log_g"].reshape(-1, c["H"]).exp()[..., None, None]
            s["S"].mul_(e).add_(k[..., None] * s["v"][:, 0].float()[..., None, :])
            o = torch.matmul(q[..., None, :], s["S"]).transpose(1, 2)
        else:
            o, S = _prefill(s["q"], s["k"], s["v"], s["log_g"], s["S"], None)
            s["S"].copy_(S)
        return {"o": o.to(s["q"].dtype), "S": s["S"]}
    if op == "decode_tree":
        o, _, _ = _delta(_by_head(s["q"]), _by_head(s["k"]), _by_head(s["v"]),
                         _by_head(s["log_g"]), _by_head(s["beta"]), s["S"],
                         _ancestors(s["parents"]))
        there = (s["parents"] >= -1)[:, :, None, None]
        s["o"].copy_(torch.where(there, o.transpose(1, 2).to(s["o"].dtype), s["o"]))
        return {"o": s["o"]}
    if op == "commit_path":
        N, A = s["path"].shape
        there = (s["path"] >= 0)
        row = s["path"].clamp(min=0).long()
        at = torch.arange(N, device=row.device)[:, None]

        def take(x):
            y = x[at, row].float()
            return (y * there.view(N, A, *[1] * (y.dim() - 2))).transpose(1, 2)

        k = take(s["k"])
        chain = torch.ones(A, A, device=row.device).tril().expand(N, A, A)
        _, u, G = _delta(None, k, take(s["v"]), take(s["log_g"]), take(s["beta"]), s["S"], chain)
        end = G[:, :, -1:]
        ke = k * (end - G).exp().float()
        s["S"].mul_(end.exp().float().transpose(-1, -2)).add_(torch.matmul(ke.transpose(-1, -2), u))
        return {"S": s["S"]}
    src = s["src"].long()
    got = s["S"][:, src.clamp(min=0)]
    s["S"][:, s["dst"].long()] = got * (src >= 0).view(1, -1, 1, 1, 1)
    return {"S": s["S"]}


def run(state):
    if not own:
        return _run_plain(state)
    import gated_delta_rule_144_b200 as kda
    s, op = state, state["case"]["op"]
    if op == "linear_fwd":
        o, hT = kda.linear_fwd(s["q"], s["k"], s["v"], s["log_g"], h0=s["h0"], cu_seqlens=s["cu"])
        return {"o": o, "hT": hT}
    if op == "linear_decode":
        o = kda.linear_decode(s["q"], s["k"], s["v"], s["log_g"], s["S"])
        return {"o": o, "S": s["S"]}
    if op == "decode_tree":
        return {"o": kda.decode_tree(s["q"], s["k"], s["v"], s["log_g"], s["beta"], s["parents"],
                                     s["S"], o=s["o"])}
    if op == "commit_path":
        kda.commit_path(s["k"], s["v"], s["log_g"], s["beta"], s["path"], s["S"])
        return {"S": s["S"]}
    kda.state_copy(s["S"], s["src"], s["dst"], page_dim=1)
    return {"S": s["S"]}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "state_copy":
        page = case["H"] * case["dk"] * case["dv"] * 4
        m = case["moved"]
        if case["how"] == "fork":   # one page read, m written
            return {"bytes": (1 + m) * case["layers"] * page, "flops": 0}
        n, P = case["pages"] - m, case["pages"]
        moves = m * n / P           # expected holes among the first n pages
        return {"bytes": (2 * moves + (m - moves)) * case["layers"] * page, "flops": 0}
    e, H = (2 if case["dtype"] == "bf16" else 4), case["H"]
    if op in ("linear_fwd", "linear_decode"):
        rows = case["T"] * case["B" if op == "linear_fwd" else "N"]
        Hk, dk, dv = case["Hk"], case["dk"], case["dv"]
        io = rows * (2 * Hk * dk + 2 * H * dv) * e
        io += 4 * H * (rows if case["gate"] == "token" else 1)
        if op == "linear_decode":
            states, N = 2, case["N"]
        else:
            N = len(_lens(case) or [0] * case["B"])
            states = 2 if case["h0"] else 1
        return {"bytes": io + states * N * H * dk * dv * 4, "flops": 4 * rows * H * dk * dv}
    d, N, T = 128, case["N"], case["T"]
    state = N * H * d * d * 4
    if op == "decode_tree":
        row = H * (4 * d * e + 4 * d + e)
        # two products of every node with the state; the products among nodes follow the tree
        return {"bytes": state + N * T * (row + 4), "flops": 4 * N * T * H * d * d}
    A = case["A"]
    row = H * (2 * d * e + 4 * d + e)
    return {"bytes": 2 * state + N * A * (row + 4), "flops": 6 * N * A * H * d * d}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda t: t.double()  # noqa: E731
    if op == "state_copy":
        S = f(s["S"])
        old = S.clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            S[:, b] = old[:, a] if a >= 0 else 0
        return {"S": S}
    if op in ("linear_fwd", "linear_decode"):
        q, k, v = f(s["q"]), f(s["k"]), f(s["v"])
        B, T, Hk, dk = q.shape
        H, dv = v.shape[2], v.shape[3]
        gate = f(s["log_g"]).exp()
        lens = _lens(case) if op == "linear_fwd" else None
        spans = ([(0, sum(lens[:i]), n) for i, n in enumerate(lens)] if lens
                 else [(slice(None), 0, T)])
        if sum(n for _, _, n in spans) > 70000:
            return None
        h0 = s["h0"] if op == "linear_fwd" else s["S"]
        o, ends = torch.zeros(B, T, H, dv, dtype=torch.float64, device=DEV), []
        for i, (b, t0, n) in enumerate(spans):
            if lens:
                S = (torch.zeros(1, H, dk, dv, dtype=torch.float64, device=DEV) if h0 is None
                     else f(h0[i:i + 1]))
            else:
                S = (torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV) if h0 is None
                     else f(h0))
            for t in range(t0, t0 + n):
                a = gate if gate.dim() == 1 else gate[:, t]
                qt, kt = (x[:, t].repeat_interleave(H // Hk, 1) for x in (q, k))
                S = a[..., None, None] * S
                S.addcmul_(kt[..., None], v[:, t, :, None, :])
                o[:, t] = torch.matmul(qt[..., None, :], S)[..., 0, :]
            ends.append(S)
        return {"o": o, "hT" if op == "linear_fwd" else "S": torch.cat(ends)}
    k, v, g, beta, S0 = f(s["k"]), f(s["v"]), f(s["log_g"]).exp(), f(s["beta"]), f(s["S"])

    def step(S, n, i):
        S = g[n, i][..., None] * S
        u = beta[n, i][..., None] * (v[n, i] - torch.matmul(k[n, i][..., None, :], S)[..., 0, :])
        return S + k[n, i][..., None] * u[..., None, :]

    N = case["N"]
    if op == "commit_path":
        path = s["path"].tolist()
        out = []
        for n in range(N):
            S = S0[n]
            for i in path[n]:
                S = step(S, n, i) if i >= 0 else S
            out.append(S)
        return {"S": torch.stack(out)}
    q = f(s["q"])
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for n, row in enumerate(s["parents"].tolist()):
        after = {-1: S0[n]}
        for i, p in enumerate(row):
            if p >= -1:
                after[i] = step(after[p], n, i)
                o[n, i] = torch.matmul(q[n, i][..., None, :], after[i])[..., 0, :]
    return {"o": o}
