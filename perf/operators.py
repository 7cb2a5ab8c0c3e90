"""Cases of the head-gated delta rule and its state cache: chunked forward, backward, decode on cache pages, page moves.

One value head, with a dk x dv state S, reads per token q, k (of its key head), v, a log-decay g <= 0 and a strength beta:

    S' = e^g S;   u = beta (v - S'^T k);   S = S' + k u^T;   o = S^T q

Hv value heads share Hk key heads (value head h uses key head h // (Hv / Hk)).  Sequences are packed back to back; each
starts from a state of its own, which may be a page of a cache.  The gates follow g = -exp(A) softplus(x + b) with
A ~ U(0, ln 8) and b ~ U(-6, 0) per head, so heads that forget within a few tokens stand beside heads that remember
thousands; q and k are unit rows of SiLU outputs, v is a SiLU output, beta a sigmoid.
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt at low batch: latency of the launches and of one chunk
        dict(name="forward one chunk", op="forward", dtype="bf16", lens="61", Hk=4, Hv=8, dk=128, dv=128, paged=False),
        # a serving step that prefills prompts of mixed lengths into pages of the state cache
        dict(name="forward packed prompts", op="forward", dtype="bf16", lens="1777,64,1,3001,512,129,900,1808", Hk=16,
             Hv=32, dk=128, dv=128, paged=True),
        # a full batch at this repository's prefill size
        dict(name="forward full batch", op="forward", dtype="bf16", lens="8192,8192,8192,8192", Hk=96, Hv=96, dk=128,
             dv=128, paged=False),
        # fp32 activations at the small head size
        dict(name="forward fp32 d64", op="forward", dtype="f32", lens="500,1,777", Hk=4, Hv=12, dk=64, dv=64, paged=False),
        # one long document of a training batch
        dict(name="backward long", op="backward", dtype="bf16", lens="4096,4096", Hk=16, Hv=32, dk=128, dv=128,
             states=False),
        # packed documents of a training batch, states carried over from the window before
        dict(name="backward packed", op="backward", dtype="bf16", lens="700,33,1,1290", Hk=4, Hv=8, dk=128, dv=128,
             states=True),
        # fp32 activations at the small head size
        dict(name="backward fp32 d64", op="backward", dtype="f32", lens="300,129", Hk=2, Hv=4, dk=64, dv=64, states=True),
        # one user's next token
        dict(name="decode one", op="decode", dtype="bf16", N=1, T=1, Hk=16, Hv=32, dk=128, dv=128, pages=4, idle=0),
        # a full serving batch, some rows of it idle
        dict(name="decode batch", op="decode", dtype="bf16", N=256, T=1, Hk=16, Hv=32, dk=128, dv=128, pages=300, idle=6),
        # a few drafted tokens per sequence in one call
        dict(name="decode drafts", op="decode", dtype="bf16", N=37, T=5, Hk=8, Hv=32, dk=128, dv=128, pages=64, idle=0),
        # samples of several prompts start from their prompts' states, and end
        dict(name="pages fork", op="fork", L=4, pages=200, page_floats=524288, live=24, n=64),
        # a cache is packed to its low pages after sequences have ended
        dict(name="pages compact", op="compact", L=3, pages=301, page_floats=262144, live=160, ended=47),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, most):
    lens = []
    while total > 0 and len(lens) < most:
        n = min(total, _log_int(rng, 1, max(1, total)))
        lens.append(n)
        total -= n
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "decode", "decode", "fork", "compact"])
    if op in ("forward", "backward"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hk * rng.choice([1, 2, 3, 4])
        if dtype == "bf16":
            dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64)])
        else:
            dk, dv = rng.choice([(64, 64), (128, 128)])
        most = (24000 if op == "forward" else 8000) if dtype == "bf16" else 2000
        total = _log_int(rng, 2, max(2, min(most, most * 32 // Hv)))
        case = dict(op=op, dtype=dtype, lens=_lens(rng, total, 12), Hk=Hk, Hv=Hv, dk=dk, dv=dv)
        if op == "forward":
            case["paged"] = rng.random() < 0.5
        else:
            case["states"] = rng.random() < 0.5
        return case
    if op == "decode":
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hv = Hk * rng.choice([1, 2, 3, 4])
        d = rng.choice([128, 128, 64])
        N = _log_int(rng, 1, 256)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), N=N, T=rng.choice([1, 1, 1, 2, 3, 6]), Hk=Hk, Hv=Hv,
                    dk=d, dv=d, pages=N + rng.randrange(0, 40), idle=rng.randrange(0, N) // 8)
    L, floats = rng.choice([1, 2, 5]), 4 * _log_int(rng, 256, 65536)
    pages = _log_int(rng, 8, 400)
    live = rng.randrange(1, pages)
    if op == "fork":
        return dict(op=op, L=L, pages=pages, page_floats=floats, live=live, n=rng.randrange(1, pages - live + 1))
    return dict(op=op, L=L, pages=pages, page_floats=floats, live=live, ended=rng.randrange(0, live))


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _unit_silu(gen, *shape):
    x = torch.nn.functional.silu(_randn(gen, *shape))
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)


def _gate(gen, shape, H):
    A = torch.rand(H, generator=gen, device="cuda") * math.log(8.0)
    b = torch.rand(H, generator=gen, device="cuda") * -6.0
    return -torch.exp(A) * torch.nn.functional.softplus(_randn(gen, *shape, H) + b)


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    if op in ("forward", "backward"):
        io = DTYPES[case["dtype"]]
        lens = [int(x) for x in case["lens"].split(",")]
        N, T, Hk, Hv, dk, dv = len(lens), sum(lens), case["Hk"], case["Hv"], case["dk"], case["dv"]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s = dict(case=case, lens=lens, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 q=_unit_silu(gen, T, Hk, dk).to(io), k=_unit_silu(gen, T, Hk, dk).to(io),
                 v=torch.nn.functional.silu(_randn(gen, T, Hv, dv)).to(io), g=_gate(gen, (T,), Hv).to(io),
                 beta=torch.sigmoid(_randn(gen, T, Hv)).to(io))
        if op == "forward":
            if case["paged"]:  # sequences n < N - 1 go on from their pages, the last one is new; more pages than sequences
                P = N + 3
                perm = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32)
                s["pages"] = 0.3 * _randn(gen, P, Hv, dk, dv)
                s["start"], s["end"] = perm.clone(), perm
                s["start"][N - 1] = -1
            else:
                s["final"] = torch.empty(N, Hv, dk, dv, device="cuda")
        else:
            s["d_out"] = _randn(gen, T, Hv, dv).to(io)
            s["s0"] = 0.3 * _randn(gen, N, Hv, dk, dv) if case["states"] else None
            s["d_final"] = 0.3 * _randn(gen, N, Hv, dk, dv) if case["states"] else None
        return s
    if op == "decode":
        io = DTYPES[case["dtype"]]
        N, T, Hk, Hv, dk, dv, P = (case[n] for n in ("N", "T", "Hk", "Hv", "dk", "dv", "pages"))
        index = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32)
        if case["idle"]:
            index[torch.randperm(N, generator=gen, device="cuda")[: case["idle"]]] = -1
        return dict(case=case, index=index, pages=0.3 * _randn(gen, P, Hv, dk, dv), q=_unit_silu(gen, N, T, Hk, dk).to(io),
                    k=_unit_silu(gen, N, T, Hk, dk).to(io), v=torch.nn.functional.silu(_randn(gen, N, T, Hv, dv)).to(io),
                    g=_gate(gen, (N, T), Hv).to(io), beta=torch.sigmoid(_randn(gen, N, T, Hv)).to(io),
                    out=torch.zeros(N, T, Hv, dv, dtype=io, device="cuda"))
    L, P, E = case["L"], case["pages"], case["page_floats"]
    s = dict(case=case, cache=_randn(gen, L, P, E), refs=torch.zeros(P, dtype=torch.int32, device="cuda"))
    live = torch.randperm(P, generator=gen, device="cuda")[: case["live"]].to(torch.int32)
    s["refs"][live.long()] = 1
    if op == "fork":  # a quarter of the new sequences start from nothing, the others from a live page, some from the same one
        pick = torch.randint(0, case["live"], (case["n"],), generator=gen, device="cuda")
        s["parents"] = live[torch.minimum(pick, torch.full_like(pick, 7))].contiguous()
        s["parents"][torch.rand(case["n"], generator=gen, device="cuda") < 0.25] = -1
    else:
        s["table"] = live
        s["ended"] = live[: case["ended"]].contiguous()
        s["keep"] = torch.arange(case["live"], device="cuda") >= case["ended"]
    return s


def work(case):
    op = case["op"]
    if op in ("forward", "backward"):
        e = 2 if case["dtype"] == "bf16" else 4
        lens = [int(x) for x in case["lens"].split(",")]
        N, T, Hk, Hv, dk, dv = len(lens), sum(lens), case["Hk"], case["Hv"], case["dk"], case["dv"]
        state = 4 * N * Hv * dk * dv
        flops = T * Hv * (6 * dk * dv + CHUNK * (2 * dk + 2 * dv))
        if op == "forward":
            return {"bytes": e * T * (2 * Hk * dk + 2 * Hv * dv + 2 * Hv) + state * (2 if case["paged"] else 1), "flops": flops}
        return {"bytes": e * T * (4 * Hk * dk + 3 * Hv * dv + 4 * Hv) + state * (3 if case["states"] else 0), "flops": 2.5 * flops}
    if op == "decode":
        e = 2 if case["dtype"] == "bf16" else 4
        n, T, Hk, Hv, dk, dv = case["N"] - case["idle"], case["T"], case["Hk"], case["Hv"], case["dk"], case["dv"]
        return {"bytes": 8 * n * Hv * dk * dv + e * n * T * (2 * Hk * dk + 2 * Hv * dv + 2 * Hv), "flops": 6 * n * T * Hv * dk * dv}
    page = 4 * case["L"] * case["page_floats"]
    if op == "fork":
        return {"bytes": page * (case["n"] + min(case["live"], 8, case["n"])), "flops": 0}
    m = case["live"] - case["ended"]  # live pages above m move: about this many of them
    return {"bytes": 2 * page * max(1, m * (case["pages"] - m) // case["pages"]), "flops": 0}


# ------------------------------------------------------------------------------------------------ plain forms
def _padded(x, lens, rep=1):
    """[T, H, ...] of packed sequences as fp32 [N, H * rep, chunks, CHUNK, ...], zeros behind each sequence's end."""
    nc = max(1, -(-max(lens) // CHUNK))
    at = torch.arange(nc * CHUNK, device=x.device)
    n = torch.tensor(lens, device=x.device)
    first = torch.cumsum(n, 0) - n
    rows = torch.where(at < n[:, None], first[:, None] + at, 0)
    y = x.float()[rows] * (at < n[:, None]).view(len(lens), -1, *[1] * (x.dim() - 1))
    y = y.movedim(2, 1).repeat_interleave(rep, 1)
    return y.reshape(len(lens), y.shape[1], nc, CHUNK, *y.shape[3:])


def _packed(y, lens):
    """The inverse of _padded: [N, H, chunks, CHUNK, ...] to [T, H, ...]."""
    y = y.flatten(2, 3).movedim(1, 2)
    keep = torch.arange(y.shape[1], device=y.device) < torch.tensor(lens, device=y.device)[:, None]
    return y[keep]


def _chunk_parts(s):
    lens, rep = s["lens"], s["case"]["Hv"] // s["case"]["Hk"]
    q, k = _padded(s["q"], lens, rep), _padded(s["k"], lens, rep)
    v, g, beta = _padded(s["v"], lens), _padded(s["g"], lens), _padded(s["beta"], lens)
    G = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    kk = D * (k @ k.transpose(-1, -2))
    P = D * (q @ k.transpose(-1, -2))
    A = (beta[..., :, None] * kk).tril(-1)
    M = torch.eye(CHUNK, device=q.device).expand_as(A).contiguous()
    for i in range(1, CHUNK):  # forward substitution, a row of every chunk at a time
        M[..., i, :i] = -(A[..., i, None, :i] @ M[..., :i, :i])[..., 0, :]
    return dict(q=q, k=k, v=v, beta=beta[..., None], gamma=torch.exp(G).float()[..., None],
                lam=torch.exp(G[..., -1:] - G).float()[..., None], D=D, kk=kk.tril(-1), P=P, M=M)


def _forward_chunks(p, S, keep=False):
    """Outputs, the last state, and (keep) each chunk's start state and U."""
    outs, states, us = [], [], []
    for c in range(p["q"].shape[2]):
        x = {n: t[:, :, c] for n, t in p.items()}
        if keep:
            states.append(S)
        U = x["M"] @ (x["beta"] * (x["v"] - x["gamma"] * (x["k"] @ S)))
        us.append(U)
        if not keep:
            outs.append(x["gamma"] * (x["q"] @ S) + x["P"] @ U)
        S = x["gamma"][..., -1:, :] * S + x["k"].transpose(-1, -2) @ (x["lam"] * U)
    return outs, S, states, us


def _plain_forward(s):
    c, io = s["case"], DTYPES[s["case"]["dtype"]]
    if c["paged"]:
        S = torch.where((s["start"] >= 0)[:, None, None, None], s["pages"][s["start"].clamp_min(0).long()], 0.0)
    else:
        S = torch.zeros(len(s["lens"]), c["Hv"], c["dk"], c["dv"], device="cuda")
    outs, S, _, _ = _forward_chunks(_chunk_parts(s), S)
    out = _packed(torch.stack(outs, 2), s["lens"]).to(io)
    if c["paged"]:
        s["pages"][s["end"].long()] = S
        return out, s["pages"]
    s["final"].copy_(S)
    return out, s["final"]


def _plain_backward(s):
    c, io, lens = s["case"], DTYPES[s["case"]["dtype"]], s["lens"]
    p = _chunk_parts(s)
    zero = torch.zeros(len(lens), c["Hv"], c["dk"], c["dv"], device="cuda")
    _, S, states, us = _forward_chunks(p, zero if s["s0"] is None else s["s0"], keep=True)
    dO, dS = _padded(s["d_out"], lens), zero if s["d_final"] is None else s["d_final"]
    T = lambda t: t.transpose(-1, -2)  # noqa: E731
    got = []
    end = S
    for i in reversed(range(len(us))):
        x, do, S, U = {n: t[:, :, i] for n, t in p.items()}, dO[:, :, i], states[i], us[i]
        kd = x["k"] @ dS
        H = T(x["M"]) @ (T(x["P"]) @ do + x["lam"] * kd)
        W = x["beta"] * H
        dP, dA = (do @ T(U)).tril(), -(W @ T(U)).tril(-1)
        oS, wS, ud = x["gamma"] * (do @ T(S)), x["gamma"] * (W @ T(S)), x["lam"] * (U @ T(dS))
        dPD, dAD = dP * x["D"], dA * x["D"]
        dq = oS + dPD @ x["k"]
        dk = ud - wS + T(dPD) @ x["q"] + dAD @ x["k"] + T(dAD) @ x["k"]
        dbeta = (H * (x["v"] - x["gamma"] * (x["k"] @ S))).sum(-1) - ((H @ T(U)) * x["kk"]).sum(-1)
        E = dP * x["P"] + dA * x["kk"]
        dG = (x["q"] * oS - x["k"] * wS - x["k"] * ud).sum(-1) + E.sum(-1) - E.sum(-2)
        dg = dG.flip(-1).cumsum(-1).flip(-1) + (dS * end).sum((-1, -2))[..., None]
        got.append((dq, dk, W, dg, dbeta))
        end = S
        dS = x["gamma"][..., -1:, :] * dS + T(x["q"]) @ (x["gamma"] * do) - T(x["k"]) @ (x["gamma"] * W)
    dq, dk, dv, dg, dbeta = (_packed(torch.stack(t[::-1], 2), lens) for t in zip(*got))
    group = lambda t: t.unflatten(1, (c["Hk"], -1)).sum(2)  # noqa: E731
    r = dict(dq=group(dq).to(io), dk=group(dk).to(io), dv=dv.to(io), dg=dg.to(io), dbeta=dbeta.to(io))
    if c["states"]:
        r["d_initial_state"] = dS
    return r


def _plain_decode(s):
    c = s["case"]
    rep = c["Hv"] // c["Hk"]
    rows = (s["index"] >= 0).nonzero()[:, 0]
    page = s["index"][rows].long()
    S = s["pages"][page]
    q, k = (s[n][rows].float().repeat_interleave(rep, 2) for n in ("q", "k"))
    v, g, beta = (s[n][rows].float() for n in ("v", "g", "beta"))
    for t in range(c["T"]):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ S)[..., 0, :])
        S = S + k[:, t, :, :, None] * u[:, :, None]
        s["out"][rows, t] = (q[:, t, :, None] @ S)[..., 0, :].to(s["out"].dtype)
    s["pages"][page] = S
    return s["out"], s["pages"]


def _plain_fork(s):
    refs = s["refs"].clone()
    children = (refs == 0).nonzero()[: len(s["parents"]), 0].to(torch.int32)
    refs[children.long()] = 1
    got = s["cache"][:, s["parents"].clamp_min(0).long()]
    s["cache"][:, children.long()] = torch.where((s["parents"] >= 0)[None, :, None], got, 0.0)
    live = refs.clone()
    refs[children.long()] -= 1  # the samples end
    return children, live, refs, s["cache"]


def _plain_compact(s):
    refs, table = s["refs"].clone(), s["table"].clone()
    refs[s["ended"].long()] -= 1
    table = torch.where(s["keep"], table, -1)
    m = (refs > 0).sum()
    at = torch.arange(len(refs), device=refs.device)
    src, dst = ((refs > 0) & (at >= m)).nonzero()[:, 0], ((refs == 0) & (at < m)).nonzero()[:, 0]
    s["cache"][:, dst] = s["cache"][:, src]
    to = at.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table)
    refs[dst], refs[src] = refs[src], 0
    return table, refs, m.to(torch.int32).reshape(1), s["cache"]


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from gated_delta_rule_155_b200 import kda
        if op == "forward":
            if s["case"]["paged"]:
                return kda.kda_gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["pages"],
                                           final_state=s["pages"], initial_index=s["start"], final_index=s["end"])
            return kda.kda_gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], final_state=s["final"])
        if op == "backward":
            d0 = None if s["s0"] is None else torch.empty_like(s["s0"])
            r = kda.kda_gdr_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["d_out"], s["cu"], s["s0"], s["d_final"],
                                     d_initial_state=d0)
            return {n: t for n, t in r.items() if t is not None}
        if op == "decode":
            return kda.kda_gdr_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pages"], s["index"], s["out"]), s["pages"]
        refs = s["refs"].clone()
        if op == "fork":
            children = kda.kda_pages_fork(s["cache"], refs, s["parents"])
            live = refs.clone()
            kda.kda_pages_free(refs, children)
            return children, live, refs, s["cache"]
        table = torch.where(s["keep"], s["table"], -1)
        kda.kda_pages_free(refs, s["ended"])
        live = kda.kda_pages_compact(s["cache"], refs, table)
        return table, refs, live, s["cache"]
    return {"forward": _plain_forward, "backward": _plain_backward, "decode": _plain_decode, "fork": _plain_fork,
            "compact": _plain_compact}[op](s)


# ------------------------------------------------------------------------------------------------ 64 bits, token by token
def _steps(s, x, n):
    """Input `n` in 64 bits as [T, N, Hv, ...], padded with zeros behind each sequence's end."""
    c = s["case"]
    x = x.double().repeat_interleave(c["Hv"] // x.shape[1], 1)
    y = torch.zeros(max(s["lens"]), len(s["lens"]), *x.shape[1:], dtype=torch.float64, device=x.device)
    at = 0
    for i, m in enumerate(s["lens"]):
        y[:m, i] = x[at:at + m]
        at += m
    return y


def _back(s, y):
    return torch.cat([y[:m, i] for i, m in enumerate(s["lens"])])


def _token(S, k, v, a, b):
    Sd = a[..., None, None] * S
    r = v - torch.einsum("nhkv,nhk->nhv", Sd, k)
    return Sd, r, Sd + k[..., :, None] * (b[..., None] * r)[..., None, :]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("forward", "backward"):
        if max(s["lens"]) * len(s["lens"]) * case["Hv"] > 12_000_000 or max(s["lens"]) > 30_000:
            return None
        q, k, v, g, b = (_steps(s, s[n], n) for n in ("q", "k", "v", "g", "beta"))
        a = torch.exp(g)
        N, Hv, dk, dv = len(s["lens"]), case["Hv"], case["dk"], case["dv"]
        zero = torch.zeros(N, Hv, dk, dv, dtype=torch.float64, device="cuda")
        if op == "forward":
            S = zero
            if case["paged"]:
                S = torch.stack([s["pages"][i].double() if i >= 0 else zero[0] for i in s["start"].tolist()])
            out = torch.empty_like(v)
            for t in range(len(q)):  # behind a sequence's end g = 0 and beta = 0: its state stays
                _, _, S = _token(S, k[t], v[t], a[t], b[t])
                out[t] = torch.einsum("nhkv,nhk->nhv", S, q[t])
            if case["paged"]:
                pages = s["pages"].double()
                pages[s["end"].long()] = S
                return _back(s, out), pages
            return _back(s, out), S
        do = _steps(s, s["d_out"], "d_out")
        S = zero if s["s0"] is None else s["s0"].double()
        seg, starts = 64, []
        for t in range(len(q)):
            if t % seg == 0:
                starts.append(S)
            S = _token(S, k[t], v[t], a[t], b[t])[2]
        dS = zero if s["d_final"] is None else s["d_final"].double()
        dq, dk_, dv_, dg, db = (torch.empty_like(x) for x in (q, k, v, g, b))
        for c in reversed(range(len(starts))):
            ts, S, kept = range(c * seg, min(len(q), (c + 1) * seg)), starts[c], []
            for t in ts:
                Sd, r, S = _token(S, k[t], v[t], a[t], b[t])
                kept.append((Sd, r, S))
            for t in reversed(ts):
                Sd, r, S = kept[t - c * seg]
                dq[t] = torch.einsum("nhkv,nhv->nhk", S, do[t])
                dS = dS + q[t][..., :, None] * do[t][..., None, :]
                du = torch.einsum("nhkv,nhk->nhv", dS, k[t])
                db[t] = (du * r).sum(-1)
                dv_[t] = b[t][..., None] * du
                dk_[t] = torch.einsum("nhkv,nhv->nhk", dS, b[t][..., None] * r) - torch.einsum("nhkv,nhv->nhk", Sd, dv_[t])
                dS = dS - k[t][..., :, None] * dv_[t][..., None, :]
                dg[t] = (dS * Sd).sum((-1, -2))
                dS = a[t][..., None, None] * dS
        head = lambda y: _back(s, y).unflatten(1, (case["Hk"], -1)).sum(2)  # noqa: E731
        r = dict(dq=head(dq), dk=head(dk_), dv=_back(s, dv_), dg=_back(s, dg), dbeta=_back(s, db))
        if case["states"]:
            r["d_initial_state"] = dS
        return r
    if op == "decode":
        rep = case["Hv"] // case["Hk"]
        out, pages = s["out"].double(), s["pages"].double()
        for i, page in enumerate(s["index"].tolist()):
            if page < 0:
                continue
            S = pages[page][None]
            for t in range(case["T"]):
                k, q = (s[n][i, t].double().repeat_interleave(rep, 0)[None] for n in ("k", "q"))
                _, _, S = _token(S, k, s["v"][i, t].double()[None], torch.exp(s["g"][i, t].double())[None],
                                 s["beta"][i, t].double()[None])
                out[i, t] = torch.einsum("nhkv,nhk->nhv", S, q)[0]
            pages[page] = S[0]
        return out, pages
    refs, cache = s["refs"].tolist(), s["cache"].double()
    if op == "fork":
        free = [p for p, n in enumerate(refs) if n == 0]
        for i, parent in enumerate(s["parents"].tolist()):
            cache[:, free[i]] = s["cache"][:, parent].double() if parent >= 0 else 0.0
        return None, None, None, cache
    for p in s["ended"].tolist():
        refs[p] -= 1
    m = sum(n > 0 for n in refs)
    holes = [p for p in range(m) if refs[p] == 0]
    for src, dst in zip([p for p in range(m, len(refs)) if refs[p] > 0], holes):
        cache[:, dst] = cache[:, src]
    return None, None, None, cache
