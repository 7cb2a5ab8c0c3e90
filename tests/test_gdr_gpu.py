"""The head-gated delta rule and the state cache's pages on the GPU, against the 64-bit reference.

Tolerances (e = the reference, in 64 bits, from the values that the GPU reads):
  * a value stored in bf16 is off by at most half a step, 2^-8 |e|, by that rounding alone.
  * fp32 kernels: sums of at most 128 products, each step at most 2^-24 relative to the sum of its terms'
    absolute values, through three products a chunk: about 3 * 128 * 2^-24 = 2^-15.4 of the largest value
    in the worst case.  Bound: 2^-14 of the largest |e| of the tensor.
  * bf16 at dk = dv = 128: every operand that is not exact in bf16 is a hi + lo pair, off by at most 2^-17
    relative (hi by 2^-8, lo by 2^-9 of that), and the product of the lo parts is left out (2^-16); three
    products a chunk: about 3 * 2^-15 of the largest value at worst.  Bound: 2^-13 of the largest |e| for
    states and, on top of the bf16 rounding, for outputs and dv.  The gradients of q, k, g and beta read
    states and corrections rounded once to bf16: four roundings of 2^-8 relative to their terms, which are
    independent, so their 2-norm is at most 2^-8 of the gradient's beside the output's own; bound 2^-7 of
    the 2-norm, and 2^-4 of the rms on top of 2^-8 |e| for one element (the largest of 10^5 such errors is
    within 5 of their rms of 2^-8 rms sqrt(4), times two for terms that cancel).
"""
import numpy as np
import pytest
import torch

from oracle import gdr

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_155_b200 import build

    build.build()
    from gated_delta_rule_155_b200 import kda as k

    return k


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, Hk, Hv, dk, dv, io, seed, N=1, gate=1.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    silu = torch.nn.functional.silu
    d = dict(q=unit(silu(rn(T, Hk, dk))), k=unit(silu(rn(T, Hk, dk))), v=silu(rn(T, Hv, dv)),
             g=-gate * torch.nn.functional.softplus(rn(T, Hv) - 2.0), beta=torch.sigmoid(rn(T, Hv)))
    d = {n: x.to(DT[io]) for n, x in d.items()}
    d["s0"] = 0.3 * rn(N, Hv, dk, dv)
    d["dS"] = 0.3 * rn(N, Hv, dk, dv)
    d["dO"] = rn(T, Hv, dv).to(DT[io])
    return d


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def to(d, *names):
    return [d[n].cuda() for n in names]


NAMES = ("q", "k", "v", "g", "beta")


def tc(io, dk, dv):
    return io == "bf16" and dk == dv == 128


def near(got, ref, io, exact_path, what, stored=True):
    got, ref = (f64(got) if isinstance(got, torch.Tensor) else got), np.asarray(ref)
    assert np.isfinite(got).all(), what
    if not ref.size:
        return
    bound = (2.0 ** -14 if exact_path else 2.0 ** -13) * max(np.abs(ref).max(), 1e-30)
    if stored and io == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(ref)
    off = np.abs(got - ref)
    assert (off <= bound).all(), f"{what}: off by {off.max():.3g}, {np.max(off / bound):.2f} of the bound"


def near_grad(got, ref, io, exact_path, what):
    if exact_path:
        return near(got, ref, io, True, what)
    got, ref = f64(got), np.asarray(ref)
    assert np.isfinite(got).all(), what
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= 2.0 ** -7 * norm + 1e-30, f"{what}: {np.linalg.norm(got - ref) / norm:.3g} of the norm"
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -4 * np.sqrt(np.mean(ref * ref)) + 1e-30
    assert (np.abs(got - ref) <= bound).all(), f"{what}: {np.max(np.abs(got - ref) / bound):.2f} of the bound"


SHAPES = [  # lens, Hk, Hv, dk, dv
    ([1], 1, 1, 128, 128),
    ([64], 2, 4, 128, 128),
    ([130, 0, 1, 63, 65], 2, 6, 128, 128),
    ([257], 3, 3, 128, 128),
    ([17, 100], 1, 4, 64, 64),
    ([70, 1], 2, 2, 64, 128),
    ([70, 66], 2, 4, 128, 64),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_forward(kda, io, shape, state):
    lens, Hk, Hv, dk, dv = shape
    N, cu = len(lens), cu_of(lens)
    d = make(cu[-1], Hk, Hv, dk, dv, io, 3, N)
    s0 = d["s0"] if state else None
    sT = torch.empty(N, Hv, dk, dv, device="cuda")
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                 None if s0 is None else s0.cuda(), final_state=sT)
    kda.kda_check_device_error()
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), cu, None if s0 is None else f64(s0))
    ex = not tc(io, dk, dv)
    near(out, ro, io, ex, "out")
    near(sT, rs, io, ex, "final state", stored=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_backward(kda, io, shape, state):
    lens, Hk, Hv, dk, dv = shape
    N, cu = len(lens), cu_of(lens)
    d = make(cu[-1], Hk, Hv, dk, dv, io, 4, N)
    s0, dS = (d["s0"], d["dS"]) if state else (None, None)
    d0 = torch.empty(N, Hv, dk, dv, device="cuda")
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    args = (*to(d, *NAMES, "dO"), cug, None if s0 is None else s0.cuda(), None if dS is None else dS.cuda())
    gr = kda.kda_gdr_backward(*args, d_initial_state=d0)
    kda.kda_check_device_error()
    ref = gdr.backward(*(f64(d[n]) for n in NAMES), cu, f64(d["dO"]), None if s0 is None else f64(s0),
                       None if dS is None else f64(dS))
    ex = not tc(io, dk, dv)
    near(gr["d_initial_state"], ref["d_initial_state"], io, ex, "d_initial_state", stored=False)
    near(gr["dv"], ref["dv"], io, ex, "dv")
    for n in ("dq", "dk", "dg", "dbeta"):
        near_grad(gr[n], ref[n], io, ex, n)
    again = kda.kda_gdr_backward(*args, d_initial_state=torch.empty_like(d0))
    for n in gr:
        assert torch.equal(gr[n], again[n]), f"{n} differs between two runs"


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_long_memory(kda, io, dk):
    """Slow decays over many chunks: errors add up, sums of gates reach far."""
    d = make(1500, 1, 2, dk, dk, io, 5, gate=0.02)
    sT = torch.empty(1, 2, dk, dk, device="cuda")
    out, _ = kda.kda_gdr_forward(*(x[None] for x in to(d, *NAMES)), None, d["s0"].cuda(), final_state=sT)
    kda.kda_check_device_error()
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), [0, 1500], f64(d["s0"]))
    near(out[0], ro, io, io == "f32", "out")
    near(sT, rs, io, io == "f32", "final state", stored=False)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("case", ["reset", "frozen", "no write", "same key", "strong"])
def test_edges(kda, io, dk, case):
    T, Hk, Hv = 150, 1, 2
    d = make(T, Hk, Hv, dk, dk, io, 6)
    if case == "reset":
        d["g"][[0, 5, 63, 64, 100]] = -float("inf")
        d["g"][7] = -1e30
    elif case == "frozen":
        d["g"].zero_()
        d["beta"].fill_(1.0)
    elif case == "no write":
        d["beta"][10:90] = 0.0
    elif case == "same key":
        d["k"][:] = d["k"][:1].clone()
        d["beta"].fill_(1.0)
    else:
        d["g"].fill_(-60.0)
    sT = torch.empty(1, Hv, dk, dk, device="cuda")
    x = [t[None] for t in to(d, *NAMES)]
    out, _ = kda.kda_gdr_forward(*x, None, d["s0"].cuda(), final_state=sT)
    gr = kda.kda_gdr_backward(*x, d["dO"].cuda()[None], None, d["s0"].cuda(), d["dS"].cuda(),
                              d_initial_state=torch.empty_like(sT))
    kda.kda_check_device_error()
    a = [f64(d[n]) for n in NAMES]
    ro, rs = gdr.forward(*a, [0, T], f64(d["s0"]))
    ex = io == "f32"
    near(out[0], ro, io, ex, "out")
    near(sT, rs, io, ex, "final state", stored=False)
    ref = gdr.backward(*a, [0, T], f64(d["dO"]), f64(d["s0"]), f64(d["dS"]))
    near(gr["d_initial_state"], ref["d_initial_state"], io, ex, "d_initial_state", stored=False)
    near(gr["dv"][0], ref["dv"], io, ex, "dv")
    for n in ("dq", "dk", "dbeta"):
        near_grad(gr[n][0], ref[n], io, ex, n)
    near_grad(gr["dg"][0], ref["dg"], io, ex, "dg")


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_neighbours_and_rows_behind(kda, io, dk):
    """NaN and infinities of one sequence reach no other; tokens behind the last sequence are left alone."""
    lens, Hk, Hv = [70, 40, 100], 1, 2
    cu = cu_of(lens)
    T = cu[-1] + 30
    d = make(T, Hk, Hv, dk, dk, io, 7, 3)
    clean = {n: f64(d[n]) for n in NAMES + ("dO",)}
    for n in NAMES + ("dO",):
        d[n][70:110] = float("nan")
        d[n][cu[-1]:] = float("inf")
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full((T, Hv, dk), 7.0, dtype=DT[io], device="cuda")
    sT = torch.empty(3, Hv, dk, dk, device="cuda")
    kda.kda_gdr_forward(*to(d, *NAMES), cug, d["s0"].cuda(), out, sT)
    grads = {n: torch.full_like(d[m], 7.0).cuda() for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                                               ("dbeta", "beta"))}
    kda.kda_gdr_backward(*to(d, *NAMES, "dO"), cug, d["s0"].cuda(), d["dS"].cuda(), grads=grads)
    kda.kda_check_device_error()
    ro, rs = gdr.forward(*(clean[n] for n in NAMES), cu, f64(d["s0"]))
    ref = gdr.backward(*(clean[n] for n in NAMES), cu, clean["dO"], f64(d["s0"]), f64(d["dS"]))
    ex = io == "f32"
    for lo, hi in ((0, 70), (110, 210)):
        near(out[lo:hi], ro[lo:hi], io, ex, "out")
        for n in grads:
            near_grad(grads[n][lo:hi], ref[n][lo:hi], io, ex, n)
    near(sT[[0, 2]], rs[[0, 2]], io, ex, "final state", stored=False)
    for t in (out, *grads.values()):
        assert bool((t[cu[-1]:] == 7.0).all())


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_pages_of_states(kda, io, dk):
    """Initial and final states on pages: shared starts, a new sequence, a state that is not kept."""
    lens, Hk, Hv, P = [70, 5, 64, 0, 33], 1, 2, 9
    cu = cu_of(lens)
    d = make(cu[-1], Hk, Hv, dk, dk, io, 8, P)
    start, end = [3, 3, -1, 7, 8], [1, 0, 5, 2, -1]
    pages = d["s0"].cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), i32(cu), pages, final_state=pages, initial_index=i32(start),
                                 final_index=i32(end))
    kda.kda_check_device_error()
    s0 = np.stack([f64(d["s0"])[p] if p >= 0 else np.zeros((Hv, dk, dk)) for p in start])
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), cu, s0)
    want = f64(d["s0"]).copy()
    for n, p in enumerate(end):
        if p >= 0:
            want[p] = rs[n]
    ex = io == "f32"
    near(out, ro, io, ex, "out")
    near(pages, want, io, ex, "pages", stored=False)
    untouched = [3, 4, 6, 7, 8]
    assert torch.equal(pages[untouched].cpu(), d["s0"][untouched])


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_bad_state_pages_are_refused(kda, io, dk):
    lens, Hk, Hv, P = [20, 20, 20, 20], 1, 1, 5
    cu = cu_of(lens)
    d = make(cu[-1], Hk, Hv, dk, dk, io, 9, P)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(start, end):
        pages = d["s0"].cuda()
        kda.kda_gdr_forward(*to(d, *NAMES), i32(cu), pages, final_state=pages, initial_index=i32(start), final_index=i32(end))
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == 7
        kda.kda_check_device_error()      # the word was cleared
        return pages.cpu()

    pages = call([0, 1, 2, 3], [0, 0, 5, -1])      # named twice; out of range
    assert torch.equal(pages[1:], d["s0"][1:]) and not torch.equal(pages[0], d["s0"][0])
    pages = call([0, 1, 2, 3], [1, -1, 4, -1])     # page 1 is where sequence 1 starts
    assert torch.equal(pages[:4], d["s0"][:4]) and not torch.equal(pages[4], d["s0"][4])
    pages = call([9, -1, -1, -1], [0, -1, -1, -1])  # a start out of range counts as zeros
    _, rs = gdr.forward(*(f64(d[n]) for n in NAMES), cu)
    near(pages[0], rs[0], io, io == "f32", "state", stored=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,T,Hk,Hv,dk,dv", [(1, 1, 1, 1, 128, 128), (3, 1, 2, 4, 128, 128), (5, 3, 1, 3, 128, 128),
                                             (4, 1, 2, 2, 64, 64), (2, 4, 1, 2, 64, 128), (2, 2, 1, 2, 128, 64),
                                             (90, 1, 2, 8, 128, 128)])
@pytest.mark.parametrize("paged", [False, True])
def test_decode(kda, io, N, T, Hk, Hv, dk, dv, paged):
    P = N + 3 if paged else N
    d = make(N * T, Hk, Hv, dk, dv, io, 10, P)
    x = {n: d[n].view(N, T, *d[n].shape[1:]) for n in NAMES}
    index = None
    if paged:
        index = torch.randperm(P, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
        if N > 2:
            index[1] = -1
    state = d["s0"].cuda()
    out = torch.full((N, T, Hv, dv), 7.0, dtype=DT[io], device="cuda")
    kda.kda_gdr_decode(*(x[n].cuda() for n in NAMES), state, None if index is None else index.cuda(), out)
    kda.kda_check_device_error()
    ro, rs = gdr.decode(*(f64(x[n]) for n in NAMES), f64(d["s0"]), None if index is None else index.tolist())
    rows = [n for n in range(N) if index is None or index[n] >= 0]
    near(out[rows], ro[rows], io, True, "out")
    near(state, rs, io, True, "state", stored=False)
    if paged:
        rest = [p for p in range(P) if p not in index.tolist()]
        assert torch.equal(state[rest].cpu(), d["s0"][rest])
        assert all(bool((out[n] == 7.0).all()) for n in range(N) if n not in rows)


def test_decode_without_a_token_axis_and_bad_pages(kda):
    N, Hv, dk = 4, 2, 128
    d = make(N, 1, Hv, dk, dk, "bf16", 11, 4)
    state = d["s0"].cuda()
    out = torch.full((N, Hv, dk), 7.0, dtype=torch.bfloat16, device="cuda")
    index = torch.tensor([2, 2, 4, 0], dtype=torch.int32)     # named twice; out of range
    kda.kda_gdr_decode(*to(d, *NAMES), state, index.cuda(), out)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == 7
    ro, rs = gdr.decode(*(f64(d[n])[:, None] for n in NAMES), f64(d["s0"]), index.tolist())
    near(out[[0, 3]], ro[[0, 3], 0], "bf16", True, "out")
    near(state, rs, "bf16", True, "state", stored=False)
    assert bool((out[1:3] == 7.0).all())


@pytest.mark.parametrize("L,P,E,dtype", [(1, 5, 4, torch.float32), (3, 40, 2052, torch.float32), (2, 9, 8192, torch.bfloat16),
                                         (1, 3000, 8, torch.int16)])
@pytest.mark.parametrize("seed", [0, 1])
def test_pages_against_a_plain_model(kda, L, P, E, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    cache = torch.randint(-1000, 1000, (L, P, E), generator=gen).to(dtype)
    refs = (torch.rand(P, generator=gen) < 0.5).to(torch.int32)
    refs[0] = 2
    live = refs.nonzero()[:, 0]
    n = int((refs == 0).sum()) + (2 if seed else 0)       # with seed 1: more than there are free pages
    parents = live[torch.randint(0, len(live), (n,), generator=gen)].to(torch.int32)
    parents[torch.rand(n, generator=gen) < 0.3] = -1
    c, r = cache.cuda(), refs.cuda()
    children = kda.kda_pages_fork(c, r, parents.cuda())
    kda.kda_check_device_error()
    wc, wr, wch = gdr.fork(cache.float().numpy(), refs.numpy(), parents.tolist())
    assert children.cpu().tolist() == wch.tolist() and r.cpu().tolist() == wr.tolist()
    assert np.array_equal(c.cpu().float().numpy(), wc)

    ended = torch.randperm(P, generator=gen)[: P // 2].to(torch.int32)
    ended = torch.cat([ended[torch.from_numpy(wr)[ended.long()] > 0], torch.tensor([-1], dtype=torch.int32)])
    kda.kda_pages_free(r, ended.cuda())
    for p in ended.tolist():
        if p >= 0:
            wr[p] -= 1
    assert r.cpu().tolist() == wr.tolist()

    table = torch.from_numpy(np.flatnonzero(wr > 0).astype(np.int32))
    table = torch.cat([table.flip(0), torch.tensor([-1], dtype=torch.int32)]).cuda()
    before = table.cpu().numpy()
    count = kda.kda_pages_compact(c, r, table)
    kda.kda_check_device_error()
    wc, wr, wt, m = gdr.compact(wc, wr, before)
    assert int(count) == m and r.cpu().tolist() == wr.tolist() and table.cpu().tolist() == wt.tolist()
    assert np.array_equal(c.cpu().float().numpy(), wc)

    k = min(P // 2, 300)
    perm = torch.randperm(P, generator=gen).to(torch.int32)
    src, dst = perm[:k].clone(), perm[k:2 * k].clone()
    if k > 2:
        src[1] = src[0]       # one source twice
        src[2] = -1           # zeros
        dst[0] = -1           # nothing
    kda.kda_pages_copy(c, src.cuda(), dst.cuda())
    kda.kda_check_device_error()
    wc = gdr.copy(wc, src.tolist(), dst.tolist())
    assert np.array_equal(c.cpu().float().numpy(), wc)


def test_bad_pages_are_left_out(kda):
    cache = torch.arange(2 * 6 * 4, dtype=torch.float32).view(2, 6, 4)
    refs = torch.tensor([1, 0, 1, 0, 0, 0], dtype=torch.int32)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def refused():
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == 7

    c, r = cache.cuda(), refs.cuda()
    parents = (2, 3, -2, 6, 0, -1)                        # 3 is free, -2 and 6 are no pages
    children = kda.kda_pages_fork(c, r, i32(*parents))
    refused()
    wc, wr, wch = gdr.fork(cache.numpy(), refs.numpy(), parents)
    assert children.cpu().tolist() == wch.tolist() and r.cpu().tolist() == wr.tolist()
    assert np.array_equal(c.cpu().numpy(), wc)

    for src, dst in (((0, 1), (4, 4)), ((0, 4), (4, 5)), ((0, 1), (1, 0)), ((0, 7), (5, 1)), ((0, 2), (-3, 5))):
        c = cache.cuda()
        kda.kda_pages_copy(c, i32(*src), i32(*dst))
        refused()
        assert np.array_equal(c.cpu().numpy(), gdr.copy(cache.numpy(), src, dst)), (src, dst)
    c = cache.cuda()
    kda.kda_pages_copy(c, i32(3, 3), i32(3, 1))           # onto itself is nothing, and no conflict
    kda.kda_check_device_error()
    assert np.array_equal(c.cpu().numpy(), gdr.copy(cache.numpy(), (3, 3), (3, 1)))

    r = refs.cuda()
    kda.kda_pages_free(r, i32(0, 0, 3, 9))                # 0 twice, 3 is free, 9 is no page
    refused()
    assert r.cpu().tolist() == [0, 0, 1, 0, 0, 0]

    c, r, table = cache.cuda(), refs.cuda(), i32(2, 5, 17, -1)
    live = kda.kda_pages_compact(c, r, table)
    refused()
    assert table.cpu().tolist() == [1, -1, -1, -1] and int(live) == 2 and r.cpu().tolist() == [1, 1, 0, 0, 0, 0]
    assert torch.equal(c[:, 1].cpu(), cache[:, 2])


def _serve(kda, d, dec, pages, refs, io, dk, cu, draws):
    """Prompts prefilled into new pages, forked into samples, decoded, some ended, the cache packed, decoded on."""
    P, Hv = pages.shape[0], pages.shape[1]
    cache = pages.view(1, P, Hv, dk, dk)
    new = torch.full((len(cu) - 1,), -1, dtype=torch.int32, device="cuda")
    prompt = kda.kda_pages_fork(cache, refs, new)
    out0, _ = kda.kda_gdr_forward(*d, torch.tensor(cu, dtype=torch.int32).cuda(), pages, final_state=pages,
                                  initial_index=new, final_index=prompt)
    samples = kda.kda_pages_fork(cache, refs, prompt.repeat_interleave(draws))
    out1 = kda.kda_gdr_decode(*dec[0], pages, samples)
    ended = samples[::2].contiguous()
    kda.kda_pages_free(refs, ended)
    kda.kda_pages_free(refs, prompt)
    table = samples.clone()
    table[::2] = -1
    live = kda.kda_pages_compact(cache, refs, table)
    out2 = kda.kda_gdr_decode(*dec[1], pages, table, torch.zeros_like(out1[:, :1]))
    return out0, out1, out2, table, live


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_a_serving_run(kda, io, dk):
    lens, Hk, Hv, draws, P = [70, 1, 129], 1, 2, 3, 16
    cu, N = cu_of(lens), len(lens) * draws
    d = make(cu[-1], Hk, Hv, dk, dk, io, 12)
    dec = [make(N * T, Hk, Hv, dk, dk, io, 13 + T) for T in (2, 1)]
    dev = [[x[n].view(N, T, *x[n].shape[1:]).cuda() for n in NAMES] for x, T in zip(dec, (2, 1))]
    pages, refs = torch.randn(P, Hv, dk, dk, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[[1, 4]] = 1         # pages of someone else
    other = pages[[1, 4]].clone()
    out0, out1, out2, table, live = _serve(kda, to(d, *NAMES), dev, pages, refs, io, dk, cu, draws)
    kda.kda_check_device_error()
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), cu)
    ex = io == "f32"
    near(out0, ro, io, ex, "prefill")
    st = np.repeat(rs, draws, 0)
    r1, st = gdr.decode(*(f64(t) for t in dev[0]), st)
    near(out1, r1, io, ex, "decode")
    r2, st = gdr.decode(*(f64(t) for t in dev[1]), st)
    near(out2[1::2], r2[1::2], io, ex, "decode after packing")
    assert bool((out2[::2] == 0).all())
    rows = table.cpu().tolist()
    assert int(live) == 2 + N // 2 and max(rows) < int(live) and rows[::2] == [-1] * ((N + 1) // 2)
    near(pages[rows[1::2]], st[1::2], io, ex, "states", stored=False)
    mine = set(rows)
    kept = [p for p in range(int(live)) if p not in mine]
    assert torch.equal(pages[kept], other)


def test_a_captured_run_replays(kda):
    """The same run captured in a graph, replayed on new inputs, beside an eager run on another stream."""
    io, dk, lens, Hk, Hv, draws, P = "bf16", 128, [70, 1, 129], 1, 2, 3, 16
    cu, N = cu_of(lens), len(lens) * draws
    sets = []
    for seed in (20, 30):
        d = make(cu[-1], Hk, Hv, dk, dk, io, seed)
        dec = [make(N * T, Hk, Hv, dk, dk, io, seed + T) for T in (2, 1)]
        sets.append((to(d, *NAMES), [[x[n].view(N, T, *x[n].shape[1:]).cuda() for n in NAMES]
                                     for x, T in zip(dec, (2, 1))]))
    eager = []
    for d, dec in sets:
        pages, refs = torch.zeros(P, Hv, dk, dk, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            eager.append([t.clone() for t in _serve(kda, d, dec, pages, refs, io, dk, cu, draws)] + [pages])
        torch.cuda.current_stream().wait_stream(s)
    d, dec = [x.clone() for x in sets[0][0]], [[x.clone() for x in y] for y in sets[0][1]]
    pages, refs = torch.zeros(P, Hv, dk, dk, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    cug = torch.tensor(cu, dtype=torch.int32).cuda()
    new = torch.full((3,), -1, dtype=torch.int32, device="cuda")

    def body():
        cache = pages.view(1, P, Hv, dk, dk)
        prompt = kda.kda_pages_fork(cache, refs, new)
        out0, _ = kda.kda_gdr_forward(*d, cug, pages, final_state=pages, initial_index=new, final_index=prompt)
        samples = kda.kda_pages_fork(cache, refs, prompt.repeat_interleave(draws, output_size=N))
        out1 = kda.kda_gdr_decode(*dec[0], pages, samples)
        kda.kda_pages_free(refs, samples[::2].contiguous())
        kda.kda_pages_free(refs, prompt)
        table = samples.clone()
        table[::2] = -1
        live = kda.kda_pages_compact(cache, refs, table)
        out2 = kda.kda_gdr_decode(*dec[1], pages, table, torch.zeros_like(out1[:, :1]))
        return out0, out1, out2, table, live

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = body()
    for i in (0, 1, 0):
        for a, b in zip(d, sets[i][0]):
            a.copy_(b)
        for x, y in zip(dec, sets[i][1]):
            for a, b in zip(x, y):
                a.copy_(b)
        pages.zero_()
        refs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, pages), eager[i]):
            assert torch.equal(a, b)
    kda.kda_check_device_error()


def test_backward_captured_beside_an_eager_one(kda):
    d = make(150, 2, 4, 128, 128, "bf16", 40)
    x = [t[None].contiguous() for t in to(d, *NAMES, "dO")]
    eager = kda.kda_gdr_backward(*x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_gdr_backward(*x)
    graph.replay()
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n], eager[n])


def test_gradients_agree_with_differences(kda):
    """A directional difference of the fp32 forward pass: the loss is a sum of 10^4 products of rounding 2^-24
    each, so with a step of 2^-6 the quotient is off by about 2^-24 * 10^2 / 2^-6 = 4e-4 of the products' size
    and by the step's square (2^-12) of the third derivative; the bound is 2^-6 of the gradient's norm."""
    d = make(100, 1, 2, 64, 64, "f32", 41)
    x = {n: d[n][None].cuda() for n in NAMES}
    do, s0 = d["dO"][None].cuda(), d["s0"].cuda()
    gr = kda.kda_gdr_backward(*x.values(), do, None, s0)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(y):
        return float((kda.kda_gdr_forward(*y.values(), None, s0)[0].double() * do.double()).sum())

    for n in NAMES:
        v = torch.randn(x[n].shape, generator=gen, device="cuda")
        v = v / v.norm()
        step = 2.0 ** -6
        lo, hi = ({**x, n: x[n] + s * step * v} for s in (-1, 1))
        num, ana = (loss(hi) - loss(lo)) / (2 * step), float((gr["d" + n].double() * v.double()).sum())
        assert abs(num - ana) <= 2.0 ** -6 * float(gr["d" + n].double().norm()), (n, num, ana)


def test_binding_checks(kda):
    d = make(10, 1, 2, 64, 64, "f32", 42)
    x = to(d, *NAMES)
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_gdr_forward(*x)                                   # packed inputs without cu_seqlens
    with pytest.raises(ValueError):
        kda.kda_gdr_forward(x[0], x[1], x[2], x[3].bfloat16(), x[4], cu)
    with pytest.raises(ValueError):
        kda.kda_gdr_forward(x[0].transpose(0, 2).contiguous().transpose(0, 2), *x[1:], cu)
    with pytest.raises(ValueError):
        kda.kda_gdr_forward(*x, cu, initial_index=cu[:1])         # an index without its pages
    with pytest.raises(ValueError):
        kda.kda_gdr_decode(*x, d["s0"].cuda(), cu)                # index of another length
    with pytest.raises(ValueError):
        kda.kda_pages_fork(torch.zeros(2, 3, 4, device="cuda"), cu, cu)   # refs of another length
    with pytest.raises(kda.KdaError):
        kda.kda_pages_fork(torch.zeros(2, 2, 3, device="cuda"), cu, cu)   # 12-byte pages


def test_no_tokens_pass_the_state_through(kda):
    s0 = torch.randn(2, 2, 64, 128, device="cuda")
    z = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    x = (z(2, 0, 1, 64), z(2, 0, 1, 64), z(2, 0, 2, 128), z(2, 0, 2), z(2, 0, 2))
    sT, d0 = torch.empty_like(s0), torch.empty_like(s0)
    out, _ = kda.kda_gdr_forward(*x, None, s0, final_state=sT)
    kda.kda_gdr_backward(*x, z(2, 0, 2, 128), None, s0, s0, d_initial_state=d0)
    kda.kda_check_device_error()
    assert out.shape == (2, 0, 2, 128) and torch.equal(sT, s0) and torch.equal(d0, s0)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64), ("bf16", 64)])
def test_many_sequences(kda, io, dk):
    """More sequences than a warp looks at in one round of the slot search, lengths from zero on."""
    rng = np.random.default_rng(50)
    lens = [int(n) for n in rng.integers(0, 90, size=70)] + [0, 200, 0]
    cu, Hk, Hv = cu_of(lens), 1, 2
    d = make(cu[-1], Hk, Hv, dk, dk, io, 51, len(lens))
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    sT, d0 = torch.empty_like(d["s0"], device="cuda"), torch.empty_like(d["s0"], device="cuda")
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), cug, d["s0"].cuda(), final_state=sT)
    gr = kda.kda_gdr_backward(*to(d, *NAMES, "dO"), cug, d["s0"].cuda(), d["dS"].cuda(), d_initial_state=d0)
    kda.kda_check_device_error()
    a = [f64(d[n]) for n in NAMES]
    ro, rs = gdr.forward(*a, cu, f64(d["s0"]))
    ref = gdr.backward(*a, cu, f64(d["dO"]), f64(d["s0"]), f64(d["dS"]))
    ex = not tc(io, dk, dk)
    near(out, ro, io, ex, "out")
    near(sT, rs, io, ex, "final state", stored=False)
    near(d0, ref["d_initial_state"], io, ex, "d_initial_state", stored=False)
    near(gr["dv"], ref["dv"], io, ex, "dv")
    for n in ("dq", "dk", "dg", "dbeta"):
        near_grad(gr[n], ref[n], io, ex, n)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 128)])
def test_a_batch_is_its_parts(kda, io, dk):
    """1100 sequences (two rounds of the slot search; more chunks than the GPU has SMs, so blocks take several):
    outputs and gradients are bit for bit those of the batch's two halves, called apart."""
    rng = np.random.default_rng(60)
    lens = [int(n) for n in rng.integers(0, 20, size=1100)]
    lens[37], lens[900] = 700, 500
    cu, N, Hk, Hv = cu_of(lens), 1100, 1, 2
    d = make(cu[-1], Hk, Hv, dk, dk, io, 61)
    gen = torch.Generator(device="cuda").manual_seed(62)
    s0, dS = (0.3 * torch.randn(N, Hv, dk, dk, generator=gen, device="cuda") for _ in range(2))
    x = dict(zip(NAMES + ("dO",), to(d, *NAMES, "dO")))

    def run(a, b):
        rows, offs = slice(cu[a], cu[b]), torch.tensor([c - cu[a] for c in cu[a:b + 1]], dtype=torch.int32, device="cuda")
        y = {n: t[rows].clone() for n, t in x.items()}      # (a view would not start on 16 bytes)
        sT, d0 = torch.empty_like(s0[a:b]), torch.empty_like(s0[a:b])
        out, _ = kda.kda_gdr_forward(*(y[n] for n in NAMES), offs, s0[a:b].contiguous(), final_state=sT)
        gr = kda.kda_gdr_backward(*(y[n] for n in NAMES), y["dO"], offs, s0[a:b].contiguous(), dS[a:b].contiguous(),
                                  d_initial_state=d0)
        return [out, sT, *(gr[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state"))]

    whole, parts = run(0, N), [run(0, 470), run(470, N)]
    kda.kda_check_device_error()
    for i, t in enumerate(whole):
        assert torch.equal(t, torch.cat([p[i] for p in parts])), i


@pytest.mark.parametrize("chunk", [0, 1, 2])
@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_a_wait_that_runs_out_is_reported(kda, chunk, direction):
    """A tile load that is never issued: the bounded wait for it runs out after 1 ms, the blocks let finish what
    they issued and return, the error is reported once, and the next call on the same context is right."""
    lens, Hk, Hv = [200, 10, 130], 1, 2
    cu = cu_of(lens)
    d = make(cu[-1], Hk, Hv, 128, 128, "bf16", 70, 3)
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run():
        if direction == "forward":
            out = kda.kda_gdr_forward(*to(d, *NAMES), cug, d["s0"].cuda())[0]
        else:
            out = kda.kda_gdr_backward(*to(d, *NAMES, "dO"), cug, d["s0"].cuda(), d["dS"].cuda())["dv"]
        kda.kda_check_device_error()
        return out

    kda.kda_set_wait_test_hooks(1_000_000, chunk)
    try:
        with pytest.raises(kda.KdaError) as e:
            run()
        assert e.value.status == 5
    finally:
        kda.kda_set_wait_test_hooks(0, -1)
    kda.kda_check_device_error()
    got = run()
    a = [f64(d[n]) for n in NAMES]
    if direction == "forward":
        near(got, gdr.forward(*a, cu, f64(d["s0"]))[0], "bf16", False, "out")
    else:
        near(got, gdr.backward(*a, cu, f64(d["dO"]), f64(d["s0"]), f64(d["dS"]))["dv"], "bf16", False, "dv")


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_two_calls_at_once(kda, io, dk):
    """Calls on two streams, each with its own workspace, beside one another and in another order: the same bits."""
    sets = []
    for seed in (80, 81):
        d = make(900, 1, 3, dk, dk, io, seed, 2)
        sets.append((to(d, *NAMES, "dO"), d["s0"].cuda()))
    cug = torch.tensor([0, 610, 900], dtype=torch.int32, device="cuda")

    def call(i):
        x, s0 = sets[i]
        sT = torch.empty_like(s0)
        out, _ = kda.kda_gdr_forward(*x[:5], cug, s0, final_state=sT)
        gr = kda.kda_gdr_backward(*x, cug, s0)
        return [out, sT, *(gr[n] for n in ("dq", "dk", "dv", "dg", "dbeta"))]

    alone = [call(i) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for order in ((0, 1), (1, 0)):
        got = {}
        for i in order:
            with torch.cuda.stream(streams[i]):
                got[i] = [call(i) for _ in range(3)]
        torch.cuda.synchronize()
        kda.kda_check_device_error()
        for i in (0, 1):
            for run in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(run, alone[i]))


def test_far_pages(kda):
    """Pages behind 2^32 bytes and 2^31 elements of the cache: states read, written, copied and packed there."""
    Hv, dk, P = 32, 128, 4200                                  # 2 MB a page, 8.8 GB
    pages = torch.empty(P, Hv, dk, dk, device="cuda")
    far, N = torch.tensor([4199, 2060, 4100], dtype=torch.int32), 3
    d = make(N * 2, 16, Hv, dk, dk, "bf16", 90, N)
    pages[far.long().cuda()] = d["s0"].cuda()
    x = [t.view(N, 2, *t.shape[1:]) for t in to(d, *NAMES)]
    got = kda.kda_gdr_decode(*x, pages, far.cuda())
    ro, rs = gdr.decode(*(f64(t) for t in x), f64(d["s0"]))
    near(got, ro, "bf16", True, "decode")
    near(pages[far.long().cuda()], rs, "bf16", True, "states", stored=False)
    pages[far.long().cuda()] = d["s0"].cuda()
    cu = [0, 1, 1, 6]
    start, end = far.cuda(), torch.tensor([4198, 4196, 3000], dtype=torch.int32, device="cuda")
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), torch.tensor(cu, dtype=torch.int32, device="cuda"), pages,
                                 final_state=pages, initial_index=start, final_index=end)
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), cu, f64(d["s0"]))
    near(out, ro, "bf16", False, "forward")
    near(pages[end.long()], rs, "bf16", False, "final states", stored=False)
    cache = pages.view(1, P, Hv, dk, dk)
    kept = pages[end.long()].clone()
    kda.kda_pages_copy(cache, end, torch.tensor([4000, 1, 4195], dtype=torch.int32, device="cuda"))
    assert torch.equal(pages[[4000, 1, 4195]], kept)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[end.long()] = 1
    table = end.clone()
    assert int(kda.kda_pages_compact(cache, refs, table)) == 3
    kda.kda_check_device_error()
    assert sorted(table.tolist()) == [0, 1, 2] and torch.equal(pages[table.long()], kept)


def test_indices_below_minus_one_are_refused(kda):
    d = make(4, 1, 1, 128, 128, "bf16", 91, 4)
    state, i32 = d["s0"].cuda(), lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out = torch.full((4, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_gdr_decode(*to(d, *NAMES), state, i32(0, -2, -1, 3), out)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == 7
    assert bool((out[1:3] == 7.0).all()) and not bool((out[[0, 3]] == 7.0).any())
    assert torch.equal(state[1:3].cpu(), d["s0"][1:3])


def test_inputs_on_another_stream_and_strided_inputs(kda):
    """A call made on the stream that its inputs are made on; inputs that are not contiguous are refused."""
    s = torch.cuda.Stream()
    d = make(130, 1, 2, 128, 128, "bf16", 92)
    x = to(d, *NAMES)
    with torch.cuda.stream(s):
        y = [t.clone()[None] for t in x]
        out, _ = kda.kda_gdr_forward(*y)
        explicit, _ = kda.kda_gdr_forward(*y, stream=s)
    s.synchronize()
    ro, _ = gdr.forward(*(f64(d[n]) for n in NAMES), [0, 130])
    near(out[0], ro, "bf16", False, "out")
    assert torch.equal(out, explicit)
    wide = torch.zeros(1, 130, 2, 256, dtype=torch.bfloat16, device="cuda")[..., :128]
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_gdr_forward(y[0], y[1], wide, y[3], y[4])


def test_exponents_far_apart(kda):
    """Keys, queries and values of very different sizes in one chunk; the state's small entries keep their bits."""
    d = make(200, 1, 2, 128, 128, "bf16", 93)
    scale = 2.0 ** torch.randint(-6, 7, (200, 1, 1), generator=torch.Generator().manual_seed(1)).float()
    d["v"] = (d["v"].float() * scale).bfloat16()
    d["q"] = (d["q"].float() * scale.flip(0)).bfloat16()
    x = [t[None] for t in to(d, *NAMES)]
    sT = torch.empty_like(d["s0"], device="cuda")
    out, _ = kda.kda_gdr_forward(*x, None, d["s0"].cuda(), final_state=sT)
    kda.kda_check_device_error()
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), [0, 200], f64(d["s0"]))
    near(out[0], ro, "bf16", False, "out")
    near(sT, rs, "bf16", False, "state", stored=False)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_a_batch_of_equal_lengths_is_the_packed_call(kda, io, dk):
    """[B, T, ...] inputs, given buffers and a given workspace, gradients in place of d_final_state: the same bits
    as the packed call with allocated ones."""
    B, T, Hk, Hv = 3, 150, 2, 4
    d = make(B * T, Hk, Hv, dk, dk, io, 100, B)
    x = to(d, *NAMES, "dO")
    s0, dS = d["s0"].cuda(), d["dS"].cuda()
    cu = torch.tensor(cu_of([T] * B), dtype=torch.int32, device="cuda")
    sT, d0 = torch.empty_like(s0), torch.empty_like(s0)
    out, _ = kda.kda_gdr_forward(*x[:5], cu, s0, final_state=sT)
    gr = kda.kda_gdr_backward(*x, cu, s0, dS, d_initial_state=d0)
    y = [t.view(B, T, *t.shape[1:]) for t in x]
    ws = [torch.empty(kda.kda_gdr_workspace_size(B, B * T, Hk, Hv, dk, dk, DT[io], backward=b), dtype=torch.uint8,
                      device="cuda") for b in (False, True)]
    out2, sT2 = torch.empty_like(y[2]), torch.empty_like(s0)
    kda.kda_gdr_forward(*y[:5], None, s0, out2, sT2, workspace=ws[0])
    both = dS.clone()
    gr2 = kda.kda_gdr_backward(*y, None, s0, both, d_initial_state=both, workspace=ws[1])
    kda.kda_check_device_error()
    assert torch.equal(out, out2.view_as(out)) and torch.equal(sT, sT2) and torch.equal(both, d0)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(gr[n], gr2[n].view_as(gr[n])), n
    with pytest.raises(kda.KdaError) as e:
        kda.kda_gdr_forward(*y[:5], None, s0, out2, sT2, workspace=ws[0][:-1])
    assert e.value.status == 6
    with pytest.raises(kda.KdaError) as e:
        kda.kda_gdr_backward(*y, None, s0, workspace=ws[1][16:])
    assert e.value.status in (3, 6)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_decode_of_many_tokens_is_the_forward_pass(kda, io, dk):
    N, T, Hk, Hv = 2, 70, 1, 2
    d = make(N * T, Hk, Hv, dk, dk, io, 101, N)
    x = [t.view(N, T, *t.shape[1:]) for t in to(d, *NAMES)]
    state = d["s0"].cuda()
    out = kda.kda_gdr_decode(*x, state)
    sT = torch.empty_like(state)
    fwd, _ = kda.kda_gdr_forward(*x, None, d["s0"].cuda(), final_state=sT)
    kda.kda_check_device_error()
    ro, rs = gdr.decode(*(f64(t) for t in x), f64(d["s0"]))
    near(out, ro, io, True, "decode")
    near(state, rs, io, True, "state", stored=False)
    near(fwd, ro, io, io == "f32", "forward")
    near(sT, rs, io, io == "f32", "forward's state", stored=False)


def test_pages_with_nothing_to_do(kda):
    """No ids, no table, no free page, no live page, a cache of one page: calls that change nothing, or only refs."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.randn(2, 1, 8, device="cuda")
    was = cache.clone()
    none = i32()
    refs = i32(0)
    assert kda.kda_pages_fork(cache, refs, none).numel() == 0
    kda.kda_pages_copy(cache, none, none)
    kda.kda_pages_free(refs, none)
    assert int(kda.kda_pages_compact(cache, refs)) == 0 and torch.equal(cache, was) and refs.tolist() == [0]
    assert kda.kda_pages_fork(cache, refs, i32(-1, -1)).tolist() == [0, -1]
    assert not bool(cache.any()) and refs.tolist() == [1]
    assert kda.kda_pages_fork(cache, refs, i32(0)).tolist() == [-1]           # no page left: no error
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    assert int(kda.kda_pages_compact(cache, refs, table)) == 1 and bool((table == -1).all())
    kda.kda_check_device_error()


def test_many_key_heads(kda):
    """More heads than SMs, one token each, and a group of five value heads."""
    d = make(3, 150, 150, 128, 128, "bf16", 102, 3)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    sT = torch.empty_like(d["s0"], device="cuda")
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), cu, d["s0"].cuda(), final_state=sT)
    ro, rs = gdr.forward(*(f64(d[n]) for n in NAMES), [0, 1, 2, 3], f64(d["s0"]))
    near(out, ro, "bf16", False, "out")
    near(sT, rs, "bf16", False, "state", stored=False)
    for io, dk in (("bf16", 128), ("f32", 64)):
        d = make(90, 1, 5, dk, dk, io, 103)
        gr = kda.kda_gdr_backward(*(t[None] for t in to(d, *NAMES, "dO")))
        ref = gdr.backward(*(f64(d[n]) for n in NAMES), [0, 90], f64(d["dO"]))
        for n in ("dq", "dk", "dg", "dbeta"):
            near_grad(gr[n][0], ref[n], io, io == "f32", n)
    kda.kda_check_device_error()


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_a_call_on_a_given_stream_keeps_what_it_allocated(kda, io, dk):
    """The workspace and outputs of a call on another stream are not handed out again while it runs."""
    d = make(6000, 1, 2, dk, dk, io, 110)
    x = [t[None] for t in to(d, *NAMES, "dO")]
    want = kda.kda_gdr_forward(*x[:5])[0]
    grads = kda.kda_gdr_backward(*x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sizes = [kda.kda_gdr_workspace_size(1, 6000, 1, 2, dk, dk, DT[io], backward=b) for b in (False, True)]
    torch.cuda.synchronize()
    out = kda.kda_gdr_forward(*x[:5], stream=s)[0]
    gr = kda.kda_gdr_backward(*x, stream=s)
    for _ in range(20):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    kda.kda_check_device_error()
    assert torch.equal(out, want)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(gr[n], grads[n]), n


def test_short_calls_answer_as_the_checked_ones(kda):
    """The marshalling in C++ takes what the Python checks take and nothing else: its results and its refusals."""
    d = make(12, 2, 4, 64, 64, "f32", 111, 3)
    x = to(d, *NAMES)
    cu = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device="cuda")
    s0 = d["s0"].cuda()
    cur = torch.cuda.current_stream()
    for init, ii, fi in ((None, None, None), (s0, None, None), (s0, cu[:3].contiguous(), None)):
        ii = None if ii is None else torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
        sT = torch.empty_like(s0)
        a, _ = kda.kda_gdr_forward(*x, cu, init, None, sT, initial_index=ii)
        tT = torch.empty_like(s0)
        b, _ = kda.kda_gdr_forward(*x, cu, init, None, tT, initial_index=ii, stream=cur)
        assert torch.equal(a, b) and torch.equal(sT, tT)
    y = [t[:3].clone() for t in x]
    st = [s0.clone() for _ in range(2)]
    assert torch.equal(kda.kda_gdr_decode(*y, st[0]), kda.kda_gdr_decode(*y, st[1], stream=cur)) and torch.equal(*st)
    for bad in (x[:1] + x[:1] + x[1:4], [x[0], x[1], x[2], x[3][:, :3], x[4]], [x[0], x[1], x[2].bfloat16(), x[3], x[4]],
                [x[0].cpu(), *x[1:]], [x[0], x[1], x[2].transpose(0, 1).contiguous().transpose(0, 1), x[3], x[4]]):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_gdr_forward(*bad, cu)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_gdr_decode(*(t[:3] for t in bad), s0)
    with pytest.raises(TypeError):
        kda.kda_gdr_decode(*(t[:3].half() for t in x), s0)
    with pytest.raises(kda.KdaError):                       # 48 channels: the library's own refusal
        kda.kda_gdr_decode(*(t[:3, :, :48].clone() for t in x[:3]), *(t[:3].clone() for t in x[3:]),
                           torch.zeros(3, 4, 48, 48, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_pages_free(cu.long(), cu)
    with pytest.raises(ValueError):
        kda.kda_pages_compact(torch.zeros(1, 4, 4, device="cuda"), cu, cu.float())


def test_workspaces_that_are_none(kda):
    """A workspace on the host, of another type or of strided bytes is refused before a kernel sees it."""
    d = make(10, 2, 2, 64, 64, "f32", 43)
    x = to(d, *NAMES)
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    need = kda.kda_gdr_workspace_size(1, 10, 2, 2, 64, 64, torch.float32, backward=True)
    cache, refs = torch.zeros(2, 3, 4, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.float32, device="cuda"),
               torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            kda.kda_gdr_forward(*x, cu, workspace=ws)
        with pytest.raises(ValueError):
            kda.kda_gdr_backward(*x, torch.ones_like(x[2]), cu, workspace=ws)
        with pytest.raises(ValueError):
            kda.kda_pages_compact(cache, refs, workspace=ws)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_a_row_follow_one_another(kda, io, dk, captured):
    """Each call's kernels are brought up while what is before them on the stream ends: a run of calls whose inputs
    are written just before them, by torch and by each other, gives the bits of the run with a wait behind each step."""
    N, T, Hk, Hv, R = 3, 70, 2, 4, 4
    d = make(R * N * T, Hk, Hv, dk, dk, io, 95, N)
    src = [t.view(R, N, T, *t.shape[1:]) for t in to(d, *NAMES)]
    first, ids = d["s0"].cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    x, outs = [t[0].clone() for t in src], [torch.empty_like(src[2]) for _ in range(2)]
    grads = [torch.empty_like(src[0]) for _ in range(2)]
    pages, refs = torch.empty(1, 2 * N, Hv, dk, dk, device="cuda"), torch.empty(2 * N, dtype=torch.int32, device="cuda")

    def run(step):
        pages[0, :N].copy_(first)
        refs.fill_(0)[:N].fill_(1)
        kids = kda.kda_pages_fork(pages, refs, ids)
        step()
        for r in range(R):
            for a, b in zip(x, src):
                a.copy_(b[r])
            step()
            kda.kda_gdr_forward(*x, None, pages[0], outs[0][r], pages[0], initial_index=kids, final_index=kids)
            step()
            kda.kda_gdr_decode(*x, pages[0], kids, outs[1][r])
            step()
            gr = kda.kda_gdr_backward(*x, outs[1][r], None, pages[0, N:])
            step()
            grads[0][r].copy_(gr["dq"])
            grads[1][r].copy_(gr["dk"])
        return kids

    def answer():
        torch.cuda.synchronize()
        return [t.clone() for t in (*outs, *grads, pages)]
    assert run(torch.cuda.synchronize).tolist() == [3, 4, 5]
    want = answer()
    for t in (*outs, *grads, pages):
        t.zero_()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(lambda: None)
        for _ in range(3):
            graph.replay()
    else:
        for _ in range(3):
            run(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(answer(), want))
    kda.kda_check_device_error()


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_short_backward_calls_answer_as_the_checked_ones(kda, io, dk):
    """Packed and batched, with states and without, an empty sequence among them; and what both refuse."""
    d = make(150, 1, 3, dk, dk, io, 112, 3)
    x, do, s0, dT = to(d, *NAMES), d["v"].cuda().flip(0), d["s0"].cuda(), d["s0"].cuda().flip(0)
    cu = torch.tensor([0, 80, 80, 150], dtype=torch.int32, device="cuda")
    cur = torch.cuda.current_stream()
    batch = [t.view(3, 50, *t.shape[1:]) for t in (*x, do)]
    for ins, c in (([*x, do], cu), (batch, None)):
        for states in ((None, None), (s0, None), (s0, dT)):
            got = []
            for stream in (None, cur):
                first = torch.empty_like(s0) if states[0] is not None else None
                got.append(kda.kda_gdr_backward(*ins, c, *states, d_initial_state=first, stream=stream))
            assert list(got[0]) == list(got[1])
            assert all(torch.equal(p, q) for p, q in zip(got[0].values(), got[1].values()) if p is not None)
            assert got[0]["dq"].shape == ins[0].shape and got[0]["dg"].shape == ins[3].shape
    for bad in ([*x, do[:-1]], [*x, do.cpu()], [*x[:3], x[3][:, :2], x[4], do], [x[0][:, :, :32], *x[1:], do]):
        with pytest.raises(ValueError):
            kda.kda_gdr_backward(*bad, cu)
    with pytest.raises(ValueError):
        kda.kda_gdr_backward(*x, do, cu, s0[:2])
    with pytest.raises(kda.KdaError):                       # 48 channels: the library's own refusal
        kda.kda_gdr_backward(*(t[..., :48].clone() if t.dim() == 3 else t for t in x), do[..., :48].clone(), cu)


@pytest.mark.parametrize("N,T,Hk,Hv", [(2, 420, 16, 96), (3, 321, 50, 100), (1, 200, 1, 150), (5, 1024, 8, 32)])
def test_a_batch_whose_heads_walk_in_two_parts(kda, N, T, Hk, Hv):
    """More walks than SMs, of one length: some heads walk before the others' chunks are prepared.  The packed call,
    which takes all heads at once, gives the same bits; states in pages, in place; twice over the same workspace."""
    torch.manual_seed(113)
    unit = torch.nn.functional.normalize
    x = [unit(torch.randn(N, T, Hk, 128, device="cuda"), dim=-1).bfloat16() for _ in range(2)]
    x += [torch.randn(N, T, Hv, 128, device="cuda").bfloat16(), -torch.rand(N, T, Hv, device="cuda").bfloat16(),
          torch.rand(N, T, Hv, device="cuda").bfloat16()]
    pages = torch.randn(N + 2, Hv, 128, 128, device="cuda")
    start = torch.arange(N, 0, -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kda.kda_gdr_workspace_size(N, N * T, Hk, Hv, 128, 128, torch.bfloat16), dtype=torch.uint8, device="cuda")
    cu = torch.arange(0, N * T + 1, T, dtype=torch.int32, device="cuda")
    answers = []
    for packed in (True, False, False):
        p = pages.clone()
        y = [t.flatten(0, 1) for t in x] if packed else x
        ws.fill_(255)                              # NaN, were it read
        out, _ = kda.kda_gdr_forward(*y, cu if packed else None, p, None, p, initial_index=start, final_index=start, workspace=ws)
        answers.append((out.flatten(), p))
    graph = torch.cuda.CUDAGraph()
    p, out = pages.clone(), torch.empty_like(x[2])
    with torch.cuda.graph(graph):
        kda.kda_gdr_forward(*x, None, p, out, p, initial_index=start, final_index=start, workspace=ws)
        out.add_(0)                                # a kernel behind, which reads all of it
    p.copy_(pages)
    graph.replay()
    answers.append((out.flatten(), p))
    kda.kda_check_device_error()
    for a in answers[1:]:
        assert torch.equal(a[0], answers[0][0]) and torch.equal(a[1], answers[0][1])


def _few_long(lens, Hk, Hv, seed):
    """bf16 inputs of packed sequences whose walks leave SMs idle, and those with one-token sequences behind them,
    so many that the call takes all chunks at once."""
    torch.manual_seed(seed)
    more = 148 // Hv + 1
    T, unit = sum(lens) + more, torch.nn.functional.normalize
    x = [unit(torch.randn(T, Hk, 128, device="cuda"), dim=-1).bfloat16() for _ in range(2)]
    x += [torch.randn(T, Hv, 128, device="cuda").bfloat16(), -0.1 * torch.rand(T, Hv, device="cuda"), torch.rand(T, Hv, device="cuda")]
    x = [t.bfloat16() for t in x]
    offs = torch.tensor([0, *lens, *[1] * more], dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    return x, offs, sum(lens)


@pytest.mark.parametrize("lens,Hk,Hv", [((3000, 0, 456), 4, 16), ((4100,), 1, 32), ((64 * 40, 64 * 60 + 1, 250, 64 * 52), 3, 30),
                                        ((12345,), 2, 4)])
def test_few_long_sequences_walk_in_two_parts(kda, lens, Hk, Hv):
    """A part of every sequence's chunks walks before the others are prepared: the bits of the call that takes all at
    once; with dense states, with pages in place, without states, replayed from a graph."""
    x, offs, T = _few_long(lens, Hk, Hv, 114)
    N, M = len(lens), offs.numel() - 1
    s0 = torch.randn(M, Hv, 128, 128, device="cuda")
    sT = torch.empty_like(s0)
    want, _ = kda.kda_gdr_forward(*x, offs, s0, None, sT)
    zero, _ = kda.kda_gdr_forward(*x, offs)
    y, cu = [t[:T].clone() for t in x], offs[:N + 1].clone()
    ws = torch.empty(kda.kda_gdr_workspace_size(N, T, Hk, Hv, 128, 128, torch.bfloat16), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        ws.fill_(255)
        got = torch.empty_like(sT[:N])
        out, _ = kda.kda_gdr_forward(*y, cu, s0[:N].clone(), None, got, workspace=ws)
        assert torch.equal(out, want[:T]) and torch.equal(got, sT[:N])
        ws.fill_(255)
        out, _ = kda.kda_gdr_forward(*y, cu, workspace=ws)
        assert torch.equal(out, zero[:T])
    if N == 1:
        out, _ = kda.kda_gdr_forward(*(t[None] for t in y), None, s0[:1].clone(), None, got)
        assert torch.equal(out[0], want[:T]) and torch.equal(got, sT[:1])
    at = torch.randperm(N + 2, device="cuda")[:N].to(torch.int32)
    pages, kept = torch.randn(N + 2, Hv, 128, 128, device="cuda"), None
    pages[at.long()] = s0[:N]
    first = pages.clone()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(y[2])
    with torch.cuda.graph(graph):
        kda.kda_gdr_forward(*y, cu, pages, out, pages, initial_index=at, final_index=at, workspace=ws)
        kept = pages.clone()                       # a kernel behind, which reads all of them
    for _ in range(2):
        pages.copy_(first)
        graph.replay()
        assert torch.equal(out, want[:T]) and torch.equal(kept[at.long()], sT[:N])
        rest = [i for i in range(N + 2) if i not in at.tolist()]
        assert torch.equal(kept[rest], first[rest])
    kda.kda_check_device_error()


def test_bad_pages_of_few_long_sequences(kda):
    """In two parts as in one: a page that another sequence starts from is not written, of two that end on one page
    the first does, indices out of range count as none; each is reported."""
    lens, Hk, Hv = (3000, 80, 456), 4, 16
    x, offs, T = _few_long(lens, Hk, Hv, 115)
    y, cu = [t[:T].clone() for t in x], offs[:4].clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    first = torch.randn(6, Hv, 128, 128, device="cuda")

    def call(start, end):
        p = first.clone()
        kda.kda_gdr_forward(*y, cu, p, None, p, initial_index=start, final_index=end)
        return p
    good = call(i32(0, 1, 2), i32(3, 4, 5))
    kda.kda_check_device_error()
    for start, end, written in ((i32(0, 1, 2), i32(1, 4, 5), (4, 5)), (i32(0, 1, 2), i32(3, 3, 5), (3, 5)),
                                (i32(0, 1, 2), i32(6, 4, -7), (4,))):
        got = call(start, end)
        with pytest.raises(kda.KdaError):
            kda.kda_check_device_error()
        for p in range(6):
            assert torch.equal(got[p], good[p] if p in written else first[p]), p
    with pytest.raises(kda.KdaError):
        call(i32(9, 1, 2), i32(3, 4, 5))
        kda.kda_check_device_error()
    none = call(i32(-1, 1, 2), i32(3, 4, 5))
    got = call(i32(9, 1, 2), i32(3, 4, 5))
    assert torch.equal(got, none)
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_a_call_on_a_given_stream_takes_no_block_in_use(kda, io, dk):
    """Blocks that the current stream has freed and still writes are not what a call on another stream allocates."""
    N, T, Hk, Hv = 2, 700, 1, 2
    d = make(N * T, Hk, Hv, dk, dk, io, 120, N)
    x = [t.view(N, T, *t.shape[1:]) for t in to(d, *NAMES, "dO")]
    wide = x[0].repeat(1, 1, 2, 1)                       # the per-channel rule has as many key heads as value heads
    y = (wide, wide, x[2], -wide.abs(), x[4])
    s0, tok = d["s0"].cuda(), [t[:, 0].contiguous() for t in x[:5]]
    cache, ids = torch.randn(2, 9, 64, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    refs = torch.tensor([1, 1, 1, 0, 0, 1, 0, 0, 1], dtype=torch.int32, device="cuda")
    calls = {                                            # the function, and its arguments (made anew: some are written)
        "forward": (kda.kda_gdr_forward, lambda: (*x[:5], None, s0)),
        "backward": (kda.kda_gdr_backward, lambda: (*x, None, s0)),
        "decode": (kda.kda_gdr_decode, lambda: (*tok, s0.clone())),
        "fork": (kda.kda_pages_fork, lambda: (cache.clone(), refs.clone(), ids)),
        "compact": (kda.kda_pages_compact, lambda: (cache.clone(), refs.clone())),
        "chunked": (kda.kda_forward_chunked, lambda: (*y, s0)),
        "chunked backward": (kda.kda_backward_chunked, lambda: (*y, x[5], s0)),
    }
    spaces = [kda.kda_backward_workspace_size(N, T, Hv, dk, dk, DT[io]), kda.kda_pages_workspace_size(9),
              *(kda.kda_gdr_workspace_size(N, N * T, Hk, Hv, dk, dk, DT[io], backward=b) for b in (False, True))]
    tensors = lambda r: [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,))  # noqa: E731
                         if t is not None]
    s = torch.cuda.Stream()
    for name, (call, args) in calls.items():
        want, given = tensors(call(*args())), args()
        torch.cuda.synchronize()
        busy = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in [t.nbytes for t in want] + spaces for _ in range(2)]
        torch.cuda._sleep(100_000_000)                   # tens of ms, behind which the blocks are written
        for b in busy:
            b.fill_(255)
        del busy, b
        got = tensors(call(*given, stream=s))
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), name
    kda.kda_check_device_error()


@pytest.mark.parametrize("N,T,Hv,chunk", [
    (1, 8192, 140, 50), (1, 8192, 140, 0),     # cut at chunk 119: the first part gives up
    (1, 8192, 140, 125),                       # the second does
    (2, 420, 96, 3),                           # cut at a head
    (2, 900, 8, 5),                            # in one part
    (1, 8192, 140, -2 - 50), (1, 8192, 140, -2 - 125), (2, 420, 96, -2 - 3), (2, 900, 8, -2 - 5),   # what is before the walk
])
def test_a_walk_that_gives_up_keeps_no_state(kda, N, T, Hv, chunk):
    """A forward pass whose wait runs out leaves the final pages as they were, however it is cut, and says so; the
    same call without the failure is right afterwards."""
    torch.manual_seed(121)
    unit = torch.nn.functional.normalize
    x = [unit(torch.randn(N, T, 2, 128, device="cuda"), dim=-1).bfloat16() for _ in range(2)]
    x += [torch.randn(N, T, Hv, 128, device="cuda").bfloat16(), -0.1 * torch.rand(N, T, Hv, device="cuda"), torch.rand(N, T, Hv, device="cuda")]
    x = [t.bfloat16() for t in x]
    first = torch.randn(2 * N + 1, Hv, 128, 128, device="cuda")
    ids = torch.arange(2 * N, -1, -1, dtype=torch.int32, device="cuda")
    start, end = ids[:N].clone(), ids[N:2 * N].clone()
    ws = torch.empty(kda.kda_gdr_workspace_size(N, N * T, 2, Hv, 128, 128, torch.bfloat16), dtype=torch.uint8, device="cuda")

    def call(in_place):
        p = first.clone()
        ws.fill_(1)                            # what a part that was not computed would be taken for
        out, _ = kda.kda_gdr_forward(*x, None, p, None, p, initial_index=start, final_index=start if in_place else end, workspace=ws)
        return out, p
    want = [call(b) for b in (True, False)]
    kda.kda_check_device_error()
    for in_place, (out, pages) in zip((True, False), want):
        kda.kda_set_wait_test_hooks(1_000_000, chunk)
        try:
            _, got = call(in_place)
            with pytest.raises(kda.KdaError) as e:
                kda.kda_check_device_error()
            assert e.value.status == 5
        finally:
            kda.kda_set_wait_test_hooks(0, -1)
        assert torch.equal(got, first)
        again = call(in_place)
        kda.kda_check_device_error()
        assert torch.equal(again[0], out) and torch.equal(again[1], pages)
        assert not torch.equal(pages, first)


@pytest.mark.parametrize("chunk", [0, 2, 9])
def test_a_backward_call_whose_first_launch_gives_up_is_reported(kda, chunk):
    """The tiles of a chunk never come in the launch before the walks: both walks stop there, the error is reported
    once, and the next call is right."""
    d = make(2 * 640, 1, 2, 128, 128, "bf16", 122, 2)
    x = [t.view(2, 640, *t.shape[1:]) for t in to(d, *NAMES, "dO")]
    want = kda.kda_gdr_backward(*x, None, d["s0"].cuda(), d["dS"].cuda())
    first = torch.full((2, 2, 128, 128), 7.0, device="cuda")
    kda.kda_set_wait_test_hooks(1_000_000, -2 - chunk)
    try:
        kda.kda_gdr_backward(*x, None, d["s0"].cuda(), d["dS"].cuda(), d_initial_state=first)
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == 5
    finally:
        kda.kda_set_wait_test_hooks(0, -1)
    assert bool((first == 7.0).all())
    got = kda.kda_gdr_backward(*x, None, d["s0"].cuda(), d["dS"].cuda())
    kda.kda_check_device_error()
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
def test_marshalling_in_python_gives_the_same_calls(kda, monkeypatch, io, dk):
    d = make(150, 1, 3, dk, dk, io, 123, 3)
    x, do, cu = to(d, *NAMES), d["v"].cuda().flip(0), torch.tensor([0, 80, 80, 150], dtype=torch.int32, device="cuda")
    tok = [t[:3].contiguous() for t in x]
    ids, refs = torch.tensor([0, -1], dtype=torch.int32, device="cuda"), torch.tensor([1, 0, 2, 0, 1], dtype=torch.int32)

    def run():
        s0, r, cache = d["s0"].cuda(), refs.cuda(), torch.arange(80.0, device="cuda").view(1, 5, 16)
        sT = torch.empty_like(s0)
        out, _ = kda.kda_gdr_forward(*x, cu, s0, final_state=sT)
        gr = kda.kda_gdr_backward(*x, do, cu, s0)
        step = kda.kda_gdr_decode(*tok, s0)
        kids = kda.kda_pages_fork(cache, r, ids)
        kda.kda_pages_free(r, ids)
        live = kda.kda_pages_compact(cache, r)
        kda.kda_check_device_error()
        return [out, sT, *(gr[n] for n in ("dq", "dk", "dv", "dg", "dbeta")), step, s0, kids, r, live, cache]
    assert not isinstance(kda._calls, kda._NoCalls)              # built here
    want = run()
    monkeypatch.setattr(kda, "_calls", kda._NoCalls())
    assert all(torch.equal(a, b) for a, b in zip(run(), want))


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_copies_and_other_streams(kda, io, dk, captured):
    """Kernels that are brought up early wait for what is before them that is no kernel of their stream: a copy from
    the host, a fill, and another stream's work behind an event."""
    N, T, Hk, Hv, R = 3, 70, 2, 4, 3
    d = make(R * N * T, Hk, Hv, dk, dk, io, 124, N)
    src = [t.view(R, N, T, *t.shape[1:]) for t in (d[n].pin_memory() for n in NAMES)]
    x, first = [t[0].cuda() for t in src], d["s0"].cuda()
    state, refs, ids = first.clone(), torch.zeros(N, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")
    outs, side = [torch.empty(R, *src[2].shape[1:], dtype=DT[io], device="cuda") for _ in range(2)], torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        state.copy_(first)
        for r in range(R):
            for a, b in zip(x, src):                       # copies from the host, then a call
                a.copy_(b[r], non_blocking=True)
            kda.kda_gdr_forward(*x, None, state, outs[0][r], state)
            side.wait_stream(main)
            with torch.cuda.stream(side):                  # inputs that another stream makes, late
                torch.cuda._sleep(200_000)
                for a in x[:3]:
                    a.mul_(0.5)
            main.wait_stream(side)
            kda.kda_gdr_decode(*x, state, None, outs[1][r])
            side.wait_stream(main)
            with torch.cuda.stream(side):
                refs.zero_()
            main.wait_stream(side)
            kda.kda_pages_fork(state[None], refs, torch.full_like(ids, -1) if r == R - 2 else ids[:0])

    def plain():
        s, got = f64(d["s0"]), [[], []]
        for r in range(R):
            a = [f64(t[r]) for t in src]
            flat = [t.reshape(N * T, *t.shape[2:]) for t in a]
            o, s = gdr.forward(*flat, cu_of([T] * N), s)
            got[0].append(o.reshape(a[2].shape))
            a = [0.5 * t for t in a[:3]] + a[3:]
            o, s = gdr.decode(*a, s)
            got[1].append(o)
            if r == R - 2:
                s = np.zeros_like(s)
        return np.stack(got[0]), np.stack(got[1]), s
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(2):
            graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    kda.kda_check_device_error()
    ro, rd, rs = plain()
    near(outs[0], ro, io, io == "f32", "forward")
    near(outs[1], rd, io, io == "f32", "decode")
    near(state, rs, io, io == "f32", "states", stored=False)


@pytest.mark.parametrize("io,dk", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("forked", [False, True])
def test_captured_calls_on_a_given_stream(kda, io, dk, forked):
    """stream= while it is captured, as the current stream or forked from it: what the calls allocate is the graph's."""
    N, T, Hk, Hv = 2, 130, 1, 2
    d = make(N * T, Hk, Hv, dk, dk, io, 125, N)
    x, s0 = [t.view(N, T, *t.shape[1:]) for t in to(d, *NAMES, "dO")], d["s0"].cuda()
    out, kept = [torch.zeros_like(x[2]) for _ in range(2)], torch.zeros_like(x[0])
    refs, ids = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((2,), -1, dtype=torch.int32, device="cuda")
    cache, kids = torch.ones(1, 3, 8, device="cuda"), torch.full_like(ids, 9)
    graph, main, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        s = side if forked else main
        s.wait_stream(main)
        a, _ = kda.kda_gdr_forward(*x[:5], None, s0, stream=s)
        gr = kda.kda_gdr_backward(*x, None, s0, stream=s)
        k = kda.kda_pages_fork(cache, refs, ids, stream=s)
        main.wait_stream(s)
        out[0].copy_(a)
        kept.copy_(gr["dq"])
        kids.copy_(k)
        del a, gr, k                                       # read on one stream, made on the other
        junk = [torch.full_like(x[2], 7.0) for _ in range(8)]
        s.wait_stream(main)
        b, _ = kda.kda_gdr_forward(*x[:5], None, s0, stream=s)
        main.wait_stream(s)
        out[1].copy_(b)
    want = kda.kda_gdr_forward(*x[:5], None, s0)[0]
    dq = kda.kda_gdr_backward(*x, None, s0)["dq"]
    for _ in range(2):
        for t in (*out, kept, refs):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want) and torch.equal(kept, dq)
        assert kids.tolist() == [0, 1] and bool((junk[0] == 7.0).all())
    kda.kda_check_device_error()
