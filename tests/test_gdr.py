"""Head-gated delta rule and state-cache pages without a GPU: the 64-bit reference against differences
and an independent form, and the refusals of the entry points (each before any launch)."""
import ctypes

import numpy as np
import pytest

from oracle import gdr


def _inputs(rng, T, Hk, Hv, dk, dv, N):
    return (rng.normal(size=(T, Hk, dk)), rng.normal(size=(T, Hk, dk)) / np.sqrt(dk), rng.normal(size=(T, Hv, dv)),
            -rng.uniform(0, 2, size=(T, Hv)), rng.uniform(size=(T, Hv)), rng.normal(size=(N, Hv, dk, dv)))


def test_reference_is_the_dense_product_form():
    """S_T = sum over tokens of the dense factors e^g (I - beta k k^T) and writes beta k v^T."""
    rng = np.random.default_rng(1)
    q, k, v, g, b, s0 = _inputs(rng, 7, 2, 4, 5, 3, 1)
    out, S = gdr.forward(q, k, v, g, b, [0, 7], s0)
    for h in range(4):
        s = s0[0, h]
        for t in range(7):
            kk = k[t, h // 2][:, None]
            s = np.exp(g[t, h]) * (np.eye(5) - b[t, h] * kk @ kk.T) @ s + b[t, h] * kk @ v[t, h][None]
            np.testing.assert_allclose(out[t, h], s.T @ q[t, h // 2], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(S[0, h], s, rtol=1e-12, atol=1e-12)


def test_reference_gradients_are_its_differences():
    rng = np.random.default_rng(2)
    q, k, v, g, b, s0 = _inputs(rng, 6, 2, 4, 3, 4, 2)
    cu = [0, 2, 6]
    do, dS = rng.normal(size=v.shape), rng.normal(size=s0.shape)
    got = gdr.backward(q, k, v, g, b, cu, do, s0, dS)
    x = dict(q=q, k=k, v=v, g=g, beta=b, s0=s0)

    def loss(y):
        out, S = gdr.forward(y["q"], y["k"], y["v"], y["g"], y["beta"], cu, y["s0"])
        return (out * do).sum() + (S * dS).sum()

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("s0", "d_initial_state")):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in x[name].shape)
            d = 1e-5
            hi, lo = ({**x, name: x[name].copy()} for _ in range(2))
            hi[name][at] += d
            lo[name][at] -= d
            # central differences: d^2 / 6 of the third derivative and 2^-52 / d of the loss's rounding
            np.testing.assert_allclose(got[grad][at], (loss(hi) - loss(lo)) / (2 * d), rtol=1e-6, atol=1e-7)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_155_b200 import build

    build.build()
    from gated_delta_rule_155_b200 import kda

    return kda.library()


P = ctypes.c_void_p
A = P(0x100000)      # aligned, never dereferenced: every call below is refused on the host
MIS = P(0x100008)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 6


def test_forward_refusals(lib):
    def call(q=A, k=A, v=A, g=A, b=A, s0=None, i0=None, out=A, sT=None, i1=None, pages=0, cu=A, ws=A, wsb=1 << 50, N=3,
             T=100, Hk=2, Hv=4, dk=128, dv=128, io=0):
        return lib.kda_gdr_forward(q, k, v, g, b, s0, i0, out, sT, i1, pages, cu, ws, wsb, N, T, Hk, Hv, dk, dv, io, None)
    assert call(q=None) == INVALID and call(b=None) == INVALID
    assert call(out=None) == INVALID
    assert call(N=0) == INVALID and call(T=-1) == INVALID and call(Hk=0) == INVALID
    assert call(Hv=5) == INVALID                       # not a multiple of Hk
    assert call(io=9) == INVALID
    assert call(cu=None) == INVALID                    # 100 tokens are not 3 equal sequences
    assert call(i0=A, pages=4) == INVALID              # an index without its buffer
    assert call(sT=A, i1=A, pages=0) == INVALID        # an index into no pages
    assert call(dk=96) == UNSUPPORTED and call(dv=256) == UNSUPPORTED
    assert call(T=1 << 30) == UNSUPPORTED
    assert call(Hk=1 << 15, Hv=1 << 17) == UNSUPPORTED
    assert call(v=MIS) == MISALIGNED and call(s0=MIS) == MISALIGNED and call(cu=P(0x100002)) == MISALIGNED
    assert call(ws=None) == WORKSPACE and call(wsb=64) == WORKSPACE
    assert call(ws=P(0x100010)) == MISALIGNED          # 256-byte alignment


def test_backward_refusals(lib):
    def call(do=A, dg=A, s0=None, d0=None, ws=A, wsb=1 << 50, N=2, T=64, Hk=2, Hv=4, dk=128, dv=64, cu=None):
        return lib.kda_gdr_backward(A, A, A, A, A, s0, cu, do, None, A, A, A, dg, A, d0, ws, wsb, N, T, Hk, Hv, dk, dv, 1,
                                    None)
    assert call(do=None) == INVALID and call(dg=None) == INVALID
    assert call(T=63) == INVALID
    assert call(dk=32) == UNSUPPORTED
    assert call(d0=MIS) == MISALIGNED
    assert call(ws=None) == WORKSPACE and call(wsb=1) == WORKSPACE


def test_decode_refusals(lib):
    def call(state=A, index=None, pages=0, out=A, N=2, T=1, Hk=2, Hv=4, dk=128, dv=128, q=A):
        return lib.kda_gdr_decode(q, A, A, A, A, state, index, pages, out, N, T, Hk, Hv, dk, dv, 1, None)
    assert call(state=None) == INVALID and call(out=None) == INVALID
    assert call(T=0) == INVALID and call(N=0) == INVALID and call(Hv=3) == INVALID
    assert call(index=A, pages=0) == INVALID
    assert call(dk=80) == UNSUPPORTED
    assert call(N=1 << 16, T=1 << 16) == UNSUPPORTED
    assert call(q=MIS) == MISALIGNED and call(index=P(0x100001), pages=3) == MISALIGNED


def test_pages_refusals(lib):
    def fork(cache=A, nb=64, L=2, pages=5, refs=A, parents=A, children=A, n=3):
        return lib.kda_pages_fork(cache, nb, L, pages, refs, parents, children, n, None)
    assert fork(cache=None) == INVALID and fork(refs=None) == INVALID and fork(children=None) == INVALID
    assert fork(L=0) == INVALID and fork(pages=0) == INVALID and fork(n=-1) == INVALID and fork(nb=0) == INVALID
    assert fork(nb=24) == UNSUPPORTED                  # pages are moved 16 bytes at a time
    assert fork(cache=MIS) == MISALIGNED and fork(refs=P(0x100002)) == MISALIGNED
    assert fork(n=0, parents=None, children=None) == 0
    assert lib.kda_pages_copy(A, 64, 1, 4, None, A, 2, None) == INVALID
    assert lib.kda_pages_copy(A, 64, 1, 4, A, P(0x100001), 2, None) == MISALIGNED
    assert lib.kda_pages_free(None, 4, A, 2, None) == INVALID
    assert lib.kda_pages_free(A, 4, None, 2, None) == INVALID
    n = ctypes.c_size_t(0)
    assert lib.kda_pages_workspace_size(0, ctypes.byref(n)) == INVALID
    assert lib.kda_pages_workspace_size(7, ctypes.byref(n)) == 0 and 4 * 7 <= n.value <= 8 * 8

    def compact(table=A, n=3, ws=A, wsb=1 << 20):
        return lib.kda_pages_compact(A, 64, 1, 7, A, table, n, None, ws, wsb, None)
    assert compact(table=None) == INVALID
    assert compact(ws=None) == WORKSPACE and compact(wsb=8) == WORKSPACE


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    size = lambda *a: (lib.kda_gdr_workspace_size(*a, ctypes.byref(n)), n.value)  # noqa: E731
    assert size(3, 0, 2, 4, 128, 128, 1, 1) == (0, 0)
    st, f = size(3, 100, 2, 4, 128, 128, 1, 0)
    st2, b = size(3, 100, 2, 4, 128, 128, 1, 1)
    assert st == st2 == 0 and b > f >= 3 * 4 * 2 * 64 * 64 * 4
    assert lib.kda_gdr_workspace_size(3, 100, 2, 4, 128, 128, 1, 0, None) == INVALID
    assert size(3, 100, 3, 4, 128, 128, 1, 0)[0] == INVALID


def test_status_string_of_bad_pages(lib):
    assert b"page" in lib.kda_status_string(7)


def test_shared_buffers_are_refused(lib):
    """Written buffers that are inputs, or two of which are one."""
    other = [P(0x200000 + 0x10000 * i) for i in range(12)]

    def forward(out):
        return lib.kda_gdr_forward(*other[:5], None, None, out, None, None, 0, None, A, 1 << 50, 2, 64, 2, 4, 128, 128, 0, None)

    def backward(outs):
        return lib.kda_gdr_backward(*other[:5], None, None, other[5], None, *outs, None, A, 1 << 50, 2, 64, 2, 4, 128, 128, 1, None)

    def decode(out):
        return lib.kda_gdr_decode(*other[:5], A, None, 0, out, 2, 1, 2, 4, 128, 128, 1, None)
    for i in range(5):
        assert forward(other[i]) == INVALID and decode(other[i]) == INVALID
        for j in range(6):
            outs = other[6:11]
            outs[i] = other[j]
            assert backward(outs) == INVALID
        outs = other[6:11]
        outs[i] = other[6 + (i + 1) % 5]
        assert backward(outs) == INVALID
    for at in (0x300000, 0x300008, 0x2ffff8):           # the same ids, or some of them
        assert lib.kda_pages_fork(A, 64, 2, 5, A, P(0x300000), P(at), 3, None) == INVALID


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("io,dk", [(1, 128), (0, 64)])
def test_a_workspace_of_the_largest_call_does_for_all(lib, io, dk, backward):
    """The size never falls with the sequences, the tokens or the value heads."""
    n = ctypes.c_size_t(0)

    def size(N, T, Hv):
        assert lib.kda_gdr_workspace_size(N, T, 1, Hv, dk, dk, io, backward, ctypes.byref(n)) == 0
        return n.value
    Ns, Ts, Hs = [1, 2, 3, 4, 5, 8, 16, 100, 148, 149], [0, 1, 63, 64, 500, 1200, 4096, 8192, 65536], [1, 4, 8, 30, 32, 33, 96, 148, 160]
    for N in Ns:
        for T in Ts:
            for H in Hs:
                here = size(N, T, H)
                assert all(size(N + 1, T, H) >= here and size(N, T + d, H) >= here and size(N, T, H + d) >= here for d in (1, 64, 100))


def test_a_written_buffer_is_no_other_argument(lib):
    """Every pair of a written argument and another one, given as one pointer, is refused before any launch, but for
    the pairs that are documented (final_state over initial_state, d_initial_state over d_final_state)."""
    def pairs(call, written, read, allowed=()):
        at = {n: P(0x1000000 + 0x10000 * i) for i, n in enumerate((*written, *read))}
        for i, w in enumerate(written):
            for other in (*written[:i], *read):
                if (w, other) not in allowed:
                    assert call({**at, w: at[other]}) == INVALID, (w, other)
    io = ("q", "k", "v", "g", "beta")

    def forward(x):
        return lib.kda_gdr_forward(*(x[n] for n in io), x["s0"], x["i0"], x["out"], x["sT"], x["i1"], 4, x["cu"], x["ws"],
                                   1 << 50, 2, 64, 2, 4, 128, 128, 0, None)
    pairs(forward, ("out", "sT", "ws"), (*io, "s0", "i0", "i1", "cu"), {("sT", "s0")})

    def backward(dk, T, x):
        return lib.kda_gdr_backward(*(x[n] for n in io), x["s0"], x["cu"], x["do"], x["dT"], x["dq"], x["dk"], x["dv"], x["dg"],
                                    x["db"], x["d0"], x["ws"], 1 << 50, 2, T, 2, 4, dk, dk, 1, None)
    for dk in (64, 128):
        pairs(lambda x: backward(dk, 64, x), ("dq", "dk", "dv", "dg", "db", "d0", "ws"), (*io, "do", "s0", "dT", "cu"),
              {("d0", "dT")})
    pairs(lambda x: backward(128, 0, {n: x.get(n) for n in (*io, "do", "dT", "dq", "dk", "dv", "dg", "db", "ws", *x)}),
          ("d0",), ("s0", "cu"))                       # no tokens: the states are still read and written

    def decode(x):
        return lib.kda_gdr_decode(*(x[n] for n in io), x["state"], x["index"], 4, x["out"], 2, 1, 2, 4, 128, 128, 1, None)
    pairs(decode, ("out", "state"), (*io, "index"))

    def fork(x):
        return lib.kda_pages_fork(x["cache"], 64, 2, 5, x["refs"], x["parents"], x["children"], 3, None)
    pairs(fork, ("cache", "refs", "children"), ("parents",))

    def copy(x):
        return lib.kda_pages_copy(x["cache"], 64, 2, 5, x["src"], x["dst"], 3, None)
    pairs(copy, ("cache",), ("src", "dst"))
    pairs(lambda x: lib.kda_pages_free(x["refs"], 5, x["ids"], 3, None), ("refs",), ("ids",))

    def compact(x):
        return lib.kda_pages_compact(x["cache"], 64, 2, 5, x["refs"], x["table"], 3, x["live"], x["ws"], 1 << 20, None)
    pairs(compact, ("cache", "refs", "table", "live", "ws"), ())
