"""The head-gated delta rule head by head: heads of very different sizes in one call, each against its own largest value.

Tolerances, as parts of the largest |reference| of the same sequence and head (states) or head (the rest), with rounding
errors taken as independent, as they are where signs are random:
  * fp32 products are split tf32: a factor is off by at most 2^-23, the lo x lo term left out is at most 2^-24, and eight
    products at a time are added with one rounding (2^-24).  The three are alike, so a product is off by about
    sqrt(3) 2^-23 = 2^-22 of the rms of its results; a decay by __expf adds 2^-22 to its terms.  Four products in a row a
    chunk, and twelve chunks whose errors add at worst (the recurrence does not enlarge them): sqrt(48) 2^-22 = 2^-19.2 of
    the rms.  The largest of 10^5 such errors is 4.5 of their rms, the largest value of a head at least 3 of its own:
    2^-18.6.  Bound: 2^-17 for outputs and states.  A gradient is a sum of up to four such terms, with up to eight products
    in a row: 2^-16; dg is a sum over the chunk of row sums less column sums, each as large as the largest: 2^-15.
  * bf16 at dk = dv = 128: a hi + lo pair is off by at most 2^-18, and the lo x lo term left out, where both factors are
    pairs, is at most 2^-18: sqrt(2) 2^-18 / sqrt(3) = 2^-18.3 a product, three in a row a chunk, twelve chunks: 2^-15.7
    of the rms at worst, 2^-15.1 of the largest value.  Bound: 2^-14 for states, outputs and dv (2^-8 |e| on top where
    stored in bf16).  The gradients of q, k, g and beta read states and corrections rounded once to bf16: 2^-8 of the
    2-norm at most (each term by four roundings of 2^-9 / sqrt(3), independent) beside 2^-9 by their own.  The terms of dg
    that a chunk's tokens share have one error for all of them, and a head has few chunks: twice that.  Bound: 2^-7 of the
    2-norm of a key head's dq and dk and of a head's dbeta, 2^-6 of a head's dg.
  * decode: sums of 128 products, each rounded once, a token: 2^-24 sqrt(128) = 2^-20.5 of the rms at worst; bound 2^-19.
"""
import numpy as np
import pytest
import torch

from oracle import gdr

from test_gdr_gpu import DT, NAMES, cu_of, f64, make, tc, to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_155_b200 import build

    build.build()
    from gated_delta_rule_155_b200 import kda as k

    return k


def heads_of_all_sizes(T, Hk, Hv, dk, dv, io, seed, N):
    """Values, states and their gradients of head h times 2^(5 (h mod 4) - 8); every third head forgets quickly."""
    d = make(T, Hk, Hv, dk, dv, io, seed, N)
    size = 2.0 ** (5.0 * (torch.arange(Hv) % 4) - 8.0)
    for n in ("v", "dO"):
        d[n] = (d[n].float() * size[:, None]).to(DT[io])
    for n in ("s0", "dS"):
        d[n] = d[n] * size[:, None, None]
    d["g"] = (d["g"].float() * torch.where(torch.arange(Hv) % 3 == 0, 20.0, 1.0)).to(DT[io])
    return d


def near_by_head(got, ref, axes, part, stored, what):
    """`axes`: those that one largest value is taken over."""
    got, ref = f64(got), np.asarray(ref)
    assert np.isfinite(got).all(), what
    bound = part * np.abs(ref).max(axis=axes, keepdims=True) + (2.0 ** -8 * np.abs(ref) if stored else 0.0) + 1e-30
    off = np.abs(got - ref) / bound
    assert (off <= 1.0).all(), f"{what}: {off.max():.2f} of the bound"


@pytest.mark.parametrize("io,dk,dv", [("f32", 64, 64), ("f32", 64, 128), ("f32", 128, 64), ("f32", 128, 128),
                                      ("bf16", 64, 64), ("bf16", 64, 128), ("bf16", 128, 64), ("bf16", 128, 128)])
@pytest.mark.parametrize("lens,Hk,Hv", [([130, 1, 63], 2, 4), ([700, 3], 4, 4), ([64, 257], 1, 6)])
def test_every_head_keeps_its_bits(kda, io, dk, dv, lens, Hk, Hv):
    N, cu, exact, stored = len(lens), cu_of(lens), not tc(io, dk, dv), io == "bf16"
    d = heads_of_all_sizes(cu[-1], Hk, Hv, dk, dv, io, 130, N)
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    sT, d0 = torch.empty_like(d["s0"], device="cuda"), torch.empty_like(d["s0"], device="cuda")
    out, _ = kda.kda_gdr_forward(*to(d, *NAMES), cug, d["s0"].cuda(), final_state=sT)
    gr = kda.kda_gdr_backward(*to(d, *NAMES, "dO"), cug, d["s0"].cuda(), d["dS"].cuda(), d_initial_state=d0)
    kda.kda_check_device_error()
    a = [f64(d[n]) for n in NAMES]
    ro, rs = gdr.forward(*a, cu, f64(d["s0"]))
    ref = gdr.backward(*a, cu, f64(d["dO"]), f64(d["s0"]), f64(d["dS"]))
    part = 2.0 ** -17 if exact else 2.0 ** -14
    near_by_head(out, ro, (0, 2), part, stored, "out")
    near_by_head(sT, rs, (2, 3), part, False, "final state")
    part = 2.0 ** -16 if exact else 2.0 ** -14
    near_by_head(gr["dv"], ref["dv"], (0, 2), part, stored, "dv")
    near_by_head(d0, ref["d_initial_state"], (2, 3), part, False, "d_initial_state")
    if exact:
        near_by_head(gr["dq"], ref["dq"], (0, 2), part, stored, "dq")
        near_by_head(gr["dk"], ref["dk"], (0, 2), part, stored, "dk")
        near_by_head(gr["dbeta"], ref["dbeta"], (0,), part, stored, "dbeta")
        near_by_head(gr["dg"], ref["dg"], (0,), 2.0 ** -15, stored, "dg")
    else:
        for n, axes, part in (("dq", (0, 2), 2.0 ** -7), ("dk", (0, 2), 2.0 ** -7), ("dbeta", (0,), 2.0 ** -7), ("dg", (0,), 2.0 ** -6)):
            off, norm = (np.sqrt((x * x).sum(axis=axes)) for x in (f64(gr[n]) - ref[n], ref[n]))
            assert (off <= part * norm).all(), f"{n}: {(off / norm).max() / part:.2f} of the bound"


@pytest.mark.parametrize("io,dk,dv", [("f32", 64, 64), ("f32", 128, 128), ("bf16", 64, 128), ("bf16", 128, 128)])
def test_decode_keeps_every_heads_bits(kda, io, dk, dv):
    N, T, Hk, Hv = 3, 4, 2, 4
    d = heads_of_all_sizes(N * T, Hk, Hv, dk, dv, io, 131, N)
    x, state = [t.view(N, T, *t.shape[1:]) for t in to(d, *NAMES)], d["s0"].cuda()
    out = kda.kda_gdr_decode(*x, state)
    kda.kda_check_device_error()
    ro, rs = gdr.decode(*(f64(t) for t in x), f64(d["s0"]))
    near_by_head(out, ro, (0, 1, 3), 2.0 ** -19, io == "bf16", "out")
    near_by_head(state, rs, (2, 3), 2.0 ** -19, False, "state")
