"""The block norms and their gradient against the formulas in 64 bits.

Tolerances, as 2-norm of the difference over 2-norm of the reference: a bf16
result is rounded once, by at most the unit roundoff of its 8-bit significand,
2^-8 of each value; an fp32 one is a sum over at most a few thousand columns or
rows held in fp32, and a handful of operations on it: 5e-6.
"""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from linattn_ref import block_norm, off

pytestmark = pytest.mark.gpu
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 5e-6}
BF, F = torch.bfloat16, torch.float32

# dtype, rdtype, tokens, width, groups, gate, weights given
CASES = [
    (BF, BF, 1, 8, 1, "silu", True),
    (BF, F, 3, 512, 8, "sigmoid", True),       # a warp for each row, groups of 64
    (F, F, 5, 264, 11, None, False),           # groups of 24: neither one nor a power of two
    (BF, BF, 700, 1024, 1, "silu", True),
    (F, F, 33, 1544, 1, "sigmoid", True),      # odd number of vectors
    (BF, F, 9, 5120, 80, "silu", True),
    (BF, BF, 4, 5120, 5, "silu", False),       # groups wider than a warp's vectors
    (F, F, 3, 16384, 2, "silu", True),         # the widest
    (BF, BF, 2500, 64, 1, "sigmoid", True),    # more rows than CTAs
]


def make(dt, rdt, T, D, gate, weights, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x = dict(r=rnd(T, D).to(rdt), y=(3 * rnd(T, D)).to(dt), z=rnd(T, D).to(dt) if gate else None,
             w_pre=1 + 0.3 * rnd(D), w_post=1 + 0.3 * rnd(D) if weights else None,
             alpha=0.5 * rnd(D) if weights else None, dr_out=rnd(T, D).to(rdt), dn=rnd(T, D).to(dt))
    return x, {k: None if t is None else t.cuda() for k, t in x.items()}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def fwd_args(x):
    return dict(z=x["z"], w_post=x["w_post"], alpha=x["alpha"])


@pytest.mark.parametrize("dt,rdt,T,D,groups,gate,weights", CASES)
def test_forward_and_gradient(dt, rdt, T, D, groups, gate, weights):
    x, d = make(dt, rdt, T, D, gate, weights)
    kw = dict(gate=gate, ngroups=groups, eps=1e-5)
    ro, n, rstd = ssd.block_norm_fwd(d["r"], d["y"], d["w_pre"], return_rstd=True, **fwd_args(d), **kw)
    g = ssd.block_norm_bwd(d["r"], d["y"], d["w_pre"], d["dr_out"], d["dn"], rstd, **fwd_args(d), **kw)
    torch.cuda.synchronize()
    w = {k: f64(v) for k, v in x.items()}
    rr, rn, rg = block_norm(w["r"], w["y"], w["w_pre"], **fwd_args(w), **kw, dr_out=w["dr_out"], dn=w["dn"])
    assert off(f64(ro), rr) < TOL[rdt] and off(f64(n), rn) < TOL[dt]
    for name, tol in (("dr", TOL[rdt]), ("dy", TOL[dt]), ("dz", TOL[dt]), ("dw_pre", TOL[F]),
                      ("dw_post", TOL[F]), ("dalpha", TOL[F])):
        if g[name] is None:
            assert (name == "dz" and gate is None) or (name in ("dw_post", "dalpha") and not weights)
            continue
        assert off(f64(g[name]), rg[name]) < tol, name
    # without the factors, in place, and again: the same bits
    r2 = d["r"].clone()
    ro2, n2 = ssd.block_norm_fwd(r2, d["y"], d["w_pre"], r_out=r2, **fwd_args(d), **kw)
    g2 = ssd.block_norm_bwd(d["r"], d["y"], d["w_pre"], d["dr_out"], d["dn"], rstd, **fwd_args(d), **kw)
    assert ro2 is r2 and torch.equal(ro2, ro) and torch.equal(n2, n)
    assert all(a is b or torch.equal(a, b) for a, b in zip(g.values(), g2.values()))


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_gradient_against_differences(gate):
    """Central differences of the fp32 forward along random directions: their error
    is the step squared times third derivatives (1e-4 of the gradient times the
    direction) and 1e-7 of the result over the step."""
    T, D, groups, h = 6, 96, 3, 1e-2
    _, d = make(F, F, T, D, gate, True, seed=1)
    kw = dict(gate=gate, ngroups=groups)
    names = ["r", "y", "w_pre", "z", "w_post", "alpha"]

    def f(p):
        ro, n = ssd.block_norm_fwd(p["r"], p["y"], p["w_pre"], **fwd_args(p), **kw)
        return (ro.double() * d["dr_out"]).sum() + (n.double() * d["dn"]).sum()

    _, _, rstd = ssd.block_norm_fwd(d["r"], d["y"], d["w_pre"], return_rstd=True, **fwd_args(d), **kw)
    g = ssd.block_norm_bwd(d["r"], d["y"], d["w_pre"], d["dr_out"], d["dn"], rstd, **fwd_args(d), **kw)
    for i, name in enumerate(names):
        torch.manual_seed(i)
        v = torch.randn_like(d[name])
        diff = (f({**d, name: d[name] + h * v}) - f({**d, name: d[name] - h * v})) / (2 * h)
        want = (g["d" + name].double() * v).sum()
        assert abs(diff - want) < 2e-3 * g["d" + name].double().norm() * v.double().norm(), name


def test_strides_streams_and_extremes():
    T, D = 40, 256
    _, d = make(BF, BF, T, D, "silu", True, seed=2)
    wide = torch.cat([d["y"], d["z"], d["y"]], 1)
    kw = dict(gate="silu", ngroups=4)
    want = ssd.block_norm_fwd(d["r"], d["y"], d["w_pre"], **fwd_args(d), **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ssd.block_norm_fwd(d["r"], wide[:, 2 * D:], d["w_pre"], z=wide[:, D:2 * D],
                                 w_post=d["w_post"], alpha=d["alpha"], **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a closed gate and a block of zeros leave the residual; NaN stays in its row
    z = torch.full_like(d["z"], -1e4)
    ro, _ = ssd.block_norm_fwd(d["r"], d["y"], d["w_pre"], z=z, **kw)
    assert torch.equal(ro, d["r"])
    ro, _ = ssd.block_norm_fwd(d["r"], torch.zeros_like(d["y"]), d["w_pre"], z=d["z"], **kw)
    assert torch.equal(ro, d["r"])
    y = d["y"].clone()
    y[7] = float("nan")
    ro, n = ssd.block_norm_fwd(d["r"], y, d["w_pre"], **{**fwd_args(d), "z": d["z"]}, **kw)
    keep = [t for t in range(T) if t != 7]
    assert torch.equal(ro[keep], want[0][keep]) and torch.equal(n[keep], want[1][keep])
    assert torch.isnan(n[7].float()).all()


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    ro, n, rstd = ssd.block_norm_fwd(e, e, w, return_rstd=True)
    g = ssd.block_norm_bwd(e, e, w, e, e, rstd, alpha=w)
    assert ro.numel() == 0 and torch.all(g["dw_pre"] == 0) and torch.all(g["dalpha"] == 0)


def test_binding_refuses():
    x, d = make(BF, BF, 4, 64, "silu", True)
    f = lambda **kw: ssd.block_norm_fwd(**{**dict(r=d["r"], y=d["y"], w_pre=d["w_pre"], z=d["z"], gate="silu"), **kw})
    f()
    for bad, err in ((dict(gate="relu"), ValueError), (dict(z=None), ValueError),
                     (dict(z=d["z"].float()), TypeError), (dict(r=d["r"][:3]), ValueError),
                     (dict(w_pre=d["w_pre"].bfloat16()), TypeError), (dict(alpha=d["w_pre"][:32]), ValueError),
                     (dict(y=d["y"].t().contiguous().t()), ValueError), (dict(ngroups=16), ssd.SSDError),
                     (dict(ngroups=3), ssd.SSDError), (dict(eps=-1.0), ssd.SSDError),
                     (dict(out=d["y"]), ssd.SSDError)):
        with pytest.raises(err):
            f(**bad)
