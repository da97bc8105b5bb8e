"""The selective scan value by value against the recurrence in 64 bits: sums whose terms
cancel, gates and steps far from 0, states of every memory.  In what follows u = 2^-24, one
rounding to fp32; the hardware's exponential is off by 4 u at most, its reciprocal by 2 u."""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from selscan_ref import selscan, sigmoid
from test_gpu_selscan import DT, args, dev, f64, make, options, ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def near(got, want, slack):
    """Every value within `slack` of the reference."""
    off = np.abs(f64(got) - want) - slack
    assert (off <= 0).all(), (float(off.max()), np.unravel_index(off.argmax(), off.shape), float((off > 0).mean()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["states", "skip"])
@pytest.mark.parametrize("N", [8, 16, 48])
def test_gate_gradient_where_states_cancel(dtype, kind, N):
    """dz of single tokens, dout (C.h + D x) silu'(z), where the states' terms cancel one another
    but for the 64th part of one, or D x but for 2^-9 of it.  A term has 3 roundings (delta x,
    times B, times C), their sum as many as N / 8 + 5, D x one: 16 u of the terms' absolute sum.  |z| is 4
    at most, so that silu' is off by 2^-18 of its two terms."""
    n, D = 64, 24
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x, dout, z = rnd(n, D).to(DT[dtype]), rnd(n, D).to(DT[dtype]), rnd(n, D).clamp(-4, 4).to(DT[dtype])
    dt = (0.02 + rnd(1, D).abs()).expand(n, D).to(DT[dtype]).contiguous()
    A, skip = -torch.rand(D, N, generator=g), rnd(D)
    if kind == "states":
        half = rnd(n, N // 2).to(DT[dtype])
        k = torch.randint(33, 64, (n, N // 2), generator=g).float() / 64
        other = -k
        other[:, 0] += 1 / 64
        B, C = torch.cat([half, half], 1), torch.cat([k, other], 1).to(DT[dtype])
        skip = torch.zeros(D)
    else:
        B, C = (rnd(1, N).expand(n, N).to(DT[dtype]).contiguous() for _ in range(2))
        skip = (-dt[0].double() * (B[0].double() * C[0].double()).sum() * (1 - 2.0 ** -9)).float()
    ops = [t.cuda() for t in (x, dt, A, B[:, None], C[:, None])]
    kw = dict(D=skip.cuda(), z=z.cuda(), nseqs=n)
    _, _, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    got = ssd.selscan_bwd(*ops, dout.cuda(), st, **kw)["dz"]
    x, dt, B, C, z, dout, skip = (f64(t) for t in (x, dt, B, C, z, dout, skip))
    terms = (dt * x)[:, :, None] * (B * C)[:, None]
    y, size = terms.sum(2) + skip * x, np.abs(terms).sum(2) + np.abs(skip * x)
    s = sigmoid(z)
    slope, parts = s * (1 + z * (1 - s)), s * (1 + np.abs(z) * (1 - s))
    want = dout * y * slope
    near(got, want, HALF[dtype] * np.abs(want) + 16 * U * np.abs(dout * slope) * size + 2.0 ** -18 * np.abs(dout * y) * parts)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 16, 40])
def test_every_value(dtype, N):
    """y, dx, ddt, dz, dB and dC value by value: half a step of their type, and 2e-5 of the terms'
    absolute sum (decays of a memory of 50 tokens, each off by 4 u; delta by 8 u)."""
    lens = [70, 1, 33]
    x = make(dtype, lens, 2, 24, N, 1, True, False, seed=22)
    d = dev(x)
    y, _, st = ssd.selscan_fwd(*args(d), return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, **options(d))
    want_y, _, want = ref(x, lens, grads=True)
    # the same sums of the terms' absolute values, the gate taken into dout
    z, dout = f64(x["z"]), f64(x["dout"])
    s = sigmoid(z)
    dt, bias, X, Dk = f64(x["dt"]), f64(x["bias"]), np.abs(f64(x["x"])), np.abs(f64(x["D"]))
    gy = np.abs(dout * z * s)
    size_y, _, size = selscan(X, dt, f64(x["A"]), np.abs(f64(x["B"])), np.abs(f64(x["C"])), lens, Dk, None, bias, True, None, gy)
    delta, slope = np.logaddexp(dt + bias, 0), sigmoid(dt + bias)
    u = (size["dx"] - Dk * gy) / delta
    sizes = {"dx": size["dx"], "dB": size["dB"], "dC": size["dC"], "ddt": (2 * X * u) * slope - size["ddt"],   # x u and |A| w, not x u - |A| w
             "dz": np.abs(dout) * size_y * s * (1 + np.abs(z) * (1 - s))}
    inside = slice(0, sum(lens))
    near(y[inside], want_y[inside], (HALF[dtype] * np.abs(want_y) + 2e-5 * size_y * np.abs(z * s))[inside])
    for k, v in sizes.items():
        near(g[k][inside], want[k][inside], (HALF[dtype] * np.abs(want[k]) + 2e-5 * v)[inside])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 48])
def test_sums_over_states_lean_to_no_side(dtype, N):
    """ddt_bias of one token, where every term is positive: x dout sum B C.  Its dozen roundings to
    nearest are off by 0.6 u each, 2 u together, to no side: 0.05 u of 2048 channels' mean, and 0.6 u (3.6e-8)
    is allowed.  Terms cut to 22 bits would be off by 1.2 u on average, to one."""
    D = 2048
    g = torch.Generator().manual_seed(23)
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g)).to(DT[dtype])
    x, dt, dout, B, C = pos(1, D), pos(1, D), pos(1, D), pos(1, 1, N), pos(1, 1, N)
    A = -pos(D, N).float()
    ops = [t.cuda() for t in (x, dt, A, B, C)]
    kw = dict(dt_bias=torch.zeros(D, device="cuda"))
    _, _, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    got = f64(ssd.selscan_bwd(*ops, dout.cuda(), st, **kw)["ddt_bias"])
    want = f64(x[0]) * f64(dout[0]) * (f64(B) * f64(C)).sum()
    lean = ((got - want) / want).mean()
    assert abs(lean) < 3.6e-8, lean


@pytest.mark.parametrize("extra", [0, 1])
@pytest.mark.parametrize("cut", [True, False])
@pytest.mark.parametrize("rate", [1e-3, 1e-2, 0.04, 0.1, 1.0])
def test_states_of_every_memory_lean_to_no_side(rate, cut, extra):
    """2400 (2401) tokens whose states decay by `rate` a token on average: final states, and the
    initial state's gradient, against 64 bits.  The fast exponential is low by 5.5e-9 on average
    near 1 and by 2.4e-8 from 0.01 on, and a state of inputs of either sign remembers
    exp(-2 rate) / (1 - exp(-2 rate)) tokens: what these lose together would be missing.  A third of that may be,
    or 1e-7.  (Roundings: 0.7 u a token, of 500 tokens 16 u, of 1024 states' mean 0.5 u, 3e-8.)"""
    lost = (5.5e-9 if rate < 2e-3 else 2.4e-8) * np.exp(-2 * rate) / (1 - np.exp(-2 * rate))
    T, D, N = 2400 + extra, 64, 16
    g = torch.Generator().manual_seed(24)
    rnd = lambda *s: torch.randn(*s, generator=g)
    uni = lambda *s: torch.rand(*s, generator=g)
    x, B, C, dout = rnd(T, D), rnd(T, 1, N), rnd(T, 1, N), rnd(T, D)
    dt, A = rate * (0.5 + uni(T, D)), -(0.8 + 0.4 * uni(D, N))
    ops = [t.cuda() for t in (x, dt, A, B, C)]
    # (a bound on the lengths that is too low only guides the cut: whole sequences)
    kw = dict(cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device="cuda"), max_seqlen=0 if cut else 1)
    _, fin, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    got = ssd.selscan_bwd(*ops, dout.cuda(), st, return_dinit=True, **kw)["dinit_state"]
    _, wfin, want = selscan(*(f64(t) for t in (x, dt, A, B, C)), [T], softplus=False, dout=f64(dout))
    for a, b in ((fin, wfin), (got, want["dinit_state"])):
        lean = ((f64(a) - b) * b).sum() / (b * b).sum()
        assert abs(lean) < max(lost / 3, 1e-7), lean


@pytest.mark.parametrize("rate", [1e-2, 0.02, 0.04, 0.1])
def test_states_lean_to_no_side_between_corrections(rate):
    """The same of 2408 tokens: the state gets back what 16 tokens lose (16 * 2.4e-8 at most) behind each 16th, and
    should be as much too large there as too small before it, so nearly right behind an 8th: 1e-7 as
    above and two tokens' loss."""
    T, D, N = 2408, 64, 16
    g = torch.Generator().manual_seed(28)
    rnd = lambda *s: torch.randn(*s, generator=g)
    uni = lambda *s: torch.rand(*s, generator=g)
    x, B, dt, A = rnd(T, D), rnd(T, 1, N), rate * (0.5 + uni(T, D)), -(0.8 + 0.4 * uni(D, N))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, fin = ssd.selscan_fwd(*(t.cuda() for t in (x, dt, A, B, B)), cu_seqlens=cu, max_seqlen=1)
    _, want = selscan(*(f64(t) for t in (x, dt, A, B, B)), [T], softplus=False)
    lean = ((f64(fin) - want) * want).sum() / (want * want).sum()
    assert abs(lean) < 1.5e-7, lean


def far(dtype):
    """Numbers from -200 to 200, of the given type, dense where exponentials still count."""
    v = torch.cat([torch.linspace(-200, 200, 353), torch.linspace(-90, -10, 511), torch.linspace(-10, 10, 160)])
    return v.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_far_from_zero(dtype):
    """delta = softplus(v) and its derivative for v from -200 to 200, of single tokens.  The exponential 5 u
    (v log2(e) with its remainder, 4 u and a rounding), the quotient 2 + 1 + 1 u, the polynomial
    and its sum 3 u, times x and B 2 u: 16 u allowed; the derivative 5 + 1 + 2 + 1 u and 4 products.  What is
    below 2^-126 is flushed."""
    v = far(dtype)
    D, N = len(v), 4
    g = torch.Generator().manual_seed(25)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    x, B, C, dout = rnd(1, D), rnd(1, 1, N), rnd(1, 1, N), rnd(1, D)
    A = torch.zeros(D, N)
    ops = [t.cuda() for t in (x, v[None], A, B, C)]
    kw = dict(dt_softplus=True, dt_bias=torch.zeros(D, device="cuda"))
    _, fin, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    cache = torch.zeros(1, D, N, device="cuda")
    ssd.selscan_step(*ops, cache, **kw)
    X, V, Bf, Cf = f64(x[0])[:, None], f64(v), f64(B[0]), f64(C[0])
    want = np.logaddexp(V, 0)[:, None] * X * Bf
    slack = 16 * U * np.abs(want) + 2.0 ** -125 * np.abs(X * Bf)
    near(fin[0], want, slack)
    near(cache[0], want, slack)
    got = ssd.selscan_bwd(*ops, dout.cuda(), st, **kw)
    terms = f64(x[0]) * f64(dout[0]) * (Bf * Cf).sum()
    size = np.abs(f64(x[0]) * f64(dout[0])) * np.abs(Bf * Cf).sum()
    slope = np.exp(-np.logaddexp(-V, 0))
    near(got["ddt_bias"], terms * slope, 16 * U * size * slope + 2.0 ** -125 * size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_far_from_zero(dtype):
    """silu(z) and its derivative for z from -200 to 200, of single tokens with D x alone.  fp32: the
    exponential 5 u, the quotient 1 + 2 u, two products: 12 u allowed; the derivative s + z s (1 - s) 12 u of both
    terms, and where s is nearly 1, z times the 6 u that it is off.  bf16: without the exponential's remainder,
    which takes 1.2 u for each of |z|."""
    z = far(dtype)
    D, N = len(z), 4
    g = torch.Generator().manual_seed(26)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    x, dout, B = rnd(1, D), rnd(1, D), torch.zeros(1, 1, N, dtype=DT[dtype])
    ops = [t.cuda() for t in (x, rnd(1, D), -torch.ones(D, N), B, B)]
    kw = dict(D=torch.ones(D).cuda(), z=z[None].cuda())
    y, _, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    cache = torch.zeros(1, D, N, device="cuda")
    y1 = ssd.selscan_step(*ops, cache, **kw)
    got = ssd.selscan_bwd(*ops, dout.cuda(), st, **kw)
    X, Z, G = f64(x[0]), f64(z), f64(dout[0])
    s = np.exp(-np.logaddexp(-Z, 0))
    more = 12 + (0 if dtype == "f32" else 1.2 * np.abs(Z))
    flush = 2.0 ** -125 * np.abs(Z)
    want = X * Z * s
    for v in (y, y1):
        near(v[0], want, (HALF[dtype] + more * U) * np.abs(want) + flush * np.abs(X))
    want = G * X * s * (1 + Z * (1 - s))
    size = np.abs(G * X) * ((more * s * (1 + np.abs(Z) * (1 - s)) + 6 * np.abs(Z) * s) * U + flush)
    near(got["dz"][0], want, HALF[dtype] * np.abs(want) + size)
    want = G * Z * s                                   # dx = D gy
    near(got["dx"][0], want, (HALF[dtype] + more * U) * np.abs(want) + flush * np.abs(G))
