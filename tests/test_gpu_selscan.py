"""The selective scan: prompts, gradients and single tokens against the recurrence in 64 bits.

Tolerances, as 2-norm of the difference over 2-norm of the reference.  fp32: a decay is an
approximated exponential, off by 2^-22 of it at most; delta is at least 0.02 and A at most
-1 here, so that a state remembers 50 tokens and is off by 50 * 2^-22 at most, and delta
itself by 2^-21 (an exponential, a quotient, a polynomial): 2e-5 with the sums' own
roundings.  bf16 outputs are rounded once from fp32: 2^-8 of each value at most, and 2e-5.
"""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from selscan_ref import off, selscan

pytestmark = pytest.mark.gpu
TOL = {"bf16": 2.0 ** -8 + 2e-5, "f32": 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# dtype, lengths, rows behind them, channels, states, groups, gate, initial state
CASES = [
    ("bf16", [1], 0, 8, 16, 1, True, False),
    ("f32", [1, 2, 7, 8, 9, 0, 31, 32, 33, 64, 65], 3, 40, 16, 1, True, True),
    ("bf16", [100, 0, 0, 41], 0, 96, 16, 3, True, True),
    ("f32", [130, 5], 2, 72, 10, 3, False, True),          # a number of states that is no power of two
    ("bf16", [70, 3], 0, 136, 8, 1, True, False),
    ("f32", [33, 90], 0, 16, 4, 2, True, True),
    ("f32", [40], 0, 24, 1, 1, True, True),
    ("f32", [40, 35], 0, 24, 7, 1, False, True),
    ("bf16", [75, 20], 1, 80, 32, 1, True, True),
    ("f32", [50, 35], 0, 24, 27, 1, True, True),
    ("f32", [75, 20], 1, 48, 64, 2, True, True),
    ("bf16", [40, 35], 0, 40, 63, 1, True, True),
]


def make(dtype, lens, pad, D, N, G, gate, state, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    T, n = sum(lens) + pad, len(lens)
    x = dict(x=rnd(T, D), dt=0.5 * rnd(T, D), B=rnd(T, G, N), C=rnd(T, G, N), z=rnd(T, D) if gate else None, dout=rnd(T, D))
    x = {k: None if v is None else v.to(DT[dtype]) for k, v in x.items()}
    x["A"] = -torch.arange(1, N + 1) * torch.exp(0.1 * rnd(D, N).abs())
    x["D"], x["bias"] = rnd(D), -1.0 + 0.3 * rnd(D)
    x["h0"] = rnd(n, D, N) if state else None
    x["dfin"] = rnd(n, D, N) if state else None
    x["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return x


def dev(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def ref(x, lens, grads=False, softplus=True):
    return selscan(f64(x["x"]), f64(x["dt"]), f64(x["A"]), f64(x["B"]), f64(x["C"]), lens, f64(x["D"]), f64(x["z"]),
                   f64(x["bias"]), softplus, f64(x["h0"]), f64(x["dout"]) if grads else None, f64(x["dfin"]))


def args(d):
    return (d["x"], d["dt"], d["A"], d["B"], d["C"])


def options(d):
    return dict(D=d["D"], z=d["z"], dt_bias=d["bias"], dt_softplus=True, cu_seqlens=d["cu"])


def sliced(d):
    """The same operands as columns of wider tensors, B and C at an odd offset."""
    T, D = d["x"].shape
    G, N = d["B"].shape[1:]
    wide = lambda t: torch.cat([torch.randn_like(t), t], 1)[:, D:]
    bc = torch.zeros(T, 3 + 2 * G * N, device="cuda", dtype=d["x"].dtype)
    bc[:, 3:3 + G * N], bc[:, 3 + G * N:] = d["B"].reshape(T, -1), d["C"].reshape(T, -1)
    s = dict(d, x=wide(d["x"]), dt=wide(d["dt"]), z=None if d["z"] is None else wide(d["z"]))
    s["B"], s["C"] = bc[:, 3:3 + G * N].view(T, G, N), bc[:, 3 + G * N:].view(T, G, N)
    return s


def check(dtype, lens, y, fin, g, want, state):
    at = 0
    for s, L in enumerate(lens):   # each sequence by itself: a short one must not hide
        rows = slice(at, at + L)
        assert off(f64(y[rows]), want[0][rows]) < TOL[dtype], (s, L)
        assert off(f64(fin[s]), want[1][s]) < TOL["f32"], (s, L)
        if g is not None:
            for k in ("dx", "ddt", "dz", "dB", "dC"):
                if g[k] is not None:
                    assert off(f64(g[k][rows]), want[2][k][rows]) < TOL[dtype], (k, s, L)
            if state:
                assert off(f64(g["dinit_state"][s]), want[2]["dinit_state"][s]) < TOL["f32"], (s, L)
        at += L
    assert not y[at:].any()
    if g is not None:
        for k in ("dx", "ddt", "dz", "dB", "dC"):
            assert g[k] is None or not g[k][at:].any(), k
        for k in ("dA", "dD", "ddt_bias"):
            assert off(f64(g[k]), want[2][k]) < TOL["f32"], k


@pytest.mark.parametrize("dtype,lens,pad,D,N,G,gate,state", CASES)
def test_prompt_and_gradient(dtype, lens, pad, D, N, G, gate, state):
    x = make(dtype, lens, pad, D, N, G, gate, state)
    want = ref(x, lens, grads=True)
    d = dev(x)
    for v in (d, sliced(d)):
        for longest in (0, max(lens)):
            y, fin, st = ssd.selscan_fwd(*args(v), init_state=v["h0"], max_seqlen=longest, return_states=True, **options(v))
            g = ssd.selscan_bwd(*args(v), v["dout"], st, dfinal_state=v["dfin"], return_dinit=state, max_seqlen=longest, **options(v))
            torch.cuda.synchronize()
            check(dtype, lens, y, fin, g, want, state)
            assert (g["dz"] is None) == (not gate) and (g["dinit_state"] is None) == (not state)


@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("f32", 16), ("f32", 6), ("bf16", 48)])
def test_long_sequences_cut_into_ranges(dtype, N):
    """Few channels and many tokens: sequences are cut, and what is remembered crosses the cuts."""
    lens = [1500, 3, 900, 0, 257]
    x = make(dtype, lens, 1, 16, N, 1, True, True, seed=2)
    d = dev(x)
    y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
    torch.cuda.synchronize()
    check(dtype, lens, y, fin, g, ref(x, lens, grads=True), True)


def test_long_memories_cross_the_cuts():
    """Decays near 1 over a whole cut sequence: 2000 tokens, each decay off by 2^-22 at most."""
    lens = [2000]
    x = make("f32", lens, 0, 8, 4, 1, False, True, seed=4)
    x["A"] = torch.full((8, 4), -1e-3)
    d = dev(x)
    y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
    want = ref(x, lens, grads=True)
    tol = 2000 * 2.0 ** -22 + 2e-5
    assert off(f64(y), want[0]) < tol and off(f64(fin), want[1]) < tol
    for k in ("dx", "ddt", "dA", "dB", "dC", "dinit_state"):
        assert off(f64(g[k]), want[2][k]) < tol, k


def test_gradient_against_differences():
    """fp32: a central difference of step 1e-2 along a random direction is the gradient's product
    with it up to the third derivative's (1e-2)^2 / 6 share and the forward's own error over the
    step, both below 2e-3 of the norms' product (A's own step is that share of each entry)."""
    lens = [40, 3, 37]
    d = dev(make("f32", lens, 0, 16, 6, 2, True, True, seed=3))
    names = ["x", "dt", "A", "B", "C", "D", "z", "bias", "h0"]

    def f(v):
        y, fin = ssd.selscan_fwd(*args(v), init_state=v["h0"], **options(v))
        return ((y.double() * d["dout"].double()).sum() + (fin.double() * d["dfin"].double()).sum()).item()

    _, _, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
    for i, name in enumerate(names):
        torch.manual_seed(i)
        step = torch.randn_like(d[name])
        grad = g[{"bias": "ddt_bias", "h0": "dinit_state"}.get(name, "d" + name)]
        at = lambda e: f(dict(d, **{name: d[name] + e * step}))
        want = (grad.double() * step.double()).sum().item()
        assert abs((at(1e-2) - at(-1e-2)) / 2e-2 - want) < 2e-3 * (grad.norm() * step.norm()).item(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_options(dtype):
    """No D, z, bias, state or softplus: delta is dt itself, and equal lengths."""
    lens = [45, 45]
    x = make(dtype, lens, 0, 24, 16, 1, False, False, seed=6)
    x["D"] = x["bias"] = None
    x["dt"] = (0.02 + x["dt"].float().abs()).to(DT[dtype])
    d = dev(x)
    y, fin, st = ssd.selscan_fwd(*args(d), nseqs=2, return_states=True)
    g = ssd.selscan_bwd(*args(d), d["dout"], st, nseqs=2)
    want = ref(x, lens, grads=True, softplus=False)
    assert off(f64(y), want[0]) < TOL[dtype] and off(f64(fin), want[1]) < TOL["f32"]
    for k in ("dx", "ddt", "dB", "dC"):
        assert off(f64(g[k]), want[2][k]) < TOL[dtype], k
    assert off(f64(g["dA"]), want[2]["dA"]) < TOL["f32"]
    assert all(g[k] is None for k in ("dD", "dz", "ddt_bias", "dinit_state"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,G", [(16, 1), (10, 2), (64, 1), (3, 1), (8, 1)])
def test_single_tokens_continue_a_prompt(dtype, N, G):
    """A prompt's final states in the cache, then token by token, against the recurrence over
    the whole sequences."""
    lens, D = [20, 1, 9], 48
    x = make(dtype, lens, 0, D, N, G, True, False, seed=5)
    want, wfin = ref(x, lens)
    d = dev(x)
    keep, first, slot = [12, 1, 2], [0, 20, 21], [3, 0, 4]
    part = torch.cat([torch.arange(a, a + k) for a, k in zip(first, keep)]).cuda()
    pick = lambda rows: {k: d[k][rows] if k in ("x", "dt", "B", "C", "z") else d[k] for k in d}
    opt = dict(D=d["D"], dt_bias=d["bias"], dt_softplus=True)
    p = pick(part)
    _, fin = ssd.selscan_fwd(*args(p), z=p["z"], cu_seqlens=torch.tensor([0, 12, 13, 15], dtype=torch.int32, device="cuda"), **opt)
    cache = torch.full((5, D, N), 7.0, device="cuda")
    cache[slot] = fin
    for t in range(8):
        rows = [a + k + t if k + t < L else -1 for a, k, L in zip(first, keep, lens)]
        slots = torch.tensor([s if r >= 0 else -1 for s, r in zip(slot, rows)], dtype=torch.int32, device="cuda")
        p = pick([max(r, 0) for r in rows])
        y = ssd.selscan_step(*args(p), cache, z=p["z"], slots=slots, **opt)
        for i, r in enumerate(rows):
            assert off(f64(y[i]), want[r]) < TOL[dtype] if r >= 0 else not y[i].any()
    assert off(f64(cache[slot]), wfin) < TOL["f32"]
    assert (cache[[1, 2]] == 7.0).all()                # slots of no row are left alone
    # without slots, and one out of range
    p, c2 = pick([0, 1, 2]), cache.clone()
    a = ssd.selscan_step(*args(p), cache[:3].contiguous(), z=p["z"], **opt)
    b = ssd.selscan_step(*args(p), c2, z=p["z"], slots=torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda"), **opt)
    assert torch.equal(a[:2], b[:2]) and not b[2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_sequences_never_reach_a_result(dtype):
    lens = [33, 6, 40]
    clean = dev(make(dtype, lens, 4, 16, 16, 1, True, True, seed=7))
    bad = {k: v.clone() for k, v in clean.items()}
    for k in ("x", "dt", "B", "C", "z", "dout"):
        bad[k][33:39], bad[k][79:] = float("nan"), float("inf")
    bad["h0"][1] = bad["dfin"][1] = float("nan")
    res = []
    for d in (clean, bad):
        y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
        g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
        res.append((y, g["dx"], g["ddt"], g["dz"], g["dB"], g["dC"], fin, g["dinit_state"]))
    rows = list(range(33)) + list(range(39, 83))
    for a, b in zip(res[0][:6], res[1][:6]):
        assert torch.equal(a[rows], b[rows])
    for a, b in zip(res[0][6:], res[1][6:]):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_decays(dtype):
    """No memory (A = -inf), no decay (A = 0), and steps so large that every decay underflows."""
    lens = [70]
    x = make(dtype, lens, 0, 8, 4, 1, False, True, seed=8)
    x["A"][:, 0], x["A"][:, 1], x["A"][:, 2] = -float("inf"), 0.0, -1e30
    y, fin = ssd.selscan_fwd(*args(dev(x)), init_state=x["h0"].cuda(), **options(dev(x)))
    x["A"][:, 0] = -1e30
    want = ref(x, lens)
    # the sum without a decay has 70 terms, each off by delta's own error and a rounding
    assert off(f64(y), want[0]) < TOL[dtype] and off(f64(fin), want[1]) < TOL["f32"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_that_forgets(dtype):
    """Single tokens that leave little of a large state: what is left keeps its own precision.
    delta A is between -40 and 0 and rounded once in fp32 and once in delta, which moves its
    exponential by 40 * (2^-24 + 2^-21) at most, 2.2e-5 of each value; 1e-6 for the rest."""
    n, D, N = 3, 32, 16
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x, dt = torch.zeros(n, D).to(DT[dtype]), (4.0 * torch.rand(n, D, generator=g)).to(DT[dtype])
    A = -10.0 * torch.rand(D, N, generator=g)
    h = 1e4 * (rnd(n, D, N) + 3.0)
    B, C = rnd(n, 1, N).to(DT[dtype]), rnd(n, 1, N).to(DT[dtype])
    want = h.double() * torch.exp(torch.nn.functional.softplus(dt.double())[:, :, None] * A.double())
    cache = h.cuda()
    ssd.selscan_step(x.cuda(), dt.cuda(), A.cuda(), B.cuda(), C.cuda(), cache, dt_softplus=True)
    assert ((cache.double().cpu() - want).abs() <= 2.3e-5 * want.abs() + 1e-30).all()
    # a rate that is not a number stays one in its own state
    A[1, 2] = float("nan")
    again = h.cuda()
    ssd.selscan_step(x.cuda(), dt.cuda(), A.cuda(), B.cuda(), C.cuda(), again, dt_softplus=True)
    assert again[:, 1, 2].isnan().all()
    again[:, 1, 2] = cache[:, 1, 2]
    assert torch.equal(again, cache)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 48])
def test_channels_that_cancel(dtype, N):
    """Single tokens whose channels cancel in dB and dC: three of the same x and dt, with dout in
    the ratio 4 : -3 : -1.  What is left is rounding: three of each term's factors (3 * 2^-24; the
    channels share delta), and 24 terms' sum (24 * 2^-24): 1.7e-6 of the terms' absolute sum, 4e-6 allowed,
    and the output's own half step."""
    n, D = 2, 24
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g)
    three = lambda t: t.repeat_interleave(3, 1).to(DT[dtype])
    x, dt = three(rnd(n, D // 3)), three(rnd(n, D // 3))
    d = torch.randint(1, 16, (n, D // 3), generator=g).float()
    dout = (three(d).float() * torch.tensor([1.0, -0.75, -0.25]).repeat(D // 3)).to(DT[dtype])
    B, C, A = rnd(n, 1, N).to(DT[dtype]), rnd(n, 1, N).to(DT[dtype]), -torch.rand(D, N, generator=g)
    ops = [t.cuda() for t in (x, dt, A, B, C)]
    kw = dict(dt_softplus=True, nseqs=n)
    _, _, st = ssd.selscan_fwd(*ops, return_states=True, **kw)
    got = ssd.selscan_bwd(*ops, dout.cuda(), st, **kw)
    terms = (torch.nn.functional.softplus(dt.double()) * x.double() * dout.double())
    for k, other in (("dB", C), ("dC", B)):
        want = terms.sum(1)[:, None, None] * other.double()
        size = terms.abs().sum(1)[:, None, None] * other.double().abs()
        assert ((got[k].double().cpu() - want).abs() <= want.abs() * torch.finfo(DT[dtype]).eps / 2 + 4e-6 * size).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_of_no_tokens_alone(dtype):
    """No tokens at all: states and their gradients pass through, the others are zero."""
    x = make(dtype, [0, 0], 0, 16, 16, 1, True, True, seed=10)
    d = dev(x)
    y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
    assert y.shape == (0, 16) and torch.equal(fin, d["h0"]) and torch.equal(g["dinit_state"], d["dfin"])
    assert not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))


def test_state_in_place_and_offsets_past_32_bits():
    D, T, n = 8192, 270000, 100
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tail = dict(x=rnd(n, D).bfloat16(), dt=rnd(n, D).bfloat16(), B=rnd(n, 1, 16).bfloat16(), C=rnd(n, 1, 16).bfloat16())
    A = -torch.rand(D, 16, generator=g, device="cuda") - 0.5
    full = {}
    for k, v in tail.items():
        full[k] = torch.zeros(T, *v.shape[1:], device="cuda", dtype=torch.bfloat16)
        full[k][-n:] = v
    h0 = rnd(2, D, 16)
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    want, wfin, st = ssd.selscan_fwd(tail["x"], tail["dt"], A, tail["B"], tail["C"], dt_softplus=True, init_state=h0[1:].contiguous(), return_states=True)
    gw = ssd.selscan_bwd(tail["x"], tail["dt"], A, tail["B"], tail["C"], tail["x"], st, dt_softplus=True)
    y, fin, st = ssd.selscan_fwd(full["x"], full["dt"], A, full["B"], full["C"], dt_softplus=True, cu_seqlens=cu, init_state=h0,
                                 final_out=h0, return_states=True)
    gr = ssd.selscan_bwd(full["x"], full["dt"], A, full["B"], full["C"], full["x"], st, dt_softplus=True, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert fin.data_ptr() == h0.data_ptr()
    # the last sequence may be walked in one piece here and in ranges there
    assert off(f64(y[-n:]), f64(want)) < TOL["bf16"] and off(f64(h0[1:]), f64(wfin)) < TOL["f32"]
    for k in ("dx", "ddt", "dB", "dC"):
        assert off(f64(gr[k][-n:]), f64(gw[k])) < TOL["bf16"], k


def test_repeated_calls_agree():
    d = dev(make("bf16", [700, 33, 290], 0, 200, 16, 1, True, True, seed=11))
    flush = torch.empty(1 << 26, device="cuda")
    seen = None
    for _ in range(10):
        flush.zero_()
        y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
        g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
        now = [y, fin] + list(g.values())
        assert seen is None or all(torch.equal(a, b) for a, b in zip(now, seen))
        seen = now


def test_many_sequences():
    """More sequences than rows, most of them empty."""
    lens = [1 if s % 7 == 0 else 0 for s in range(3000)]
    x = make("f32", lens, 0, 16, 16, 1, True, True, seed=9)
    d = dev(x)
    y, fin, st = ssd.selscan_fwd(*args(d), init_state=d["h0"], return_states=True, **options(d))
    g = ssd.selscan_bwd(*args(d), d["dout"], st, dfinal_state=d["dfin"], return_dinit=True, **options(d))
    want = ref(x, lens, grads=True)
    assert off(f64(y), want[0]) < TOL["f32"] and off(f64(fin), want[1]) < TOL["f32"]
    for k in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dinit_state"):
        assert off(f64(g[k]), want[2][k]) < TOL["f32"], k
