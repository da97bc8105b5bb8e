"""The short convolution over packed rows: prompts, gradients and single tokens against
the definition in 64 bits.

Tolerances, as 2-norm of the difference over 2-norm of the reference.  bf16 outputs are
rounded once from fp32: 2^-8 of each value at most, and 2e-5 as for fp32.  fp32 outputs
are sums of up to 9 products (2^-24 of each term a step, the terms being of the sum's
size) times a sigmoid (two approximations of 2^-22); sums over a few hundred tokens add
at most that many 2^-24: 2e-5.
"""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from selscan_ref import off, short_conv

pytestmark = pytest.mark.gpu
TOL = {"bf16": 2.0 ** -8 + 2e-5, "f32": 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# dtype, lengths, rows behind them, channels, taps, activation, bias, initial state
CASES = [
    ("bf16", [1], 0, 8, 4, "silu", True, False),
    ("bf16", [1, 2, 3, 4, 31, 32, 33, 0, 64, 65], 3, 40, 4, "silu", True, True),
    ("f32", [2, 0, 0, 5, 100, 1, 1, 1], 0, 24, 4, "silu", False, True),
    ("f32", [7, 130], 1, 1032, 2, None, True, True),
    ("bf16", [3, 66, 9, 8], 0, 16, 8, "silu", True, True),
    ("f32", [3, 66, 9, 8], 2, 16, 8, None, True, True),
    ("bf16", [300], 0, 2048, 3, None, True, False),
    ("f32", [5, 6, 7], 0, 8, 5, "silu", True, True),
    ("bf16", [5, 6, 7], 0, 8, 6, "silu", True, False),
    ("f32", [5, 6, 90], 0, 8, 7, "silu", True, True),
]


def make(dtype, lens, pad, D, W, bias, state, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    T = sum(lens) + pad
    return dict(x=rnd(T, D).to(DT[dtype]), w=rnd(D, W) * W ** -0.5, b=rnd(D) if bias else None,
                init=rnd(len(lens), W - 1, D).to(DT[dtype]) if state else None, dout=rnd(T, D).to(DT[dtype]),
                dfin=rnd(len(lens), W - 1, D).to(DT[dtype]) if state else None,
                cu=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32))


def dev(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def ref(x, lens, act, grads=True):
    b = np.zeros(x["w"].shape[0]) if x["b"] is None else f64(x["b"])
    return short_conv(f64(x["x"]), f64(x["w"]), b, lens, act, f64(x["init"]), f64(x["dout"]) if grads else None, f64(x["dfin"]))


@pytest.mark.parametrize("dtype,lens,pad,D,W,act,bias,state", CASES)
def test_prompt_and_gradient(dtype, lens, pad, D, W, act, bias, state):
    x = make(dtype, lens, pad, D, W, bias, state)
    d = dev(x)
    # x as the columns of a wider tensor
    wide = torch.randn(len(x["x"]), 2 * D, device="cuda").to(DT[dtype])
    wide[:, D:] = d["x"]
    kw = dict(bias=d["b"], activation=act, cu_seqlens=d["cu"], init_state=d["init"])
    want = ref(x, lens, act)
    for xin in (d["x"], wide[:, D:]):
        o, fin = ssd.short_conv_fwd(xin, d["w"], **kw)
        g = ssd.short_conv_bwd(xin, d["w"], d["dout"], dfinal_state=d["dfin"], **kw)
        torch.cuda.synchronize()
        at = 0
        for s, L in enumerate(lens):   # each sequence by itself: a short one must not hide
            assert off(f64(o[at:at + L]), want[0][at:at + L]) < TOL[dtype], (s, L)
            assert off(f64(g["dx"][at:at + L]), want[2][at:at + L]) < TOL[dtype], (s, L)
            at += L
        assert np.array_equal(f64(fin), want[1])       # copies
        assert not o[at:].any() and not g["dx"][at:].any()
        assert off(f64(g["dweight"]), want[3]) < TOL["f32"]
        assert (g["dbias"] is None) == (not bias)
        if bias:
            assert off(f64(g["dbias"]), want[4]) < TOL["f32"]
        assert (g["dinit_state"] is None) == (not state)
        if state:
            assert off(f64(g["dinit_state"]), want[5]) < TOL[dtype]


def test_gradient_against_differences():
    """fp32: a central difference of step 1e-2 along a random direction is the gradient's
    product with it up to the third derivative's (1e-2)^2 / 6 share and the forward's own
    error over the step, both below 1e-3 of the norms' product."""
    lens = [40, 3, 27]
    d = dev(make("f32", lens, 0, 16, 4, True, True, seed=3))
    kw = dict(activation="silu", cu_seqlens=d["cu"])

    def f(x, w, b, init):
        o, fin = ssd.short_conv_fwd(x, w, bias=b, init_state=init, **kw)
        return ((o.double() * d["dout"].double()).sum() + (fin.double() * d["dfin"].double()).sum()).item()

    args = [d["x"], d["w"], d["b"], d["init"]]
    g = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], bias=d["b"], init_state=d["init"], dfinal_state=d["dfin"], **kw)
    for i, name in enumerate(("dx", "dweight", "dbias", "dinit_state")):
        torch.manual_seed(i)
        step = torch.randn_like(args[i])
        at = lambda e: f(*[a + e * step if j == i else a for j, a in enumerate(args)])
        want = (g[name].double() * step.double()).sum().item()
        assert abs((at(1e-2) - at(-1e-2)) / 2e-2 - want) < 1e-3 * (g[name].norm() * step.norm()).item(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_lengths_and_no_state(dtype):
    lens = [37] * 4
    x = make(dtype, lens, 0, 32, 4, True, False)
    d = dev(x)
    a = ssd.short_conv_fwd(d["x"], d["w"], bias=d["b"], activation="silu", cu_seqlens=d["cu"])
    b = ssd.short_conv_fwd(d["x"], d["w"], bias=d["b"], activation="silu", nseqs=4)
    ga = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], bias=d["b"], activation="silu", cu_seqlens=d["cu"])
    gb = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], bias=d["b"], activation="silu", nseqs=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert all(torch.equal(ga[k], gb[k]) for k in ("dx", "dweight", "dbias"))
    # no rows at all
    none = ssd.short_conv_fwd(d["x"][:0], d["w"], nseqs=2)
    assert none[0].shape == (0, 32) and not none[1].any()
    g0 = ssd.short_conv_bwd(d["x"][:0], d["w"], d["dout"][:0], bias=d["b"], nseqs=2)
    assert not g0["dweight"].any() and not g0["dbias"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 4, 8])
def test_single_tokens_continue_a_prompt(dtype, W):
    """A prompt's final states in the cache, then token by token, are the whole sequence's
    outputs, bit for bit: the same sums in the same order."""
    lens, D = [20, 1, 9], 48
    x = make(dtype, lens, 0, D, W, True, False, seed=5)
    d = dev(x)
    kw = dict(bias=d["b"], activation="silu")
    whole, last = ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"], **kw)
    keep = [12, 1, 2]
    first = [0, 20, 21]
    part = torch.cat([torch.arange(a, a + k) for a, k in zip(first, keep)]).cuda()
    pcu = torch.tensor([0, 12, 13, 15], dtype=torch.int32, device="cuda")
    o, fin = ssd.short_conv_fwd(d["x"][part], d["w"], cu_seqlens=pcu, **kw)
    assert torch.equal(o, whole[part])
    cache = torch.full((5, W - 1, D), 7.0, device="cuda").to(DT[dtype])
    slot = [3, 0, 4]
    cache[slot] = fin
    for t in range(8):
        rows = [a + k + t if k + t < L else -1 for a, k, L in zip(first, keep, lens)]
        slots = torch.tensor([s if r >= 0 else -1 for s, r in zip(slot, rows)], dtype=torch.int32, device="cuda")
        x1 = d["x"][[max(r, 0) for r in rows]]
        o = ssd.short_conv_step(x1, d["w"], cache, slots=slots, **kw)
        for i, r in enumerate(rows):
            assert torch.equal(o[i], whole[r]) if r >= 0 else not o[i].any()
    assert torch.equal(cache[slot], last)
    assert (cache[[1, 2]] == 7.0).all()                # slots of no row are left alone
    # without slots, and one out of range
    c2 = cache.clone()
    a = ssd.short_conv_step(d["x"][:3], d["w"], cache[:3].contiguous(), **kw)
    b = ssd.short_conv_step(d["x"][:3], d["w"], c2, slots=torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda"), **kw)
    assert torch.equal(a[:2], b[:2]) and not b[2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_sequences_never_reach_a_result(dtype):
    """Infinities and NaN in one sequence's rows, in its state and in the rows of none."""
    lens = [33, 6, 40]
    x = make(dtype, lens, 4, 16, 4, True, True, seed=7)
    clean = dev(x)
    bad = {k: None if v is None else v.clone() for k, v in clean.items()}
    bad["x"][33:39], bad["x"][79:] = float("nan"), float("inf")
    bad["init"][1], bad["dfin"][1], bad["dout"][33:39], bad["dout"][79:] = (float("nan"),) * 4
    res = []
    for d in (clean, bad):
        kw = dict(bias=d["b"], activation="silu", cu_seqlens=d["cu"], init_state=d["init"])
        o, fin = ssd.short_conv_fwd(d["x"], d["w"], **kw)
        g = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], dfinal_state=d["dfin"], **kw)
        res.append((o, g["dx"], fin, g["dinit_state"]))
    rows = list(range(33)) + list(range(39, 83))
    for a, b in zip(res[0][:2], res[1][:2]):
        assert torch.equal(a[rows], b[rows])
    for a, b in zip(res[0][2:], res[1][2:]):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last sequence alone against itself in a short call."""
    D, T = 8192, 270000
    x = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    tail = torch.randn(100, D, device="cuda").bfloat16()
    x[-100:] = tail
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    cu = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    o, fin = ssd.short_conv_fwd(x, w, bias=b, activation="silu", cu_seqlens=cu)
    want, wfin = ssd.short_conv_fwd(tail, w, bias=b, activation="silu")
    assert torch.equal(o[-100:], want) and torch.equal(fin[1], wfin[0])
    g = ssd.short_conv_bwd(x, w, x, bias=b, activation="silu", cu_seqlens=cu)
    gw = ssd.short_conv_bwd(tail, w, tail, bias=b, activation="silu")
    assert torch.equal(g["dx"][-100:], gw["dx"])


def test_many_sequences():
    """More sequences than rows, most of them empty."""
    n, D = 3000, 16
    lens = [1 if s % 7 == 0 else 0 for s in range(n)]
    x = make("f32", lens, 0, D, 4, True, True, seed=9)
    d = dev(x)
    kw = dict(bias=d["b"], activation="silu", cu_seqlens=d["cu"], init_state=d["init"])
    o, fin = ssd.short_conv_fwd(d["x"], d["w"], **kw)
    g = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], dfinal_state=d["dfin"], **kw)
    want = ref(x, lens, "silu")
    assert off(f64(o), want[0]) < TOL["f32"] and np.array_equal(f64(fin), want[1])
    assert off(f64(g["dx"]), want[2]) < TOL["f32"] and off(f64(g["dinit_state"]), want[5]) < TOL["f32"]
    assert off(f64(g["dweight"]), want[3]) < TOL["f32"]
