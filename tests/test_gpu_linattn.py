"""Linear attention with a decay for each head: prompts, gradients and single
tokens against the token-by-token recurrence in 64 bits.

Tolerances, as 2-norm of the difference over 2-norm of the reference.  A bf16
result is rounded once and has two operands of its last products rounded to bf16
(the chunk's weights and the state), each by less than 2^-9 of it in the root
mean square (2^-8 at most): 3 * 2^-9.  An fp32 result (fp32 inputs, and every state) is a sum of a few
thousand products held in fp32: 2e-5.
"""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from linattn_ref import linattn, off

pytestmark = pytest.mark.gpu
TOL = {"bf16": 3 * 2.0 ** -9, "f32": 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# dtype, lengths, H, G, K, V, initial state
CASES = [
    ("bf16", [1], 1, 1, 16, 16, False),
    ("bf16", [1, 2, 127, 128, 129], 2, 1, 64, 64, True),
    ("bf16", [300, 0, 5, 64], 4, 2, 128, 128, True),      # an empty sequence, shared q and k
    ("bf16", [257], 3, 3, 96, 80, False),                 # sizes that are no powers of two
    ("bf16", [1300, 513, 2], 2, 2, 128, 48, True),        # sequences cut into ranges
    ("f32", [1], 2, 1, 32, 16, True),
    ("f32", [1, 63, 64, 65, 0], 2, 1, 64, 64, True),
    ("f32", [200, 33], 4, 2, 112, 128, False),
    ("f32", [1100, 600], 2, 1, 48, 80, True),
]


def make(dtype, lens, H, G, K, V, state, seed=0, decay=None):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x = dict(q=rnd(T, G, K).to(DT[dtype]), k=rnd(T, G, K).to(DT[dtype]), v=rnd(T, H, V).to(DT[dtype]),
             dout=rnd(T, H, V).to(DT[dtype]))
    x["a"] = -torch.exp2(-9.0 * torch.arange(1, H + 1) / H) if decay is None else torch.tensor(decay)
    x["S0"] = rnd(len(lens), H, V, K) if state else None
    x["dfin"] = rnd(len(lens), H, V, K) if state else None
    x["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return x


def dev(x):
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def f64(t):
    return None if t is None else t.double().numpy()


def ref(x, lens, scale, grads=False):
    return linattn(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["a"].numpy(), lens, scale, f64(x["S0"]),
                   f64(x["dout"]) if grads else None, f64(x["dfin"]) if grads else None)


def num(t):
    return t.double().cpu().numpy()


def sync_ok():
    torch.cuda.synchronize()
    assert ssd.ssd_take_device_errors() == 0


@pytest.mark.parametrize("dtype,lens,H,G,K,V,state", CASES)
def test_prompt(dtype, lens, H, G, K, V, state):
    x = make(dtype, lens, H, G, K, V, state)
    d = dev(x)
    for max_seqlen in (0, max(lens)):
        o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"], scale=0.3,
                                 init_state=d["S0"], max_seqlen=max_seqlen)
        sync_ok()
        ro, rf = ref(x, lens, 0.3)
        at = 0
        for s, L in enumerate(lens):   # each sequence by itself: a short one must not hide
            assert off(num(o[at:at + L]), ro[at:at + L]) < TOL[dtype], (s, L)
            assert off(num(fin[s]), rf[s]) < TOL["f32"], (s, L)
            at += L


@pytest.mark.parametrize("dtype,lens,H,G,K,V,state", CASES)
def test_gradient(dtype, lens, H, G, K, V, state):
    x = make(dtype, lens, H, G, K, V, state, seed=1)
    d = dev(x)
    got = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], cu_seqlens=d["cu"], scale=0.3,
                          init_state=d["S0"], dfinal_state=d["dfin"])
    sync_ok()
    want = ref(x, lens, 0.3, grads=True)[2:]
    at = 0
    for s, L in enumerate(lens):
        for name, g, w in zip(("dq", "dk", "dv"), got, want):
            assert off(num(g[at:at + L]), w[at:at + L]) < TOL[dtype], (name, s, L)
        if state:
            assert off(num(got[3][s]), want[3][s]) < TOL["f32"], (s, L)
        at += L
    assert (got[3] is None) == (not state)


def test_gradient_against_differences():
    """The result is linear in each of q, k, v and the initial state, so a
    difference of two forward passes along a direction is the gradient's product
    with it, up to the fp32 forward's own error: of the order of 1e-6 of the
    terms, which are at most about 100 times their sum here."""
    lens = [150, 70]
    x = make("f32", lens, 2, 1, 32, 48, True, seed=2)
    d = dev(x)
    kw = dict(cu_seqlens=d["cu"], scale=0.5)

    def f(q, k, v, S0):
        o, fin = ssd.linattn_fwd(q, k, v, d["a"], init_state=S0, **kw)
        return (o.double() * d["dout"].double()).sum() + (fin.double() * d["dfin"].double()).sum()

    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], init_state=d["S0"],
                        dfinal_state=d["dfin"], **kw)
    args = [d["q"], d["k"], d["v"], d["S0"]]
    base = f(*args)
    for i in range(4):
        torch.manual_seed(i)
        step = torch.randn_like(args[i])
        moved = [a + step if j == i else a for j, a in enumerate(args)]
        want = (g[i].double() * (moved[i] - args[i]).double()).sum()
        size = g[i].double().norm() * step.double().norm()
        assert abs(f(*moved) - base - want) < 1e-4 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-float("inf"), -40.0], [-0.9, 0.5]])
def test_decays(dtype, decay):
    """No decay, a very slow one, none of the past kept, underflow within a chunk; a
    positive value counts as 0."""
    lens = [400]
    x = make(dtype, lens, 2, 1, 64, 64, True, seed=3, decay=decay)
    d = dev(x)
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"], init_state=d["S0"])
    grads = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], cu_seqlens=d["cu"],
                            init_state=d["S0"], dfinal_state=d["dfin"])
    sync_ok()
    want = ref(x, lens, 64 ** -0.5, grads=True)
    for h in range(2):
        assert off(num(o[:, h]), want[0][:, h]) < TOL[dtype]
        assert off(num(fin[:, h]), want[1][:, h]) < TOL["f32"]
        assert off(num(grads[2][:, h]), want[4][:, h]) < TOL[dtype]
        if decay[h] > -30:   # below, dS_0 underflows to 0 on both sides
            assert off(num(grads[3][:, h]), want[5][:, h]) < TOL["f32"]
    assert off(num(grads[0]), want[2]) < TOL[dtype] and off(num(grads[1]), want[3]) < TOL[dtype]


@pytest.mark.parametrize("decay", [[-0.60, -0.66], [-0.655, -0.3]])
def test_fast_decays_and_large_values(decay):
    """Decays on both sides of the one up to which a chunk's decay is applied as row
    and column factors, and values whose products leave fp16's range."""
    lens = [300, 129]
    x = make("bf16", lens, 2, 2, 128, 64, True, seed=9, decay=decay)
    for n in ("q", "k", "v", "dout"):
        x[n] = (300 * x[n].float()).bfloat16()
    d = dev(x)
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"], init_state=d["S0"])
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], cu_seqlens=d["cu"],
                        init_state=d["S0"], dfinal_state=d["dfin"])
    sync_ok()
    want = ref(x, lens, 128 ** -0.5, grads=True)
    for h in range(2):
        assert off(num(o[:, h]), want[0][:, h]) < TOL["bf16"]
        assert off(num(fin[:, h]), want[1][:, h]) < TOL["f32"]
        for i in range(3):
            assert off(num(g[i][:, h]), want[2 + i][:, h]) < TOL["bf16"]
        assert off(num(g[3][:, h]), want[5][:, h]) < TOL["f32"]


def test_few_tokens_keep_both_terms():
    """Without a state, an output of a chunk of few tokens (64; 32 for fast decays) is a
    sum of a few products, or one: its weights keep 16 bits.  Element by element, with
    A the sum of the products' magnitudes: 2^-8 of the result for its own rounding, and
    2^-14 A for the weights (2^-16), their sums over K (K 2^-24 < 2^-16) and exponentials."""
    lens = [1] * 20 + [2, 5, 31, 32, 33, 63, 64]
    x = make("bf16", lens, 2, 2, 96, 64, False, seed=12, decay=[-0.01, -0.9])
    d = dev(x)
    o, _ = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"])
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], cu_seqlens=d["cu"])
    sync_ok()
    args = [f64(x[n]) for n in ("q", "k", "v")]
    run = lambda f: linattn(*[f(t) for t in args], x["a"].numpy(), lens, 96 ** -0.5, None, f(f64(x["dout"])))
    want, mag = run(lambda t: t), run(np.abs)
    for h, n in ((0, sum(lens)), (1, sum(lens[:24]))):
        for i, t in ((0, o), (2, g[0]), (3, g[1]), (4, g[2])):
            err = np.abs(num(t) - want[i])[:n, h]
            bound = 2.0 ** -8 * np.abs(want[i]) + 2.0 ** -14 * mag[i]
            assert (err <= bound[:n, h]).all(), (h, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("long", [0, 2500])
def test_very_many_sequences(dtype, long):
    """More sequences than two steps of the search over their offsets tell apart, of 0
    to 3 tokens, by themselves and with a long one among them that is cut."""
    lens = [i % 4 for i in range(700)] + [long] + [(3 * i) % 4 for i in range(700)]
    x = make(dtype, lens, 1, 1, 16, 32, True, seed=14)
    d = dev(x)
    for max_seqlen in (0, max(lens)):
        kw = dict(cu_seqlens=d["cu"], init_state=d["S0"], max_seqlen=max_seqlen)
        o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw)
        g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw)
        sync_ok()
        want = ref(x, lens, 16 ** -0.5, grads=True)
        assert off(num(o), want[0]) < TOL[dtype] and off(num(fin), want[1]) < TOL["f32"]
        for i in range(3):
            assert off(num(g[i]), want[2 + i]) < TOL[dtype]
        assert off(num(g[3]), want[5]) < TOL["f32"]


def test_one_long_sequence():
    """A single sequence's ranges are made to fill the GPU (their number follows from
    the length alone), with and without offsets; so are those of equal sequences."""
    for lens in ([5000], [2600, 2600]):
        x = make("bf16", lens, 2, 1, 32, 48, True, seed=13)
        d = dev(x)
        for kw in (dict(cu_seqlens=d["cu"], max_seqlen=max(lens)), dict(nseqs=len(lens))):
            o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], init_state=d["S0"], **kw)
            g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], init_state=d["S0"],
                                dfinal_state=d["dfin"], **kw)
            sync_ok()
            want = ref(x, lens, 32 ** -0.5, grads=True)
            assert off(num(o), want[0]) < TOL["bf16"] and off(num(fin), want[1]) < TOL["f32"]
            for i in range(3):
                assert off(num(g[i]), want[2 + i]) < TOL["bf16"]
            assert off(num(g[3]), want[5]) < TOL["f32"]


def test_long_sequences_among_many_empty_ones():
    """Sequences cut into ranges, many that are empty, and no bound of the lengths:
    most of the work list has nothing to do, and every sequence's state arrives."""
    lens = [0] * 40 + [1500] + [0] * 200 + [2100, 1] + [0] * 60
    x = make("bf16", lens, 2, 2, 64, 64, True, seed=10)
    d = dev(x)
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"], init_state=d["S0"])
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], cu_seqlens=d["cu"],
                        init_state=d["S0"], dfinal_state=d["dfin"])
    sync_ok()
    want = ref(x, lens, 64 ** -0.5, grads=True)
    assert off(num(o), want[0]) < TOL["bf16"] and off(num(fin), want[1]) < TOL["f32"]
    for i in range(3):
        assert off(num(g[i]), want[2 + i]) < TOL["bf16"]
    assert off(num(g[3]), want[5]) < TOL["f32"]
    empty = [s for s, L in enumerate(lens) if L == 0]
    assert torch.equal(fin[empty], d["S0"][empty])


def test_rows_far_apart():
    """Rows whose offsets pass 2^31 elements give what a compact copy gives."""
    T, wide = 70000, 32768
    base = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")   # 4.6 GB
    torch.manual_seed(0)
    cut = lambda at, n: base[:, at:at + n]
    q, k, v = cut(0, 64).view(T, 1, 64), cut(16384, 64).view(T, 1, 64), cut(32768 - 128, 128).view(T, 2, 64)
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, device="cuda"))
    a = torch.tensor([-0.01, -0.2], device="cuda")
    cu = torch.tensor([0, 100, 69000, 70000], dtype=torch.int32, device="cuda")
    o, fin = ssd.linattn_fwd(q, k, v, a, cu_seqlens=cu)
    o1, fin1 = ssd.linattn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), a, cu_seqlens=cu)
    sync_ok()
    assert torch.equal(o, o1) and torch.equal(fin, fin1)


def test_cache_past_32_bits():
    """A slot whose offset passes 2^31 elements of the cache."""
    H, V, K, nslots = 32, 128, 128, 4200
    cache = torch.empty(nslots, H, V, K, device="cuda")                # 8.8 GB
    x = make("bf16", [1, 1], H, H, K, V, True, seed=11)
    d = dev(x)
    slots = torch.tensor([nslots - 1, 3], dtype=torch.int32, device="cuda")
    cache[slots.long()] = d["S0"]
    o = ssd.linattn_step(d["q"], d["k"], d["v"], d["a"], cache, slots=slots)
    small = d["S0"].clone()
    o1 = ssd.linattn_step(d["q"], d["k"], d["v"], d["a"], small)
    assert torch.equal(o, o1) and torch.equal(cache[slots.long()], small)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_rows_do_not_leak(dtype):
    """NaN and infinities in another sequence and in rows of no sequence; the
    latter's results are 0."""
    lens = [70, 30, 200]
    x = make(dtype, lens, 2, 2, 64, 96, True, seed=4)
    clean = dev(x)
    pad = 37
    for n in ("q", "k", "v", "dout"):
        t = torch.cat([x[n], torch.full((pad, *x[n].shape[1:]), float("nan"), dtype=x[n].dtype)])
        t[70:100] = float("inf")
        x[n] = t
    x["S0"][1] = float("nan")
    d = dev(x)
    kw = lambda z: dict(cu_seqlens=z["cu"], init_state=z["S0"])
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw(d))
    o0, fin0 = ssd.linattn_fwd(clean["q"], clean["k"], clean["v"], clean["a"], **kw(clean))
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw(d))
    g0 = ssd.linattn_bwd(clean["q"], clean["k"], clean["v"], clean["dout"], clean["a"],
                         dfinal_state=clean["dfin"], **kw(clean))
    sync_ok()
    for a, b in [(o, o0), *zip(g[:3], g0[:3])]:
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[100:300], b[100:300])
        assert torch.all(a[300:] == 0)
    for a, b in [(fin, fin0), (g[3], g0[3])]:
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert torch.isnan(o[70:100]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_streams_and_repeats(dtype):
    """Rows that are slices of one projection's, another stream than the tensors'
    own, in-place states: the same bits each time."""
    lens, H, G, K, V = [90, 700], 4, 2, 32, 64
    x = make(dtype, lens, H, G, K, V, True, seed=5)
    d = dev(x)
    T = sum(lens)
    kw = dict(cu_seqlens=d["cu"], init_state=d["S0"])
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw)
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw)
    wide = torch.cat([d["q"].reshape(T, -1), d["k"].reshape(T, -1), d["v"].reshape(T, -1)], 1)
    q, k = (wide[:, i * G * K:(i + 1) * G * K].view(T, G, K) for i in (0, 1))
    v = wide[:, 2 * G * K:].view(T, H, V)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S = d["S0"].clone()
        o1, f1 = ssd.linattn_fwd(q, k, v, d["a"], cu_seqlens=d["cu"], init_state=S, final_out=S)
        g1 = ssd.linattn_bwd(q, k, v, d["dout"], d["a"], dfinal_state=d["dfin"], **kw)
    side.synchronize()
    assert f1 is S and torch.equal(o, o1) and torch.equal(fin, f1)
    assert all(torch.equal(a, b) for a, b in zip(g, g1))
    # equal lengths without a table
    o2, f2 = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], nseqs=2, init_state=d["S0"])
    cu = torch.tensor([0, 395, 790], dtype=torch.int32, device="cuda")
    o3, f3 = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=cu, init_state=d["S0"], max_seqlen=395)
    assert torch.equal(o2, o3) and torch.equal(f2, f3)


def test_table_outside_the_tensors_is_clamped():
    x = dev(make("bf16", [100], 1, 1, 64, 64, False, seed=6))
    cu = torch.tensor([-5, 40, 30, 1000], dtype=torch.int32, device="cuda")
    o, fin = ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"], cu_seqlens=cu)
    sync_ok()
    assert o.shape == (100, 1, 64) and torch.isfinite(fin).all()


def test_no_tokens():
    """Empty sequences pass the state on."""
    q = torch.empty(0, 1, 32, device="cuda")
    v = torch.empty(0, 2, 16, device="cuda")
    a = torch.tensor([-0.1, -0.2], device="cuda")
    S = torch.randn(3, 2, 16, 32, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, fin = ssd.linattn_fwd(q, q, v, a, cu_seqlens=cu, init_state=S)
    g = ssd.linattn_bwd(q, q, v, v, a, cu_seqlens=cu, init_state=S, dfinal_state=2 * S)
    assert o.numel() == 0 and torch.equal(fin, S) and torch.equal(g[3], 2 * S)


@pytest.mark.parametrize("dtype,b,H,G,K,V", [
    ("bf16", 1, 1, 1, 16, 16), ("bf16", 5, 6, 2, 128, 64), ("f32", 3, 4, 4, 48, 112),
    ("bf16", 9, 2, 1, 96, 80), ("f32", 2, 3, 1, 32, 128)])
def test_step(dtype, b, H, G, K, V):
    x = make(dtype, [1] * b, H, G, K, V, True, seed=7)
    d = dev(x)
    nslots = b + 3
    torch.manual_seed(b)
    cache = torch.randn(nslots, H, V, K)
    slots = torch.randperm(nslots)[:b].to(torch.int32)
    x["S0"] = cache[slots.long()]
    idle = b // 2 if b > 2 else None
    if idle is not None:
        slots[idle] = -1
    c = cache.cuda()
    o = ssd.linattn_step(d["q"], d["k"], d["v"], d["a"], c, slots=slots.cuda(), scale=0.7)
    torch.cuda.synchronize()
    ro, rf = ref(x, [1] * b, 0.7)
    want = cache.double().numpy().copy()
    for i in range(b):
        if i == idle:
            assert torch.all(o[i] == 0)
            continue
        want[slots[i]] = rf[i]
        assert off(num(o[i]), ro[i]) < TOL[dtype]
    assert off(num(c), want) < 1e-6
    untouched = [s for s in range(nslots) if s not in slots.tolist()]
    assert torch.equal(c.cpu()[untouched], cache[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps(dtype):
    """A prompt into the cache, then token by token: as one longer prompt."""
    L, n, H, G, K, V = 150, 6, 4, 2, 64, 32
    x = dev(make(dtype, [L + n], H, G, K, V, False, seed=8))
    o, fin = ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"])
    cache = torch.zeros(4, H, V, K, device="cuda")
    o1, _ = ssd.linattn_fwd(x["q"][:L], x["k"][:L], x["v"][:L], x["a"], init_state=cache[2:3],
                            final_out=cache[2:3])
    assert off(num(o1), num(o[:L])) < TOL[dtype]
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in range(L, L + n):
        ot = ssd.linattn_step(x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1], x["a"], cache, slots=slots)
        assert off(num(ot[0]), num(o[t])) < TOL[dtype]
    assert off(num(cache[2]), num(fin[0])) < TOL["f32"]


def test_binding_refuses():
    x = dev(make("bf16", [8], 2, 1, 32, 32, True))
    f = ssd.linattn_fwd
    with pytest.raises(TypeError):
        f(x["q"].half(), x["k"].half(), x["v"].half(), x["a"])
    with pytest.raises(TypeError):
        f(x["q"], x["k"].float(), x["v"], x["a"])
    with pytest.raises(TypeError):
        f(x["q"], x["k"], x["v"], x["a"].double())
    with pytest.raises(ValueError):
        f(x["q"], x["k"][:4], x["v"], x["a"])
    with pytest.raises(ValueError):
        f(x["q"], x["k"], x["v"], x["a"], init_state=x["S0"].transpose(2, 3)[:, :, :16])
    with pytest.raises(ValueError):
        f(x["q"].transpose(0, 2).contiguous().transpose(0, 2), x["k"], x["v"], x["a"])
    with pytest.raises(ValueError):
        f(x["q"], x["k"], x["v"], x["a"], cu_seqlens=x["cu"].long())
    with pytest.raises(ssd.SSDError):
        f(x["q"][..., :24], x["k"][..., :24], x["v"], x["a"])
    with pytest.raises(ssd.SSDError):
        f(x["q"], x["k"], x["v"], x["a"], nseqs=3)
    with pytest.raises(ssd.SSDError):
        f(x["q"], x["k"], x["v"], x["a"], out=x["v"])
