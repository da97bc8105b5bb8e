"""Linear attention at the edges of what its arguments may be: no sequence, rows of no
sequence behind long ones."""
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from linattn_ref import off
from test_gpu_linattn import DT, TOL, dev, make, num, ref, sync_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 200, 10000])
@pytest.mark.parametrize("H,G", [(4, 4), (4, 2)])
def test_rows_without_a_sequence(dtype, tokens, H, G):
    """Offsets [0]: every row belongs to no sequence, whatever it holds, and its
    results are 0; the calls after that one are as ever."""
    x = dev(make(dtype, [tokens], H, G, 64, 64, False))
    for n in ("q", "k", "v", "dout"):
        x[n][::7] = float("nan")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((tokens, H, 64), 7.0, dtype=DT[dtype], device="cuda")
    for max_seqlen in (0, 100):
        o, fin = ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"], cu_seqlens=cu, max_seqlen=max_seqlen, out=out)
        g = ssd.linattn_bwd(x["q"], x["k"], x["v"], x["dout"], x["a"], cu_seqlens=cu, max_seqlen=max_seqlen)
        sync_ok()
        assert o is out and fin.shape == (0, H, 64, 64) and g[3] is None
        for t in (o, *g[:3]):
            assert torch.all(t == 0)
        out.fill_(7.0)
    # the runtime has no error left over
    w = torch.ones(64, device="cuda")
    ssd.block_norm_fwd(torch.ones(3, 64, device="cuda"), torch.ones(3, 64, device="cuda"), w)
    sync_ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_tail_of_no_sequence(dtype):
    """Rows of no sequence, longer than a range, behind a sequence that is cut and behind
    one that is not."""
    for lens, pad, max_seqlen in (([2500, 3], 3000, 0), ([300, 200], 3000, 300)):
        x = make(dtype, lens, 2, 1, 32, 80, True, seed=15)
        for n in ("q", "k", "v", "dout"):
            x[n] = torch.cat([x[n], torch.full((pad, *x[n].shape[1:]), float("inf"), dtype=x[n].dtype)])
        d = dev(x)
        kw = dict(cu_seqlens=d["cu"], init_state=d["S0"], max_seqlen=max_seqlen)
        o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw)
        g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw)
        sync_ok()
        T = sum(lens)
        want = ref({n: t if n in ("a", "S0", "dfin", "cu") else t[:T] for n, t in x.items()}, lens, 32 ** -0.5,
                   grads=True)
        for t, w in ((o, want[0]), *zip(g[:3], want[2:5])):
            assert off(num(t[:T]), w) < TOL[dtype] and torch.all(t[T:] == 0)
        assert off(num(fin), want[1]) < TOL["f32"] and off(num(g[3]), want[5]) < TOL["f32"]


def test_rows_that_share_memory_are_refused():
    x = dev(make("bf16", [40], 2, 1, 32, 64, False))
    f = lambda **kw: ssd.linattn_fwd(**{**dict(q=x["q"], k=x["k"], v=x["v"], log_decay=x["a"]), **kw})
    f()
    for n in ("q", "k", "v"):
        with pytest.raises(ValueError):
            f(**{n: x[n][:1].expand(x[n].shape)})
    r, y = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for kw in (dict(y=y[:1].expand(4, 64), z=y), dict(y=y, z=y[:1].expand(4, 64))):
        with pytest.raises(ValueError):
            ssd.block_norm_fwd(r, w_pre=w, gate="silu", **kw)
    sync_ok()


def test_more_rows_of_no_sequence_than_32_bits_count():
    """2^25 rows of 64 columns behind a short sequence, uncut: their elements pass 2^31."""
    T, K, V = (1 << 25) + 100, 16, 64
    q = torch.zeros(T, 1, K, device="cuda")
    v = torch.zeros(T, 1, V, device="cuda")                      # 8.6 GB, and as much for o
    out = torch.full((T, 1, V), 7.0, device="cuda")
    torch.manual_seed(16)
    q[:100], v[:100] = torch.randn(100, 1, K, device="cuda"), torch.randn(100, 1, V, device="cuda")
    a = torch.tensor([-0.1], device="cuda")
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    o, _ = ssd.linattn_fwd(q, q, v, a, cu_seqlens=cu, max_seqlen=100, out=out)
    want, _ = ssd.linattn_fwd(q[:100], q[:100], v[:100], a)
    sync_ok()
    assert o is out and torch.equal(o[:100], want)
    assert not torch.any(o[100:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [95, -95])
def test_range_of_fp32(dtype, power):
    """States and products near the ends of fp32's range come through in both directions,
    whatever the decay: each case is an ordinary one with two operands times 2^(power / 2)
    or a state and its operand times 2^power, whose results are those times powers of two."""
    lens = [300, 129, 40]
    decay = [-0.6, -0.3, -0.01, -2.0]
    x = make(dtype, lens, 4, 4, 64, 64, True, seed=17, decay=decay)
    d = dev(x)
    kw = dict(cu_seqlens=d["cu"])
    want = ref(x, lens, 0.125, grads=True)
    s, h = 2.0 ** power, 2.0 ** (power // 2)

    def run(q=1.0, k=1.0, v=1.0, dout=1.0, S0=1.0, dfin=1.0):
        m = {n: d[n] * f for n, f in (("q", q), ("k", k), ("v", v), ("dout", dout), ("S0", S0), ("dfin", dfin))}
        o, fin = ssd.linattn_fwd(m["q"], m["k"], m["v"], d["a"], init_state=m["S0"], scale=0.125, **kw)
        g = ssd.linattn_bwd(m["q"], m["k"], m["v"], m["dout"], d["a"], init_state=m["S0"], scale=0.125,
                            dfinal_state=m["dfin"], **kw)
        sync_ok()
        return o, fin, *g

    def near(got, factors):
        for i, (t, f) in enumerate(zip(got, factors)):
            for head in range(4):
                assert off(num(t[:, head]) / f, want[i][:, head]) < TOL["f32" if i in (1, 5) else dtype], (i, head)

    # o, final state, dq, dk, dv, dS0
    near(run(v=s, S0=s), (s, s, s, s, 1, 1))
    near(run(dout=s, dfin=s), (1, 1, s, s, s, s))
    near(run(q=h, k=h, S0=h, dfin=h), (h * h, h, h, h, h * h, h))
    near(run(v=h, dout=h, S0=h, dfin=h), (h, h, h * h, h * h, h, h))


# which rows of each output depend on token t's row of each input: those from t on, up to
# t, t's alone, or none
SEEN = {"q": dict(o="only", dq=None, dk="upto", dv="upto"), "k": dict(o="from", dq="from", dk=None, dv="only"),
        "v": dict(o="from", dq="from", dk="only", dv=None), "dout": dict(o=None, dq="only", dk="upto", dv="upto")}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length,token", [(400, 0), (400, 5), (400, 63), (400, 64), (400, 127), (400, 128), (400, 333),
                                          (400, 399), (40, 17), (2600, 1500), (1, 0)])
def test_a_token_reaches_no_row_that_does_not_see_it(dtype, length, token):
    """An infinity or a NaN in one token's row: the rows that depend on it are not finite,
    all others have the bits they had without it."""
    x = make(dtype, [length], 2, 2, 32, 80, True, seed=21, decay=[-0.05, -0.4])
    kw = lambda d: dict(cu_seqlens=d["cu"], init_state=d["S0"])

    def run(d):
        o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw(d))
        dq, dk, dv, d0 = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw(d))
        sync_ok()
        return dict(o=o, dq=dq, dk=dk, dv=dv), fin, d0

    clean, fin0, d00 = run(dev(x))
    rows = torch.arange(length, device="cuda")
    for name, sees in SEEN.items():
        for value, column in ((float("inf"), slice(None)), (float("nan"), 7)):
            d = dev(x)
            d[name][token, 0, column] = value
            got, fin, d0 = run(d)
            for out, how in sees.items():
                hit = {"from": rows >= token, "upto": rows <= token, "only": rows == token, None: rows < 0}[how]
                g, c = got[out][:, 0], clean[out][:, 0]
                assert torch.equal(g[~hit], c[~hit]), (name, out)
                assert torch.equal(got[out][:, 1], clean[out][:, 1]), (name, out)
                # v and dout share their columns with o and dv, and k and q with dq and dk:
                # there the other columns are as they were
                same = column != slice(None) and (name, out) in (("v", "o"), ("k", "dq"), ("q", "dk"), ("dout", "dv"))
                if same:
                    rest = [i for i in range(g.shape[1]) if i != column]
                    assert torch.equal(g[:, rest], c[:, rest]), (name, out)
                    assert not torch.isfinite(g[hit][:, column]).any(), (name, out)
                else:
                    assert not torch.isfinite(g[hit]).any(), (name, out)
            # the states: the final one sees k and v, the initial one's gradient q and dout
            assert torch.equal(fin, fin0) == (name in ("q", "dout"))
            assert torch.equal(d0, d00) == (name in ("k", "v"))


def bf16_rounding(want):
    """2-norm of what one rounding to bf16 adds to a result, over the result's."""
    return off(num(torch.from_numpy(want).bfloat16()), want)


@pytest.mark.parametrize("lens,H,G,K,V", [([1000, 300], 4, 4, 128, 128), ([700], 6, 2, 96, 80), ([3000], 2, 1, 64, 64)])
def test_bf16_has_one_rounding_more_than_its_own(lens, H, G, K, V):
    """Each term of an output has one operand rounded to bf16 (a weight, or the state), so
    that the terms' independent errors add up to what one rounding of the output makes;
    with the output's own, sqrt(2) of that.  A tenth more for the spread of a sample."""
    x = make("bf16", lens, H, G, K, V, True, seed=22)
    d = dev(x)
    kw = dict(cu_seqlens=d["cu"], init_state=d["S0"])
    o, _ = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], **kw)
    g = ssd.linattn_bwd(d["q"], d["k"], d["v"], d["dout"], d["a"], dfinal_state=d["dfin"], **kw)
    sync_ok()
    want = ref(x, lens, K ** -0.5, grads=True)
    for t, w in ((o, want[0]), *zip(g[:3], want[2:5])):
        assert off(num(t), w) < 1.1 * 2 ** 0.5 * bf16_rounding(w)


def test_calls_in_a_graph():
    """Every call can be captured: a replay gives the bits of a call."""
    x = dev(make("bf16", [700, 90], 4, 2, 64, 64, True, seed=23))
    s = dev(make("bf16", [1, 1], 4, 2, 64, 64, True, seed=24))
    r, w = torch.randn(790, 256, device="cuda"), torch.ones(256, device="cuda")
    kw = dict(cu_seqlens=x["cu"], init_state=x["S0"])

    def calls(cache):
        o, fin = ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"], **kw)
        g = ssd.linattn_bwd(x["q"], x["k"], x["v"], x["dout"], x["a"], dfinal_state=x["dfin"], **kw)
        y = ssd.linattn_step(s["q"], s["k"], s["v"], s["a"], cache)
        ro, n, rstd = ssd.block_norm_fwd(r, o.reshape(790, 256), w, ngroups=4, return_rstd=True)
        gn = ssd.block_norm_bwd(r, o.reshape(790, 256), w, ro, n, rstd, ngroups=4)
        return [o, fin, *g, y, ro, n, gn["dr"], gn["dy"], gn["dw_pre"]]

    calls(s["S0"].clone())
    eager_cache, cache = s["S0"].clone(), s["S0"].clone()
    want = calls(eager_cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(cache)
    for t in got:
        t.zero_()
    graph.replay()
    sync_ok()
    assert torch.equal(cache, eager_cache)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
