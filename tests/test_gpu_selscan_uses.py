"""How the short convolution and the selective scan are used beside other work: captured in
a graph and replayed on new inputs, on streams of their own, two at once, with the caller's
own outputs and workspace, refusals that leave everything as it was."""
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd

pytestmark = pytest.mark.gpu
T, D, N, W = 900, 96, 16, 4
LENS = [500, 0, 396]


def operands(seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    n = len(LENS)
    cu = [0]
    for L in LENS:
        cu.append(cu[-1] + L)
    return dict(x=rnd(T, D).to(dtype), dt=(rnd(T, D) - 2).to(dtype), B=rnd(T, 1, N).to(dtype), C=rnd(T, 1, N).to(dtype),
                z=rnd(T, D).to(dtype), dout=rnd(T, D).to(dtype), A=-rnd(D, N).abs() - 0.1, D=rnd(D), bias=rnd(D), h0=rnd(n, D, N),
                dfin=rnd(n, D, N), w=rnd(D, W), b=rnd(D), init=rnd(n, W - 1, D).to(dtype), cfin=rnd(n, W - 1, D).to(dtype),
                cache=rnd(T, D, N), rows=rnd(T, W - 1, D).to(dtype),
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                slots=torch.randperm(T, generator=g, device="cuda").to(torch.int32))


def everything(d):
    """One call of each entry point; the caches are changed in place."""
    ck = dict(bias=d["b"], activation="silu")
    o, cf = ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"], init_state=d["init"], **ck)
    cg = ssd.short_conv_bwd(d["x"], d["w"], d["dout"], cu_seqlens=d["cu"], init_state=d["init"], dfinal_state=d["cfin"], **ck)
    s1 = ssd.short_conv_step(d["x"], d["w"], d["rows"], slots=d["slots"], **ck)
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    sk = dict(D=d["D"], z=d["z"], dt_bias=d["bias"], dt_softplus=True)
    y, f, st = ssd.selscan_fwd(*a, cu_seqlens=d["cu"], init_state=d["h0"], return_states=True, **sk)
    g = ssd.selscan_bwd(*a, d["dout"], st, cu_seqlens=d["cu"], dfinal_state=d["dfin"], return_dinit=True, **sk)
    s2 = ssd.selscan_step(*a, d["cache"], slots=d["slots"], **sk)
    # (`st` has rows that belong to no sequence and are not written)
    return [o, cf, *cg.values(), s1, d["rows"], y, f, *g.values(), s2, d["cache"]]


def test_captured_and_replayed():
    d = operands(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything({k: v.clone() for k, v in d.items()})     # first calls load modules
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    live = {k: v.clone() for k, v in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(live)
    for seed in (1, 2, 1):
        new = operands(seed)
        for k in live:
            live[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, everything(new)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    ins = [operands(3), operands(4)]
    want = [[t.clone() for t in everything({k: v.clone() for k, v in d.items()})] for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        runs = [{k: v.clone() for k, v in d.items()} for d in ins]
        torch.cuda.synchronize()
        for d, s in zip(runs, streams):
            with torch.cuda.stream(s):
                got.append(everything(d))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_callers_buffers():
    d = operands(5, torch.float32)
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    kw = dict(dt_softplus=True, cu_seqlens=d["cu"], init_state=d["h0"])
    y, f = ssd.selscan_fwd(*a, **kw)
    out, fin, ws = torch.empty_like(y), torch.empty_like(f), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    y2, f2 = ssd.selscan_fwd(*a, out=out, final_out=fin, workspace=ws, **kw)
    assert y2 is out and f2 is fin and torch.equal(y, y2) and torch.equal(f, f2)
    o, c = ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"])
    o2, c2 = ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"], out=out, final_out=torch.empty_like(c))
    assert o2 is out and torch.equal(o, o2) and torch.equal(c, c2)
    # without final states
    assert ssd.selscan_fwd(*a, return_final_state=False, **kw)[1] is None
    assert torch.equal(ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"], return_final_state=False)[0], o)


def test_refusals_change_nothing():
    d = operands(6)
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    cache = d["cache"].clone()
    bad = [lambda: ssd.selscan_step(*a, d["cache"], out=d["x"]),                       # y in x
           lambda: ssd.selscan_fwd(*a, dt_softplus=True, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: ssd.selscan_fwd(*a, nseqs=7),                                       # 7 does not divide 900
           lambda: ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=d["cu"], init_state=d["init"], final_out=d["init"]),
           lambda: ssd.short_conv_step(d["x"][1:], d["w"], d["rows"], out=d["x"][:-1])]
    for f in bad:
        with pytest.raises(ssd.SSDError):
            f()
    with pytest.raises(ValueError):
        ssd.selscan_step(*a, d["cache"].cpu())
    with pytest.raises(TypeError):
        ssd.selscan_fwd(d["x"].half(), *a[1:])
    with pytest.raises(ValueError):
        ssd.short_conv_fwd(d["x"][:, ::2], d["w"])                                     # columns not side by side
    torch.cuda.synchronize()
    assert torch.equal(cache, d["cache"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_that_are_not_what_they_should_be(dtype):
    """Offsets past the rows, negative or falling lead to no read or write outside the tensors
    (they are clamped): the rows behind the outputs keep their guard values."""
    d = operands(7, dtype)
    for cu in ([0, 5000, 6000, 7000], [-5, 400, 200, 2000], [0, 900, 0, 900]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        buf = torch.full((T + 8, D), 3.0, device="cuda").to(dtype)
        y = buf[:T]
        ssd.selscan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], cu_seqlens=cu, init_state=d["h0"], out=y)
        ssd.short_conv_fwd(d["x"], d["w"], cu_seqlens=cu, init_state=d["init"], out=y)
        _, _, st = ssd.selscan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], cu_seqlens=cu, return_states=True)
        ssd.selscan_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dout"], st, cu_seqlens=cu, return_dinit=True)
        ssd.short_conv_bwd(d["x"], d["w"], d["dout"], cu_seqlens=cu, init_state=d["init"])
        torch.cuda.synchronize()
        assert (buf[T:] == 3.0).all()


def test_step_offsets_past_32_bits():
    """A cache of more than 2^31 numbers: the last slot's row against a small cache's."""
    D, N, slots = 8192, 64, 4200
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dt, B, C, A = rnd(2, D), rnd(2, D), rnd(2, 1, N), rnd(2, 1, N), -rnd(D, N).abs()
    cache = torch.zeros(slots, D, N, device="cuda")
    cache[-1] = rnd(D, N)
    small = cache[-2:].clone()
    s = torch.tensor([slots - 2, slots - 1], dtype=torch.int32, device="cuda")
    y = ssd.selscan_step(x, dt, A, B, C, cache, dt_softplus=True, slots=s)
    w = ssd.selscan_step(x, dt, A, B, C, small, dt_softplus=True)
    assert torch.equal(y, w) and torch.equal(cache[-2:], small)
