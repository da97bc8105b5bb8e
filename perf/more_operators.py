"""The cases in which the short convolution and the selective scan are measured.

``run`` makes one pass: with ``own`` false in plain torch operations (32 bits,
rounded once at the end), with ``own`` true through the package's entry points.
``exact`` computes the same outputs from the definitions in 64 bits: the
recurrence token by token, and every gradient written out by hand.

Short convolution, per channel, with the W - 1 rows before a sequence from its
initial state (0 without one):
    p_t = bias + sum_k w_k x_{t-W+1+k},      o_t = silu(p_t) or p_t.
Selective scan, per channel with N states:
    d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
    y_t = (C_t . h_t + D x_t) silu(z_t).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _conv(name, op, dtype, seqs, tokens, D, W, act=True, state=True, pad=0):
    return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "pad": pad, "D": D, "W": W,
            "act": act, "state": state}


def _scan(name, op, dtype, seqs, tokens, D, N, G=1, gate=True, state=True, pad=0):
    return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "pad": pad, "D": D, "N": N,
            "G": G, "gate": gate, "state": state}


def listed():
    return [
        # one short prompt: the latency of the convolution's smallest use
        _conv("conv_prompt_short", "conv", "bf16", 1, 33, 5120, 4),
        # a serving batch of prompts of different lengths, continued from stored states
        _conv("conv_prompt_packed", "conv", "bf16", 12, 16384, 5120, 4),
        # a training step's forward and gradients on packed documents
        _conv("conv_train", "conv_train", "bf16", 6, 16384, 2048, 4, state=False),
        # the same in fp32, three taps, no activation, odd lengths and rows of no sequence behind them
        _conv("conv_train_odd", "conv_train", "f32", 7, 5003, 1544, 3, act=False, pad=5),
        # one stream's next token
        {"name": "conv_step_one", "op": "conv_step", "dtype": "bf16", "batch": 1, "slots": 4, "D": 5120, "W": 4, "act": True},
        # 64 streams' next tokens (the decoding workload's sizes), slots in any order
        {"name": "conv_step_batch", "op": "conv_step", "dtype": "bf16", "batch": 64, "slots": 72, "D": 5120, "W": 4, "act": True},
        # one very long prompt (the long-context workload's 24 heads of 64 as channels)
        _scan("scan_prompt_long", "scan", "bf16", 1, 65536, 1536, 16),
        # a serving batch of prompts of different lengths, continued from stored states
        _scan("scan_prompt_packed", "scan", "bf16", 12, 16384, 5120, 16),
        # a training step's forward and gradients on packed documents
        _scan("scan_train", "scan_train", "bf16", 6, 8192, 2048, 16, state=False),
        # fp32, channels in groups, a number of states that is no power of two, odd lengths, rows of no sequence
        _scan("scan_train_odd", "scan_train", "f32", 7, 2501, 1032, 10, G=3, pad=3),
        # one stream's next token
        {"name": "scan_step_one", "op": "scan_step", "dtype": "bf16", "batch": 1, "slots": 4, "D": 5120, "N": 16, "G": 1, "gate": True},
        # 64 streams' next tokens
        {"name": "scan_step_batch", "op": "scan_step", "dtype": "bf16", "batch": 64, "slots": 72, "D": 5120, "N": 16, "G": 1, "gate": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_step":
        batch = _log_int(rng, 1, 64)
        return {"op": op, "dtype": dtype, "batch": batch, "slots": batch + rng.randrange(1, 9),
                "D": 8 * _log_int(rng, 1, 640), "W": rng.choice([2, 3, 4, 4, 5, 8]), "act": rng.random() < 0.7}
    if op == "scan_step":
        G, batch = rng.choice([1, 1, 2, 4]), _log_int(rng, 1, 64)
        return {"op": op, "dtype": dtype, "batch": batch, "slots": batch + rng.randrange(1, 9),
                "D": G * 8 * _log_int(rng, 1, 640 // G), "N": rng.choice([4, 8, 10, 16, 16, 32, 64]), "G": G,
                "gate": rng.random() < 0.7}
    pad = rng.choice([0, 0, 0, 1, 7])
    state = rng.random() < 0.6
    if op in ("conv", "conv_train"):
        D = 8 * _log_int(rng, 4, 640)
        tokens = _log_int(rng, 1, min(65536, 16384 * 5120 // (D * (3 if op == "conv_train" else 1))))
        return _unnamed(_conv("", op, dtype, min(tokens, _log_int(rng, 1, 40)), tokens, D,
                              rng.choice([2, 3, 4, 4, 4, 5, 8]), rng.random() < 0.7, state, pad))
    G, N = rng.choice([1, 1, 1, 2, 3]), rng.choice([4, 8, 10, 16, 16, 16, 32, 64])
    D = G * 8 * _log_int(rng, 4, 640 // G)
    most = (1 << 28 if op == "scan_train" else 1 << 30) // (D * N)
    tokens = _log_int(rng, 1, min(8192 if op == "scan_train" else 65536, most))
    return _unnamed(_scan("", op, dtype, min(tokens, _log_int(rng, 1, 40)), tokens, D, N, G,
                          rng.random() < 0.7, state, pad))


def _unnamed(case):
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """Lengths of the packed sequences, from the case alone (so that every seed has the same work)."""
    n, T = case["seqs"], case["tokens"]
    cuts = sorted(int(T * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _sequences(s, lens, dev):
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    s["lens"] = lens
    s["cu_seqlens"] = torch.tensor(cu, device=dev, dtype=torch.int32)
    s["max_seqlen"] = max(lens)


def _taps(case, lens, dev):
    """The plain convolution's rows: x's, then the initial states', then one of zeros.
    src [T, W] is each token's taps, last [seqs, W - 1] the final states' rows."""
    W, T, n = case["W"], case["tokens"], len(lens)
    total = T + case["pad"]
    none = total + n * (W - 1)
    seq = torch.repeat_interleave(torch.arange(n), torch.tensor(lens))
    start = torch.tensor([0] + lens[:-1]).cumsum(0)

    def rows(seq, pos):   # row of position pos (negative: before the sequence)
        before = total + seq * (W - 1) + (pos + W - 1) if case["state"] else torch.full_like(pos, none)
        return torch.where(pos >= 0, start[seq] + pos, before)

    pos = torch.arange(T) - start[seq]
    src = rows(seq[:, None], pos[:, None] + torch.arange(W)[None, :] - (W - 1))
    q = torch.arange(n)[:, None].expand(n, W - 1)
    last = rows(q, torch.tensor(lens)[:, None] - (W - 1) + torch.arange(W - 1)[None, :])
    return src.to(dev), last.to(dev)


def _chunks(lens, dev):
    """The plain scan's chunks of 64 tokens: token index and validity [n, 64], and for
    each sequence's c-th chunk its number (by c: the sequences that have one, and theirs)."""
    first, ln, at, number, levels = [], [], 0, 0, []
    for s, L in enumerate(lens):
        for c in range(0, L, _CHUNK):
            first.append(at + c)
            ln.append(min(_CHUNK, L - c))
            if c // _CHUNK == len(levels):
                levels.append(([], []))
            levels[c // _CHUNK][0].append(s)
            levels[c // _CHUNK][1].append(number)
            number += 1
        at += L
    t = lambda v: torch.tensor(v, device=dev, dtype=torch.int64)
    i = torch.arange(_CHUNK, device=dev)
    valid = i[None, :] < t(ln)[:, None]
    return {"idx": torch.where(valid, t(first)[:, None] + i[None, :], 0), "valid": valid, "n": number,
            "levels": [(t(a), t(b)) for a, b in levels]}


def _slots(s, g, dev):
    """Which slot each row of the batch continues; one row of a larger batch holds no stream."""
    c = s["case"]
    slots = torch.randperm(c["slots"], generator=g, device=dev)[:c["batch"]].to(torch.int32)
    if c["batch"] > 2:
        slots[c["batch"] // 2] = -1
    s["slots"] = slots
    s["rows"] = torch.nonzero(slots >= 0)[:, 0]
    s["rows_slots"] = slots[s["rows"]].to(torch.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
    s = {"case": case}
    op, dt, D = case["op"], _DT[case["dtype"]], case["D"]
    step = op.endswith("step")
    T = case["batch"] if step else case["tokens"] + case["pad"]
    if not step:
        lens = _lengths(case)
        _sequences(s, lens, dev)
        n = len(lens)
    if op.startswith("conv"):
        W = case["W"]
        # x is the first half of the columns of one projection's output
        s["x"] = rnd(T, 2 * D).to(dt)[:, :D]
        s["weight"], s["bias"] = rnd(D, W) * W ** -0.5, 0.1 * rnd(D)
        if step:
            s["cache"] = rnd(case["slots"], W - 1, D).to(dt)
            _slots(s, g, dev)
            return s
        s["src"], s["last"] = _taps(case, lens, dev)
        s["init_state"] = rnd(n, W - 1, D).to(dt) if case["state"] else None
        if op == "conv_train":
            s["dout"] = rnd(T, D).to(dt)
            s["dfinal"] = rnd(n, W - 1, D).to(dt) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    R = 8 * max(1, D // 128)                  # rank of dt's projection, whose input lies beside B and C
    bc = rnd(T, R + 2 * G * N).to(dt)
    s["B"] = bc[:, R:R + G * N].view(T, G, N)
    s["C"] = bc[:, R + G * N:].view(T, G, N)
    s["x"] = rnd(T, D).to(dt)
    s["dt"] = (0.5 * rnd(T, D)).to(dt)
    s["z"] = rnd(T, 2 * D).to(dt)[:, D:] if case["gate"] else None
    # steps of 0.001 to 0.1 after softplus, decays of 1 to N, both as training leaves them
    rate = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=g, device=dev))
    s["dt_bias"] = rate + torch.log(-torch.expm1(-rate))
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.2 * rnd(D, N))
    s["D"] = 1 + 0.1 * rnd(D)
    if step:
        s["cache"] = rnd(case["slots"], D, N)
        _slots(s, g, dev)
        return s
    s["chunks"] = _chunks(lens, dev)
    s["init_state"] = rnd(n, D, N) if case["state"] else None
    if op == "scan_train":
        s["dout"] = rnd(T, D).to(dt)
        s["dfinal"] = rnd(n, D, N) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_conv(s, x, weight, bias, init):
    """o and the final states, in 32 bits, from 32-bit operands."""
    c = s["case"]
    rows = [x] if init is None else [x, init.reshape(-1, c["D"])]
    rows = torch.cat(rows + [x.new_zeros(1 if init is not None else 1 + len(s["lens"]) * (c["W"] - 1), c["D"])])
    p = bias
    for k in range(c["W"]):
        p = p + weight[:, k] * rows[s["src"][:, k]]
    o = _silu(p) if c["act"] else p
    if c["pad"]:
        o = torch.cat([o, o.new_zeros(c["pad"], c["D"])])
    return o, rows[s["last"]]


def _plain_conv_fwd(s):
    dt = s["x"].dtype
    init = None if s["init_state"] is None else s["init_state"].float()
    o, fin = _plain_conv(s, s["x"].float(), s["weight"], s["bias"], init)
    return {"o": o.to(dt), "final_state": fin.to(dt)}


def _plain_conv_train(s):
    dt = s["x"].dtype
    names = ["x", "weight", "bias"] + (["init_state"] if s["init_state"] is not None else [])
    v = [s[k].float().detach().requires_grad_() for k in names]
    o, fin = _plain_conv(s, v[0], v[1], v[2], v[3] if len(v) > 3 else None)
    outs, grads = [o], [s["dout"].float()]
    if s["dfinal"] is not None:
        outs.append(fin)
        grads.append(s["dfinal"].float())
    d = torch.autograd.grad(outs, v, grads)
    return {"o": o.detach().to(dt), "final_state": fin.detach().to(dt), "dx": d[0].to(dt), "dweight": d[1],
            "dbias": d[2], "dinit_state": d[3].to(dt) if len(v) > 3 else None}


def _plain_conv_step(s):
    c, rows, at, cache = s["case"], s["rows"], s["rows_slots"], s["cache"]
    x = s["x"][rows]
    old = cache[at]
    window = torch.cat([old, x[:, None]], 1)
    p = s["bias"] + (window.float() * s["weight"].t()[None]).sum(1)
    cache[at] = window[:, 1:]
    o = torch.zeros(s["x"].shape, device=x.device, dtype=torch.float32)
    o[rows] = _silu(p) if c["act"] else p
    return {"o": o.to(x.dtype), "cache": cache}


def _plain_scan(s, x, dt, A, B, C, D, dt_bias, z, h0):
    """y and the final states in 32 bits: all chunks side by side, token by token, once
    from zero for their own sums, and again from the states at their starts."""
    c, ck = s["case"], s["chunks"]
    cpg, n, N = c["D"] // c["G"], ck["n"], c["N"]
    m = ck["valid"]
    d = torch.where(m[..., None], _softplus(dt + dt_bias)[ck["idx"]], 0.0)      # [n, 64, D]
    dx = d * torch.where(m[..., None], x[ck["idx"]], 0.0)
    Bc, Cc = (torch.where(m[..., None, None], v[ck["idx"]], 0.0) for v in (B, C))
    wide = lambda v: v.repeat_interleave(cpg, 1)                                 # [n, G, N] -> [n, D, N]
    advance = lambda h, i: torch.exp(d[:, i, :, None] * A) * h + dx[:, i, :, None] * wide(Bc[:, i])
    end = x.new_zeros(n, c["D"], N)
    for i in range(_CHUNK):
        end = advance(end, i)
    whole = torch.exp(d.sum(1)[..., None] * A)
    h = x.new_zeros(len(s["lens"]), c["D"], N) if h0 is None else h0
    starts, numbers = [], []
    for seqs, number in ck["levels"]:
        at = h[seqs]
        starts.append(at)
        numbers.append(number)
        h = h.index_copy(0, seqs, whole[number] * at + end[number])
    hh = torch.cat(starts)[torch.cat(numbers).argsort()]
    y = []
    for i in range(_CHUNK):
        hh = advance(hh, i)
        y.append((hh * wide(Cc[:, i])).sum(-1))
    T = c["tokens"]
    y = torch.stack(y, 1)[m] + D * x[:T]
    if z is not None:
        y = y * _silu(z[:T])
    if c["pad"]:
        y = torch.cat([y, y.new_zeros(c["pad"], c["D"])])
    return y, h


_SCAN_IN = ("x", "dt", "A", "B", "C", "D", "dt_bias", "z", "init_state")


def _plain_scan_fwd(s):
    y, fin = _plain_scan(s, *(None if s[k] is None else s[k].float() for k in _SCAN_IN))
    return {"y": y.to(s["x"].dtype), "final_state": fin}


def _plain_scan_train(s):
    v = {k: s[k].float().detach().requires_grad_() for k in _SCAN_IN if s[k] is not None}
    y, fin = _plain_scan(s, *(v.get(k) for k in _SCAN_IN))
    outs, grads = [y], [s["dout"].float()]
    if s["dfinal"] is not None:
        outs.append(fin)
        grads.append(s["dfinal"])
    d = dict(zip(v, torch.autograd.grad(outs, list(v.values()), grads)))
    out = {"y": y.detach().to(s["x"].dtype), "final_state": fin.detach()}
    out.update({"d" + k: d[k].to(s[k].dtype) if k in d else None for k in _SCAN_IN})
    return out


def _plain_scan_step(s):
    c, rows, at, cache = s["case"], s["rows"], s["rows_slots"], s["cache"]
    x, dt = s["x"][rows].float(), s["dt"][rows].float()
    B, C = (s[k][rows].float().repeat_interleave(c["D"] // c["G"], 1) for k in ("B", "C"))
    d = _softplus(dt + s["dt_bias"])
    h = torch.exp(d[..., None] * s["A"]) * cache[at] + (d * x)[..., None] * B
    cache[at] = h
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][rows].float())
    o = torch.zeros(s["x"].shape, device=x.device, dtype=torch.float32)
    o[rows] = y
    return {"y": o.to(s["x"].dtype), "cache": cache}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"conv": _plain_conv_fwd, "conv_train": _plain_conv_train, "conv_step": _plain_conv_step,
                "scan": _plain_scan_fwd, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step}[op](state)
    import state_space_sequence_chunk_gb300 as ssd
    s, c = state, state["case"]
    if op.startswith("conv"):
        kw = dict(bias=s["bias"], activation="silu" if c["act"] else None)
        if op == "conv_step":
            o = ssd.short_conv_step(s["x"], s["weight"], s["cache"], slots=s["slots"], **kw)
            return {"o": o, "cache": s["cache"]}
        kw.update(cu_seqlens=s["cu_seqlens"], init_state=s["init_state"])
        o, fin = ssd.short_conv_fwd(s["x"], s["weight"], **kw)
        out = {"o": o, "final_state": fin}
        if op == "conv_train":
            d = ssd.short_conv_bwd(s["x"], s["weight"], s["dout"], dfinal_state=s["dfinal"], **kw)
            out.update({k: d[k] for k in ("dx", "dweight", "dbias", "dinit_state")})
        return out
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
    if op == "scan_step":
        y = ssd.selscan_step(*args, s["cache"], slots=s["slots"], **kw)
        return {"y": y, "cache": s["cache"]}
    kw.update(cu_seqlens=s["cu_seqlens"], max_seqlen=s["max_seqlen"])
    if op == "scan":
        y, fin = ssd.selscan_fwd(*args, init_state=s["init_state"], **kw)
        return {"y": y, "final_state": fin}
    y, fin, states = ssd.selscan_fwd(*args, init_state=s["init_state"], return_states=True, **kw)
    d = ssd.selscan_bwd(*args, s["dout"], states, dfinal_state=s["dfinal"],
                        return_dinit=s["init_state"] is not None, **kw)
    out = {"y": y, "final_state": fin}
    out.update({"d" + k: d["d" + k] for k in _SCAN_IN})
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, D = case["op"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    live = case["batch"] - (1 if case["batch"] > 2 else 0) if op.endswith("step") else 0
    if op.startswith("conv"):
        W = case["W"]
        w = 4 * D * (W + 1)
        if op == "conv_step":
            return {"bytes": 2 * e * live * W * D + w, "flops": (2.0 * W + 4) * live * D}
        n, st = case["tokens"] * D, e * case["seqs"] * (W - 1) * D
        fwd_b, fwd_f = 2 * e * n + w + st * (2 if case["state"] else 1), (2.0 * W + 4) * n
        if op == "conv":
            return {"bytes": fwd_b, "flops": fwd_f}
        return {"bytes": fwd_b + 3 * e * n + 2 * w + (3 * st if case["state"] else 0), "flops": fwd_f + (6.0 * W + 10) * n}
    N, G = case["N"], case["G"]
    w = 4 * D * (N + 2)
    io = 4 if case["gate"] else 3            # x, dt, z and y
    if op == "scan_step":
        return {"bytes": 8 * live * D * N + e * live * (io * D + 2 * G * N) + w, "flops": live * D * (7.0 * N + 12)}
    T, st = case["tokens"], 4 * case["seqs"] * D * N
    fwd_b = e * T * (io * D + 2 * G * N) + w + st * (2 if case["state"] else 1)
    fwd_f = T * D * (7.0 * N + 12)
    if op == "scan":
        return {"bytes": fwd_b, "flops": fwd_f}
    # again x, dt, z and dout, B and C; gradients of all but dout
    bwd_b = e * T * ((2 * io - 1) * D + 4 * G * N) + 2 * w + (2 * st if case["state"] else 0)
    return {"bytes": fwd_b + bwd_b, "flops": fwd_f + T * D * (24.0 * N + 30)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
_F = torch.float64


def _bounds(s):
    at = 0
    for L in s["lens"]:
        yield at, at + L
        at += L


def _exact_conv(s, grads):
    c = s["case"]
    W, D, dev = c["W"], c["D"], s["x"].device
    x, w, b = s["x"].to(_F), s["weight"].to(_F), s["bias"].to(_F)
    o = torch.zeros(x.shape, dtype=_F, device=dev)
    dx, dw, db = torch.zeros_like(o), torch.zeros_like(w), torch.zeros_like(b)
    fin, dinit = [], []
    for i, (a, e) in enumerate(_bounds(s)):
        L = e - a
        head = torch.zeros(W - 1, D, dtype=_F, device=dev) if s["init_state"] is None else s["init_state"][i].to(_F)
        ext = torch.cat([head, x[a:e]])
        fin.append(ext[L:])
        dext = torch.zeros_like(ext)
        if grads and s["dfinal"] is not None:
            dext[L:] += s["dfinal"][i].to(_F)
        if L > 0:
            p = b.expand(L, D).clone()
            for k in range(W):
                p += ext[k:k + L] * w[:, k]
            sg = torch.sigmoid(p)
            o[a:e] = p * sg if c["act"] else p
            if grads:
                gr = s["dout"][a:e].to(_F)
                if c["act"]:
                    gr = gr * (sg + p * sg * (1 - sg))
                db += gr.sum(0)
                for k in range(W):
                    dw[:, k] += (gr * ext[k:k + L]).sum(0)
                    dext[k:k + L] += gr * w[:, k]
        dx[a:e] = dext[W - 1:]
        dinit.append(dext[:W - 1])
    out = {"o": o, "final_state": torch.stack(fin)}
    if grads:
        out.update(dx=dx, dweight=dw, dbias=db, dinit_state=torch.stack(dinit) if s["init_state"] is not None else None)
    return out


def _exact_conv_step(s):
    c, cache = s["case"], s["cache"].to(_F)
    o = torch.zeros(s["x"].shape, dtype=_F, device=cache.device)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            ext = torch.cat([cache[slot], s["x"][i:i + 1].to(_F)])
            p = s["bias"].to(_F) + torch.einsum("kd,dk->d", ext, s["weight"].to(_F))
            o[i] = p * torch.sigmoid(p) if c["act"] else p
            cache[slot] = ext[1:]
    return {"o": o, "cache": cache}


def _softplus64(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def _exact_scan(s, grads):
    """Token by token, every sequence at once: longest first, so that a step's sequences are a prefix."""
    c = s["case"]
    cpg, dev = c["D"] // c["G"], s["x"].device
    x, A, Dk = s["x"].to(_F), s["A"].to(_F), s["D"].to(_F)
    v = s["dt"].to(_F) + s["dt_bias"].to(_F)
    d = _softplus64(v)
    B, C = s["B"].to(_F), s["C"].to(_F)
    lens = s["lens"]
    bounds = list(_bounds(s))
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = torch.tensor([bounds[i][0] for i in order], device=dev)
    h = torch.zeros(len(lens), c["D"], c["N"], dtype=_F, device=dev)
    if s["init_state"] is not None:
        h = h + s["init_state"].to(_F)[order]
    y = torch.zeros_like(x)
    live = [sum(1 for L in lens if L > t) for t in range(max(lens))]
    kept = []
    wide = lambda m: m.repeat_interleave(cpg, 1)
    for t, m in enumerate(live):
        at = start[:m] + t
        if grads:
            kept.append(h[:m].clone())
        h[:m] = torch.exp(d[at][..., None] * A) * h[:m] + (d[at] * x[at])[..., None] * wide(B[at])
        y[at] = torch.einsum("bdn,bdn->bd", h[:m], wide(C[at]))
    back = torch.tensor(order, device=dev).argsort()
    inside = torch.zeros(len(x), 1, dtype=_F, device=dev)
    inside[:c["tokens"]] = 1
    y = (y + Dk * x) * inside
    gate = 1.0
    if s["z"] is not None:
        z = s["z"].to(_F)
        sg = torch.sigmoid(z)
        gate = z * sg
    out = {"y": y * gate, "final_state": h[back]}
    if not grads:
        return out
    do = s["dout"].to(_F) * inside
    gy = do * gate
    r = torch.zeros_like(h)
    if s["dfinal"] is not None:
        r = r + s["dfinal"].to(_F)[order]
    dxs, dd = torch.zeros_like(x), torch.zeros_like(x)
    dB, dC, dA = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A)
    group = lambda m: m.view(m.shape[0], c["G"], cpg, c["N"]).sum(2)
    for t in range(len(live) - 1, -1, -1):
        m = live[t]
        at = start[:m] + t
        a, Bt, Ct = torch.exp(d[at][..., None] * A), wide(B[at]), wide(C[at])
        before = kept.pop()
        now = a * before + (d[at] * x[at])[..., None] * Bt
        dC[at] = group(gy[at][..., None] * now)
        rt = r[:m] + gy[at][..., None] * Ct
        u = (rt * Bt).sum(-1)
        w = rt * a * before
        dxs[at] = d[at] * u
        dd[at] = x[at] * u + (A * w).sum(-1)
        dA += (d[at][..., None] * w).sum(0)
        dB[at] = group(rt * (d[at] * x[at])[..., None])
        r[:m] = a * rt
    ddt = dd * torch.sigmoid(v)
    out.update(dx=dxs + Dk * gy, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(gy * x).sum(0), ddt_bias=ddt.sum(0),
               dz=do * y * (sg + z * sg * (1 - sg)) if s["z"] is not None else None,
               dinit_state=r[back] if s["init_state"] is not None else None)
    return out


def _exact_scan_step(s):
    c, cache = s["case"], s["cache"].to(_F)
    y = torch.zeros(s["x"].shape, dtype=_F, device=cache.device)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            x = s["x"][i].to(_F)
            d = _softplus64(s["dt"][i].to(_F) + s["dt_bias"].to(_F))
            B, C = (s[k][i].to(_F).repeat_interleave(c["D"] // c["G"], 0) for k in ("B", "C"))
            cache[slot] = torch.exp(d[:, None] * s["A"].to(_F)) * cache[slot] + (d * x)[:, None] * B
            v = torch.einsum("dn,dn->d", cache[slot], C) + s["D"].to(_F) * x
            if s["z"] is not None:
                z = s["z"][i].to(_F)
                v = v * z * torch.sigmoid(z)
            y[i] = v
    return {"y": y, "cache": cache}


def exact(case, seed):
    if case["op"] == "scan_train" and case["tokens"] * case["D"] * case["N"] > 3 << 28:
        return None   # its states alone would fill 6 GB
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_train"):
        return _exact_conv(s, op == "conv_train")
    if op == "conv_step":
        return _exact_conv_step(s)
    if op in ("scan", "scan_train"):
        return _exact_scan(s, op == "scan_train")
    return _exact_scan_step(s)
