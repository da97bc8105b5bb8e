"""The cases in which the linear-attention and block-norm operators are measured.

``run`` makes one pass: with ``own`` false in plain torch operations (32 bits,
rounded once at the end), with ``own`` true through the package's entry points.
``exact`` computes the same outputs from the definitions in 64 bits: the
recurrence token by token, and the norms' gradients written out by hand.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 128
_EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _prompt(name, kind, dtype, seqs, tokens, H, G, K, V, state):
    """kind "prompt" (forward) or "train" (forward and gradients); `tokens` in all,
    packed as `seqs` sequences: of different lengths from three sequences on."""
    return {"name": name, "op": kind, "dtype": dtype, "seqs": seqs, "tokens": tokens, "ragged": seqs > 2,
            "H": H, "G": G, "K": K, "V": V, "state": state}


def listed():
    return [
        # one short prompt: the latency of the chunked form's smallest use
        _prompt("prompt_short", "prompt", "bf16", 1, 33, 8, 8, 128, 64, True),
        # a serving batch of prompts of different lengths, continued from stored states
        _prompt("prompt_packed", "prompt", "bf16", 12, 16384, 32, 32, 128, 128, True),
        # one very long prompt with keys shared by all heads (the long-context workload's sizes)
        _prompt("prompt_long", "prompt", "bf16", 1, 65536, 24, 1, 128, 64, True),
        # fp32 prompts (the small fp32 workload's sizes)
        _prompt("prompt_f32", "prompt", "f32", 2, 4096, 8, 1, 64, 64, True),
        # a training step's forward and gradients on packed documents
        _prompt("train_packed", "train", "bf16", 6, 16384, 16, 16, 128, 128, True),
        # shared keys, head sizes that are not powers of two, odd lengths
        _prompt("train_shared_odd", "train", "bf16", 7, 5003, 12, 3, 96, 80, False),
        # one stream's next token
        {"name": "step_one", "op": "step", "dtype": "bf16", "batch": 1, "slots": 4, "H": 24, "G": 1, "K": 128, "V": 64},
        # 64 streams' next tokens (the decoding workload's sizes), slots in any order
        {"name": "step_batch", "op": "step", "dtype": "bf16", "batch": 64, "slots": 72, "H": 80, "G": 1, "K": 128, "V": 64},
        # the norms around a block for one token, each head a group of the norm after it
        {"name": "norm_token", "op": "norm", "dtype": "bf16", "rdtype": "bf16", "tokens": 1, "D": 5120, "groups": 80, "gate": "silu"},
        # the same for a long prompt, with the residual stream in fp32
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "rdtype": "f32", "tokens": 16384, "D": 5120, "groups": 80, "gate": "silu"},
        # a training step of the norms: forward and gradients
        {"name": "norm_train", "op": "norm_train", "dtype": "bf16", "rdtype": "bf16", "tokens": 16384, "D": 2048, "groups": 1, "gate": "sigmoid"},
        # odd width, fp32
        {"name": "norm_train_f32", "op": "norm_train", "dtype": "f32", "rdtype": "f32", "tokens": 1001, "D": 1544, "groups": 1, "gate": "silu"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "step", "norm", "norm_train"])
    if op in ("prompt", "train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        K, V = rng.choice([16, 32, 64, 80, 96, 128, 128]), rng.choice([16, 48, 64, 64, 112, 128, 128])
        G = rng.choice([1, 2, 3, 5, 8, 16])
        H = G * rng.choice([1, 1, 2, 4])
        cost = (4 if op == "train" else 1) * (4 if dtype == "f32" else 1)
        most = min(65536, int(16384 * 32 * 2 / (H * cost)))
        tokens = _log_int(rng, 1, most)
        seqs = min(tokens, _log_int(rng, 1, 40))
        return {"op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "ragged": rng.random() < 0.8,
                "H": H, "G": G, "K": K, "V": V, "state": rng.random() < 0.7}
    if op == "step":
        G = rng.choice([1, 2, 4])
        batch = _log_int(rng, 1, 64)
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "batch": batch,
                "slots": batch + rng.randrange(1, 9), "H": G * rng.choice([1, 4, 6, 16]), "G": G,
                "K": rng.choice([16, 64, 96, 128]), "V": rng.choice([16, 64, 80, 128])}
    groups = rng.choice([1, 1, 8, 24])
    D = groups * 8 * _log_int(rng, 1, 5120 // (8 * groups))
    dtype, rdtype = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
    return {"op": op, "dtype": dtype, "rdtype": rdtype, "tokens": _log_int(rng, 1, 16384), "D": D,
            "groups": groups, "gate": rng.choice(["silu", "sigmoid"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """Lengths of the packed sequences, from the case alone (so that every seed has the same work)."""
    n, T = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [T // n + (i < T % n) for i in range(n)]
    cuts = sorted(int(T * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _decays(H, dev):
    """log decays -2^(-12 (h+1)/H): memories from about one token to thousands."""
    return -torch.exp2(-12.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)


def _chunks(lens, dev):
    """The plain form's chunk table: token index and validity [n, 128], sequence, first token and length of each chunk."""
    seq, off, ln, first = [], [], [], []
    at = 0
    for s, L in enumerate(lens):
        for c in range(0, L, _CHUNK):
            seq.append(s)
            off.append(c)
            ln.append(min(_CHUNK, L - c))
            first.append(at + c)
        at += L
    t = lambda v: torch.tensor(v, device=dev, dtype=torch.int64)
    i = torch.arange(_CHUNK, device=dev)
    valid = i[None, :] < t(ln)[:, None]
    idx = torch.where(valid, t(first)[:, None] + i[None, :], 0)
    return {"seq": t(seq), "off": t(off), "len": t(ln), "idx": idx, "valid": valid}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
    s = {"case": case}
    op, dt = case["op"], _DT[case["dtype"]]
    if op in ("prompt", "train"):
        H, G, K, V, T = case["H"], case["G"], case["K"], case["V"], case["tokens"]
        lens = _lengths(case)
        # q, k and v are column ranges of one projection's output
        qkv = rnd(T, 2 * G * K + H * V).to(dt)
        s["q"] = qkv[:, :G * K].view(T, G, K)
        s["k"] = qkv[:, G * K:2 * G * K].view(T, G, K)
        s["v"] = qkv[:, 2 * G * K:].view(T, H, V)
        s["log_decay"] = _decays(H, dev)
        s["scale"] = K ** -0.5
        cu = [0]
        for L in lens:
            cu.append(cu[-1] + L)
        s["cu_seqlens"] = torch.tensor(cu, device=dev, dtype=torch.int32)
        s["max_seqlen"] = max(lens)
        s["chunks"] = _chunks(lens, dev)
        s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int64)
        s["init_state"] = rnd(len(lens), H, V, K) if case["state"] else None
        if op == "train":
            s["do"] = rnd(T, H, V).to(dt)
            s["dfinal"] = rnd(len(lens), H, V, K) if case["state"] else None
    elif op == "step":
        b, H, G, K, V = case["batch"], case["H"], case["G"], case["K"], case["V"]
        s["q"], s["k"] = rnd(b, G, K).to(dt), rnd(b, G, K).to(dt)
        s["v"] = rnd(b, H, V).to(dt)
        s["log_decay"], s["scale"] = _decays(H, dev), K ** -0.5
        s["cache"] = rnd(case["slots"], H, V, K)
        slots = torch.randperm(case["slots"], generator=g, device=dev)[:b].to(torch.int32)
        if b > 2:
            slots[b // 2] = -1   # a row of the batch that holds no stream
        s["slots"] = slots
        s["rows"] = torch.nonzero(slots >= 0)[:, 0]
        s["rows_slots"] = slots[s["rows"]].to(torch.int64)
    else:
        T, D, rdt = case["tokens"], case["D"], _DT[case["rdtype"]]
        s["r"], s["y"], s["z"] = rnd(T, D).to(rdt), (0.7 * rnd(T, D)).to(dt), rnd(T, D).to(dt)
        s["w_post"], s["w_pre"] = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
        s["alpha"] = 0.5 + 0.1 * rnd(D)
        if op == "norm_train":
            s["dr_out"], s["dn"] = rnd(T, D).to(rdt), rnd(T, D).to(dt)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_linattn(s, q, k, v, S0):
    """Chunked linear attention on fp32 q, k [T, G, K], v [T, H, V]: o [T, H, V] and the final states."""
    ck, a = s["chunks"], s["log_decay"]
    H, G = v.shape[1], q.shape[1]
    idx, valid = ck["idx"], ck["valid"]
    take = lambda x: torch.where(valid[:, :, None, None], x[idx], 0.0).transpose(1, 2)   # [n, heads, C, dim]
    qc, kc = (take(x).repeat_interleave(H // G, 1) for x in (q, k))
    vc = take(v)
    i = torch.arange(_CHUNK, device=a.device)
    d = i[:, None] - i[None, :]
    M = torch.where(d >= 0, torch.exp(a[:, None, None] * d.clamp(min=0)), 0.0)           # [H, C, C]
    o = ((qc @ kc.transpose(2, 3)) * M) @ vc
    tail = (ck["len"][:, None] - 1 - i).clamp(min=0)                                      # [n, C]
    w = torch.exp(a[None, :, None] * tail[:, None, :])
    U = (vc * w[..., None]).transpose(2, 3) @ kc                                          # [n, H, V, K]
    n = U.shape[0]
    Uh = U.transpose(0, 1).reshape(H, n, -1)
    # states before each chunk, and after each sequence, as one product over earlier chunks
    end = ck["off"] + ck["len"]
    dist = ck["off"][:, None] - end[None, :]
    W = torch.where(((ck["seq"][:, None] == ck["seq"][None, :]) & (dist >= 0))[None],
                    torch.exp(a[:, None, None] * dist.clamp(min=0)), 0.0)
    S = (W @ Uh).reshape(H, n, *U.shape[2:]).transpose(0, 1)
    lens = s["lens"]
    distf = lens[:, None] - end[None, :]
    Wf = torch.where((torch.arange(len(lens), device=a.device)[:, None] == ck["seq"][None, :])[None],
                     torch.exp(a[:, None, None] * distf.clamp(min=0)), 0.0)
    fin = (Wf @ Uh).reshape(H, len(lens), *U.shape[2:]).transpose(0, 1)
    if S0 is not None:
        S = S + torch.exp(a[None, :] * ck["off"][:, None])[..., None, None] * S0[ck["seq"]]
        fin = fin + torch.exp(a[None, :] * lens[:, None])[..., None, None] * S0
    o = o + torch.exp(a[:, None] * (i + 1)[None, :])[None, :, :, None] * (qc @ S.transpose(2, 3))
    return s["scale"] * o.transpose(1, 2)[valid], fin


def _plain_prompt(s):
    dt = s["v"].dtype
    o, fin = _plain_linattn(s, s["q"].float(), s["k"].float(), s["v"].float(), s["init_state"])
    return {"o": o.to(dt), "final_state": fin}


def _plain_train(s):
    dt = s["v"].dtype
    x = [s[n].float().detach().requires_grad_() for n in ("q", "k", "v")]
    S0 = s["init_state"]
    if S0 is not None:
        S0 = S0.detach().requires_grad_()
        x.append(S0)
    o, fin = _plain_linattn(s, x[0], x[1], x[2], S0)
    out, grad = [o], [s["do"].float()]
    if s["dfinal"] is not None:
        out.append(fin)
        grad.append(s["dfinal"])
    d = torch.autograd.grad(out, x, grad)
    return {"o": o.detach().to(dt), "final_state": fin.detach(), "dq": d[0].to(dt), "dk": d[1].to(dt),
            "dv": d[2].to(dt), "dinit": d[3] if S0 is not None else None}


def _plain_step(s):
    H, G = s["v"].shape[1], s["q"].shape[1]
    rows, at, cache = s["rows"], s["rows_slots"], s["cache"]
    q, k = (s[n][rows].float().repeat_interleave(H // G, 1) for n in ("q", "k"))
    v = s["v"][rows].float()
    S = torch.exp(s["log_decay"])[None, :, None, None] * cache[at] + v[..., None] * k[:, :, None, :]
    cache[at] = S
    o = torch.zeros(s["v"].shape, device=v.device, dtype=torch.float32)
    o[rows] = s["scale"] * (S * q[:, :, None, :]).sum(-1)
    return {"o": o.to(s["v"].dtype), "cache": cache}


def _plain_norm(s, r, y, z, w_post, alpha, w_pre):
    c = s["case"]
    T, D = y.shape
    yg = y.view(T, c["groups"], D // c["groups"])
    yh = (yg * torch.rsqrt((yg * yg).mean(-1, keepdim=True) + _EPS)).view(T, D)
    sg = 1.0 / (1.0 + torch.exp(-z))
    gate = z * sg if c["gate"] == "silu" else sg
    rp = r + alpha * gate * w_post * yh
    n = w_pre * rp * torch.rsqrt((rp * rp).mean(-1, keepdim=True) + _EPS)
    return rp, n


_NORM_IN = ("r", "y", "z", "w_post", "alpha", "w_pre")


def _plain_norm_fwd(s):
    rp, n = _plain_norm(s, *(s[k].float() for k in _NORM_IN))
    return {"r_out": rp.to(s["r"].dtype), "n": n.to(s["y"].dtype)}


def _plain_norm_train(s):
    x = [s[k].float().detach().requires_grad_() for k in _NORM_IN]
    rp, n = _plain_norm(s, *x)
    d = torch.autograd.grad([rp, n], x, [s["dr_out"].float(), s["dn"].float()])
    out = {"r_out": rp.detach().to(s["r"].dtype), "n": n.detach().to(s["y"].dtype)}
    out.update({"d" + k: g.to(s[k].dtype) for k, g in zip(_NORM_IN, d)})
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step,
                "norm": _plain_norm_fwd, "norm_train": _plain_norm_train}[op](state)
    import state_space_sequence_chunk_gb300 as ssd
    s = state
    if op in ("prompt", "train"):
        kw = dict(cu_seqlens=s["cu_seqlens"], max_seqlen=s["max_seqlen"], scale=s["scale"],
                  init_state=s["init_state"])
        o, fin = ssd.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], **kw)
        if op == "prompt":
            return {"o": o, "final_state": fin}
        dq, dk, dv, d0 = ssd.linattn_bwd(s["q"], s["k"], s["v"], s["do"], s["log_decay"],
                                         dfinal_state=s["dfinal"], **kw)
        return {"o": o, "final_state": fin, "dq": dq, "dk": dk, "dv": dv, "dinit": d0}
    if op == "step":
        o = ssd.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["cache"], slots=s["slots"],
                             scale=s["scale"])
        return {"o": o, "cache": s["cache"]}
    c = s["case"]
    kw = dict(z=s["z"], w_post=s["w_post"], alpha=s["alpha"], gate=c["gate"], ngroups=c["groups"], eps=_EPS)
    if op == "norm":
        r_out, n = ssd.block_norm_fwd(s["r"], s["y"], s["w_pre"], **kw)
        return {"r_out": r_out, "n": n}
    r_out, n, rstd = ssd.block_norm_fwd(s["r"], s["y"], s["w_pre"], return_rstd=True, **kw)
    g = ssd.block_norm_bwd(s["r"], s["y"], s["w_pre"], s["dr_out"], s["dn"], rstd, **kw)
    return {"r_out": r_out, "n": n, "dr": g["dr"], "dy": g["dy"], "dz": g["dz"],
            "dw_post": g["dw_post"], "dalpha": g["dalpha"], "dw_pre": g["dw_pre"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("prompt", "train"):
        e = 2 if case["dtype"] == "bf16" else 4
        T, H, G, K, V, n = case["tokens"], case["H"], case["G"], case["K"], case["V"], case["seqs"]
        st = 4 * n * H * K * V
        qkv = e * T * (2 * G * K + H * V)
        # the cheapest evaluation: the state's update and its product with q for each token
        fwd_b = qkv + e * T * H * V + st * (2 if case["state"] else 1)
        fwd_f = 4.0 * T * H * K * V
        if op == "prompt":
            return {"bytes": fwd_b, "flops": fwd_f}
        bwd_b = 2 * qkv + e * T * H * V + (3 * st if case["state"] else 0)
        return {"bytes": fwd_b + bwd_b, "flops": fwd_f + 10.0 * T * H * K * V}
    if op == "step":
        e = 2 if case["dtype"] == "bf16" else 4
        b, H, G, K, V = case["batch"], case["H"], case["G"], case["K"], case["V"]
        live = b - (1 if b > 2 else 0)
        return {"bytes": 8 * live * H * K * V + e * b * 2 * (G * K + H * V), "flops": 5.0 * live * H * K * V}
    e, er = (2 if case[k] == "bf16" else 4 for k in ("dtype", "rdtype"))
    n = case["tokens"] * case["D"]
    w = 12 * case["D"]
    if op == "norm":
        return {"bytes": n * (3 * e + 2 * er) + w, "flops": 14.0 * n}
    return {"bytes": n * (3 * e + 2 * er) + n * (5 * e + 3 * er) + 3 * w, "flops": 50.0 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_prompt(s, grads):
    """The recurrence token by token, every sequence and head at once."""
    f = torch.float64
    q, k, v = s["q"].to(f), s["k"].to(f), s["v"].to(f)
    H, hpg = v.shape[1], v.shape[1] // q.shape[1]
    lam = torch.exp(s["log_decay"].to(f))[None, :, None, None]
    lens = s["lens"].tolist()
    first = [0]
    for L in lens:
        first.append(first[-1] + L)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])   # longest first: a step's sequences are a prefix
    dev = q.device
    start = torch.tensor([first[i] for i in order], device=dev)
    S = torch.zeros(len(lens), H, v.shape[2], q.shape[2], dtype=f, device=dev)
    if s["init_state"] is not None:
        S = S + s["init_state"].to(f)[order]
    o = torch.zeros_like(v)
    dqh = torch.zeros(q.shape[0], H, q.shape[2], dtype=f, device=dev) if grads else None
    do = s["do"].to(f) if grads else None
    live = [sum(1 for L in lens if L > t) for t in range(max(lens))]
    for t, m in enumerate(live):
        at = start[:m] + t
        kt, qt = (x[at].repeat_interleave(hpg, 1) for x in (k, q))
        Sm = lam * S[:m] + v[at][..., :, None] * kt[..., None, :]
        S[:m] = Sm
        o[at] = s["scale"] * (Sm @ qt[..., None])[..., 0]
        if grads:
            dqh[at] = s["scale"] * (Sm.transpose(2, 3) @ do[at][..., None])[..., 0]
    back = torch.tensor(order, device=dev).argsort()
    out = {"o": o, "final_state": S[back]}
    if not grads:
        return out
    R = torch.zeros_like(S)
    if s["dfinal"] is not None:
        R = R + s["dfinal"].to(f)[order]
    dkh, dv = torch.zeros_like(dqh), torch.zeros_like(v)
    for t in range(len(live) - 1, -1, -1):
        m = live[t]
        at = start[:m] + t
        kt, qt = (x[at].repeat_interleave(hpg, 1) for x in (k, q))
        Rm = R[:m] + s["scale"] * do[at][..., :, None] * qt[..., None, :]
        dkh[at] = (Rm.transpose(2, 3) @ v[at][..., None])[..., 0]
        dv[at] = (Rm @ kt[..., None])[..., 0]
        R[:m] = lam * Rm
    share = lambda x: x.view(x.shape[0], H // hpg, hpg, -1).sum(2)
    out.update(dq=share(dqh), dk=share(dkh), dv=dv, dinit=R[back] if s["init_state"] is not None else None)
    return out


def _exact_step(s):
    f = torch.float64
    H, G = s["v"].shape[1], s["q"].shape[1]
    cache, o = s["cache"].to(f), torch.zeros(s["v"].shape, dtype=f, device=s["v"].device)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            k, q = (s[n][i].to(f).repeat_interleave(H // G, 0) for n in ("k", "q"))
            cache[slot] = (torch.exp(s["log_decay"].to(f))[:, None, None] * cache[slot]
                           + torch.einsum("hv,hk->hvk", s["v"][i].to(f), k))
            o[i] = s["scale"] * torch.einsum("hvk,hk->hv", cache[slot], q)
    return {"o": o, "cache": cache}


def _exact_norm(s, grads):
    f = torch.float64
    r, y, z, w, al, wn = (s[k].to(f) for k in _NORM_IN)
    c = s["case"]
    T, D = y.shape
    gw = D // c["groups"]
    grouped = lambda x: x.view(T, c["groups"], gw)
    rs = (grouped(y).pow(2).sum(-1) / gw + _EPS).pow(-0.5)[..., None]
    yh = (grouped(y) * rs).view(T, D)
    sg = torch.sigmoid(z)
    gate, dgate = (z * sg, sg + z * sg * (1 - sg)) if c["gate"] == "silu" else (sg, sg * (1 - sg))
    rp = r + al * w * gate * yh
    q = (rp.pow(2).sum(-1, keepdim=True) / D + _EPS).pow(-0.5)
    rh = rp * q
    out = {"r_out": rp, "n": wn * rh}
    if not grads:
        return out
    dn, gr = s["dn"].to(f), s["dr_out"].to(f)
    e = wn * dn
    G = gr + q * (e - rh * (e * rh).sum(-1, keepdim=True) / D)
    dyh = G * al * w * gate
    dy = grouped(dyh) - grouped(yh) * (grouped(dyh * yh).sum(-1, keepdim=True) / gw)
    out.update(dr=G, dy=(dy * rs).view(T, D), dz=G * al * w * yh * dgate,
               dw_post=(G * al * gate * yh).sum(0), dalpha=(G * w * gate * yh).sum(0), dw_pre=(dn * rh).sum(0))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "train"):
        return _exact_prompt(s, op == "train")
    if op == "step":
        return _exact_step(s)
    return _exact_norm(s, op == "norm_train")
