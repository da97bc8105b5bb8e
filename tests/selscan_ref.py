"""Plain 64-bit short convolution and selective scan (numpy, token by token), for the
tests: written from the definitions, sharing nothing with the CUDA path."""
import numpy as np


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def short_conv(x, w, b, lens, act, init=None, dout=None, dfin=None):
    """(out, final) or, with dout, also dx, dw, db, dinit (fp64 arrays)."""
    T, D = x.shape
    W = w.shape[1]
    out, dx, dw, db = np.zeros((T, D)), np.zeros((T, D)), np.zeros((D, W)), np.zeros(D)
    fin, dinit = np.zeros((len(lens), W - 1, D)), np.zeros((len(lens), W - 1, D))
    at = 0
    for s, L in enumerate(lens):
        head = np.zeros((W - 1, D)) if init is None else init[s]
        ext = np.concatenate([head, x[at:at + L]])
        dext = np.zeros_like(ext)
        fin[s] = ext[L:]
        if dfin is not None:
            dext[L:] += dfin[s]
        for t in range(L):
            p = b + sum(w[:, k] * ext[t + k] for k in range(W))
            sg = sigmoid(p)
            out[at + t] = p * sg if act else p
            if dout is not None:
                g = dout[at + t] * (sg * (1 + p * (1 - sg)) if act else 1.0)
                db += g
                for k in range(W):
                    dw[:, k] += g * ext[t + k]
                    dext[t + k] += g * w[:, k]
        dx[at:at + L], dinit[s] = dext[W - 1:], dext[:W - 1]
        at += L
    return (out, fin) if dout is None else (out, fin, dx, dw, db, dinit)


def selscan(x, dt, A, B, C, lens, D=None, z=None, bias=None, softplus=True, h0=None, dout=None, dfin=None):
    """(y, final) or, with dout, also a dict of gradients (fp64 arrays)."""
    T, W = x.shape
    N, G = A.shape[1], B.shape[1]
    per = W // G
    D = np.zeros(W) if D is None else D
    v = dt + (0 if bias is None else bias)
    delta = np.logaddexp(v, 0) if softplus else v
    slope = sigmoid(v) if softplus else np.ones_like(v)
    wide = lambda m: np.repeat(m, per, 0)                        # [G, N] -> [W, N]
    narrow = lambda m: m.reshape(G, per, N).sum(1)
    sz = None if z is None else sigmoid(z)
    y, fin = np.zeros((T, W)), np.zeros((len(lens), W, N))
    g = {k: np.zeros_like(a, dtype=np.float64) for k, a in
         (("dx", x), ("ddt", x), ("dA", A), ("dB", B), ("dC", C), ("dD", D), ("dz", x), ("ddt_bias", D), ("dinit_state", fin))}
    at = 0
    for s, L in enumerate(lens):
        h = np.zeros((W, N)) if h0 is None else h0[s].astype(np.float64)
        hist = [h]
        for t in range(at, at + L):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * wide(B[t])
            hist.append(h)
            y[t] = (h * wide(C[t])).sum(1) + D * x[t]
        fin[s] = h
        if dout is not None:
            q = np.zeros((W, N)) if dfin is None else dfin[s].astype(np.float64)
            for t in range(at + L - 1, at - 1, -1):
                gy = dout[t] * (1.0 if z is None else z[t] * sz[t])
                a = np.exp(delta[t][:, None] * A)
                before, now = hist[t - at], hist[t - at + 1]
                r = q + gy[:, None] * wide(C[t])
                u = (r * wide(B[t])).sum(1)
                w = r * a * before
                dd = x[t] * u + (A * w).sum(1)
                g["dx"][t] = delta[t] * u + D * gy
                g["ddt"][t] = dd * slope[t]
                g["dA"] += delta[t][:, None] * w
                g["dB"][t] = narrow(r * (delta[t] * x[t])[:, None])
                g["dC"][t] = narrow(gy[:, None] * now)
                g["dD"] += gy * x[t]
                if z is not None:
                    g["dz"][t] = dout[t] * y[t] * sz[t] * (1 + z[t] * (1 - sz[t]))
                q = a * r
            g["dinit_state"][s] = q
        at += L
    g["ddt_bias"] = g["ddt"].sum(0)
    if z is not None:
        y = y * z * sz
    y[at:] = 0
    return (y, fin) if dout is None else (y, fin, g)


def off(out, ref) -> float:
    """2-norm of the difference over 2-norm of the reference."""
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    assert out.shape == ref.shape
    d, n = np.linalg.norm(out - ref), np.linalg.norm(ref)
    return float(d if n == 0 else d / n)
