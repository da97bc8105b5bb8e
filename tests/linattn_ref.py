"""Plain 64-bit linear attention and block norms (numpy, token by token), for the
tests: written from the definitions, sharing nothing with the CUDA path."""
import numpy as np


def linattn(q, k, v, a, lens, scale, S0=None, dout=None, dfin=None):
    """o, final states and, with dout, dq, dk, dv, dS0 (fp64 arrays)."""
    T, G, K = q.shape
    H, V = v.shape[1:]
    hpg = H // G
    lam = np.exp(np.minimum(a.astype(np.float64), 0.0))
    o = np.zeros((T, H, V))
    fin = np.zeros((len(lens), H, V, K))
    dq, dk, dv, d0 = np.zeros((T, G, K)), np.zeros((T, G, K)), np.zeros((T, H, V)), np.zeros_like(fin)
    at = 0
    for s, L in enumerate(lens):
        for h in range(H):
            g = h // hpg
            S = np.zeros((V, K)) if S0 is None else S0[s, h].astype(np.float64)
            for t in range(at, at + L):
                S = lam[h] * S + np.outer(v[t, h], k[t, g])
                o[t, h] = scale * S @ q[t, g]
                if dout is not None:
                    dq[t, g] += scale * S.T @ dout[t, h]
            fin[s, h] = S
            if dout is None:
                continue
            R = np.zeros((V, K)) if dfin is None else dfin[s, h].astype(np.float64)
            for t in range(at + L - 1, at - 1, -1):
                R = R + scale * np.outer(dout[t, h], q[t, g])
                dk[t, g] += R.T @ v[t, h]
                dv[t, h] = R @ k[t, g]
                R = lam[h] * R
            d0[s, h] = R
        at += L
    return (o, fin) if dout is None else (o, fin, dq, dk, dv, d0)


def block_norm(r, y, w_pre, z=None, w_post=None, alpha=None, gate=None, ngroups=1, eps=1e-5,
               dr_out=None, dn=None):
    """(r_out, n) and, with gradients given, a dict of gradients (fp64 arrays)."""
    T, D = y.shape
    one = np.ones(D)
    wp, al = (one if w is None else w for w in (w_post, alpha))
    yg = y.reshape(T, ngroups, -1)
    rs = 1 / np.sqrt((yg ** 2).mean(-1, keepdims=True) + eps)
    yh = (yg * rs).reshape(T, D)
    if gate is None:
        ga, dga = np.ones_like(y), np.zeros_like(y)
    else:
        sg = 1 / (1 + np.exp(-z))
        ga, dga = (z * sg, sg * (1 + z * (1 - sg))) if gate == "silu" else (sg, sg * (1 - sg))
    ro = r + al * wp * ga * yh
    q = 1 / np.sqrt((ro ** 2).mean(-1, keepdims=True) + eps)
    rh = ro * q
    if dn is None:
        return ro, w_pre * rh
    e = w_pre * dn
    g = dr_out + q * (e - rh * (e * rh).mean(-1, keepdims=True))
    u = g * al * wp * ga
    m = (u * yh).reshape(T, ngroups, -1).mean(-1, keepdims=True)
    dy = (rs * (u.reshape(yg.shape) - yh.reshape(yg.shape) * m)).reshape(T, D)
    E = (g * ga * yh).sum(0)
    return ro, w_pre * rh, dict(dr=g, dy=dy, dz=g * al * wp * yh * dga, dw_pre=(dn * rh).sum(0),
                                dw_post=al * E, dalpha=wp * E)


def off(out, ref) -> float:
    """2-norm of the difference over 2-norm of the reference."""
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    assert out.shape == ref.shape
    d, n = np.linalg.norm(out - ref), np.linalg.norm(ref)
    return float(d if n == 0 else d / n)
