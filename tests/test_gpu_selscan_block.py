"""The example that runs the short convolution and the selective scan together: its
gradients against those of a plain implementation in 64 bits, and prompts followed by
single tokens against one pass."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    path = os.path.join(ROOT, "examples", "selective_scan_block.py")
    spec = importlib.util.spec_from_file_location("selective_scan_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    m = example()
    losses, worst = m.main()
    assert all(torch.isfinite(torch.tensor(losses)))
    # two blocks' bf16 roundings (2^-8 each, six in a block) on either side, in another order of sums
    assert worst < 2 * 6 * 2.0 ** -8
    # fp32: products of a few hundred terms in another order, 2^-24 each
    assert m.main(torch.float32)[1] < 1e-4


def plain(b, r, n, lens):
    """The block token by token in 64 bits, under autograd."""
    x, z = (n @ b["w_in"]).split(b["E"], 1)
    out, at = [], 0
    R, N, W = b["R"], b["N"], b["W"]
    for L in lens:
        ext = torch.cat([x.new_zeros(W - 1, b["E"]), x[at:at + L]])
        p = b["conv_bias"] + sum(ext[k:k + L] * b["conv"][:, k] for k in range(W))
        xs = p * torch.sigmoid(p)
        h = xs @ b["w_x"]
        delta = torch.nn.functional.softplus(h[:, :R] @ b["w_dt"] + b["dt_bias"])
        A, B, C = -torch.exp(b["A_log"]), h[:, R:R + N], h[:, R + N:]
        s = x.new_zeros(b["E"], N)
        for t in range(L):
            s = torch.exp(delta[t][:, None] * A) * s + (delta[t] * xs[t])[:, None] * B[t]
            y = s @ C[t] + b["skip"] * xs[t]
            out.append(y * z[at + t] * torch.sigmoid(z[at + t]))
        at += L
    r = r + torch.stack(out) @ b["w_out"]
    return r, b["w_pre"] * r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-5)


def test_gradients_of_a_block():
    """fp32: every parameter's gradient, through both operators, the projections between them
    and the norm.  Their sums have up to 1e5 terms of 2^-24 each, in random directions, and
    the scan's states are off by at most 2e-5: 1e-4 of the gradient's norm."""
    m = example()
    torch.manual_seed(1)
    block = m.Block(D=64, E=96, N=6, W=3, dtype=torch.float32)
    lens = [33, 1, 26]
    cu = torch.tensor([0, 33, 34, 60], dtype=torch.int32, device="cuda")
    r, n, gr, gn = (torch.randn(60, 64, device="cuda") for _ in range(4))
    for t in (r, n):
        t.requires_grad_()
    out = block.train(r, n, cu, 33)
    got = torch.autograd.grad(out, block.parameters + [r, n], [gr, gn])
    names = ["w_in", "w_x", "w_dt", "w_out", "conv", "conv_bias", "A_log", "skip", "w_pre", "dt_bias"]
    b = {k: getattr(block, k).detach().double().requires_grad_() for k in names}
    r2, n2 = (t.detach().double().requires_grad_() for t in (r, n))
    want_out = plain(dict(b, E=96, R=block.R, N=6, W=3), r2, n2, lens)
    want = torch.autograd.grad(want_out, [b[k] for k in names] + [r2, n2], [gr.double(), gn.double()])
    for k, a, w in zip(["r", "n"], out, want_out):
        assert ((a.double() - w).norm() / w.norm()).item() < 1e-4, k
    for k, a, w in zip(names + ["r", "n"], got, want):
        assert ((a.double() - w).norm() / w.norm()).item() < 1e-4, k
