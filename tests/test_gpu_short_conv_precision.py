"""The short convolution's activation value by value, far from 0."""
import numpy as np
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from test_gpu_selscan_precision import HALF, U, far, near
from test_gpu_selscan import DT, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activations_far_from_zero(dtype):
    """silu(p) and its derivative for p from -200 to 200, of single tokens of weights 0 and 1.  fp32: the
    exponential 5 u, the quotient 1 + 2 u, two products: 12 u allowed; the derivative s + p s (1 - s) 12 u of both
    terms, and where s is nearly 1, p times the 6 u that it is off.  bf16: without the exponential's remainder,
    which takes 1.2 u for each of |p|.  What is below 2^-126 is flushed."""
    x = far(dtype)
    D = len(x)
    dout = torch.randn(1, D, generator=torch.Generator().manual_seed(27)).to(DT[dtype])
    w = torch.tensor([0.0, 1.0]).repeat(D, 1).cuda()
    xin = x[None].cuda()
    o, _ = ssd.short_conv_fwd(xin, w, activation="silu")
    cache = torch.zeros(1, 1, D, device="cuda", dtype=DT[dtype])
    o1 = ssd.short_conv_step(xin, w, cache, activation="silu")
    g = ssd.short_conv_bwd(xin, w, dout.cuda(), bias=torch.zeros(D, device="cuda"), activation="silu")
    P, G = f64(x), f64(dout[0])
    s = np.exp(-np.logaddexp(-P, 0))
    more = 12 + (0 if dtype == "f32" else 1.2 * np.abs(P))
    flush = 2.0 ** -125 * np.abs(P)
    want = P * s
    for v in (o, o1):
        near(v[0], want, (HALF[dtype] + more * U) * np.abs(want) + flush)
    want = G * s * (1 + P * (1 - s))
    slack = np.abs(G) * ((more * s * (1 + np.abs(P) * (1 - s)) + 6 * np.abs(P) * s) * U + flush)
    near(g["dx"][0], want, HALF[dtype] * np.abs(want) + slack)
    near(g["dbias"], want, slack)
