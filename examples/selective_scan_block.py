"""A selective-state-space block built from the library's operators, trained and served.

The residual stream r and its norm n go from block to block:

    x, z = n W_in                                    (one projection, columns cut)
    x = silu(short causal convolution of x)
    dt', B, C = x W_x;   dt = dt' W_dt               (columns of one projection)
    y = selective scan(x, dt, A, B, C, D, gate z);   r <- r + y W_out;   n <- norm(r)

``Block.train`` runs it under autograd on packed sequences, ``Block.prompt`` and
``Block.step`` serve it: prompts of different lengths fill slots of two caches (the
convolution's last rows and the scan's states), single tokens continue them.  Run it on
a GPU:

    python examples/selective_scan_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_sequence_chunk_gb300 as ssd  # noqa: E402


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, cu_seqlens):
        o, _ = ssd.short_conv_fwd(x, weight, bias=bias, activation="silu", cu_seqlens=cu_seqlens, return_final_state=False)
        ctx.save_for_backward(x, weight, bias, cu_seqlens)
        return o

    @staticmethod
    def backward(ctx, do):
        x, weight, bias, cu = ctx.saved_tensors
        g = ssd.short_conv_bwd(x, weight, do.contiguous(), bias=bias, activation="silu", cu_seqlens=cu)
        return g["dx"], g["dweight"], g["dbias"], None


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, max_seqlen):
        kw = dict(D=D, z=z, dt_bias=dt_bias, dt_softplus=True, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
        y, _, states = ssd.selscan_fwd(x, dt, A, B, C, return_final_state=False, return_states=True, **kw)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, states)
        ctx.max_seqlen = max_seqlen
        return y

    @staticmethod
    def backward(ctx, dy):
        x, dt, A, B, C, D, z, dt_bias, cu, states = ctx.saved_tensors
        g = ssd.selscan_bwd(x, dt, A, B, C, dy.contiguous(), states, D=D, z=z, dt_bias=dt_bias, dt_softplus=True,
                            cu_seqlens=cu, max_seqlen=ctx.max_seqlen)
        return g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"], None, None


class ResidualNorm(torch.autograd.Function):
    """r + y and its root-mean-square norm: the block norm without the norm after the block."""

    @staticmethod
    def forward(ctx, r, w_pre):
        zero = torch.zeros_like(r)
        r_out, n, rstd = ssd.block_norm_fwd(r, zero, w_pre, return_rstd=True)
        ctx.save_for_backward(r, zero, w_pre, *rstd)
        return n

    @staticmethod
    def backward(ctx, dn):
        r, zero, w_pre, *rstd = ctx.saved_tensors
        g = ssd.block_norm_bwd(r, zero, w_pre, torch.zeros_like(r), dn.contiguous(), rstd)
        return g["dr"], g["dw_pre"]


class Block:
    """Width D, E channels of N states, W taps; one dtype throughout."""

    def __init__(self, D=256, E=512, N=16, W=4, dtype=torch.bfloat16, device="cuda"):
        self.D, self.E, self.N, self.W, self.R = D, E, N, W, max(8, D // 16)
        p = lambda *s: (torch.randn(*s, device=device) * s[0] ** -0.5).to(dtype).requires_grad_()
        f = lambda t: t.to(device=device, dtype=torch.float32).requires_grad_()
        self.w_in, self.w_x, self.w_dt, self.w_out = p(D, 2 * E), p(E, self.R + 2 * N), p(self.R, E), p(E, D)
        self.conv, self.conv_bias = f(torch.randn(E, W) * W ** -0.5), f(torch.zeros(E))
        self.A_log = f(torch.log(torch.arange(1, N + 1).float()).repeat(E, 1))
        self.skip, self.w_pre = f(torch.ones(E)), f(torch.ones(D))
        rate = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(E))
        self.dt_bias = f(rate + torch.log(-torch.expm1(-rate)))
        self.parameters = [self.w_in, self.w_x, self.w_dt, self.w_out, self.conv, self.conv_bias, self.A_log, self.skip,
                           self.w_pre, self.dt_bias]

    def operands(self, x):
        """dt, A, B, C of the convolution's output."""
        R, N = self.R, self.N
        h = x @ self.w_x
        return h[:, :R] @ self.w_dt, -torch.exp(self.A_log), h[:, R:R + N].unflatten(1, (1, N)), h[:, R + N:].unflatten(1, (1, N))

    def train(self, r, n, cu_seqlens, max_seqlen):
        x, z = (n @ self.w_in).split(self.E, 1)
        x = ShortConv.apply(x, self.conv, self.conv_bias, cu_seqlens)
        y = SelectiveScan.apply(x, *self.operands(x), self.skip, z, self.dt_bias, cu_seqlens, max_seqlen)
        r = r + y @ self.w_out
        return r, ResidualNorm.apply(r, self.w_pre)

    def close(self, r, y):
        r = r + y @ self.w_out
        return r, ssd.block_norm_fwd(r, torch.zeros_like(r), self.w_pre)[1]

    @torch.no_grad()
    def prompt(self, r, n, cu_seqlens, max_seqlen, rows, states, slots):
        """Runs the packed prompts from empty states and leaves theirs in rows[slots] and states[slots]."""
        x, z = (n @ self.w_in).split(self.E, 1)
        x, rows[slots.long()] = ssd.short_conv_fwd(x, self.conv, bias=self.conv_bias, activation="silu", cu_seqlens=cu_seqlens)
        y, states[slots.long()] = ssd.selscan_fwd(x, *self.operands(x), D=self.skip, z=z, dt_bias=self.dt_bias, dt_softplus=True,
                                                  cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
        return self.close(r, y)

    @torch.no_grad()
    def step(self, r, n, rows, states, slots):
        """One more token for each of the streams in `slots`."""
        x, z = (n @ self.w_in).split(self.E, 1)
        x = ssd.short_conv_step(x, self.conv, rows, bias=self.conv_bias, activation="silu", slots=slots)
        y = ssd.selscan_step(x, *self.operands(x), states, D=self.skip, z=z, dt_bias=self.dt_bias, dt_softplus=True, slots=slots)
        return self.close(r, y)

    def caches(self, slots, device="cuda"):
        return (torch.zeros(slots, self.W - 1, self.E, device=device, dtype=self.w_in.dtype),
                torch.zeros(slots, self.E, self.N, device=device))


def main(dtype=torch.bfloat16):
    torch.manual_seed(0)
    blocks = [Block(dtype=dtype), Block(dtype=dtype)]
    lens = [300, 45, 700]
    cu = torch.tensor([0, 300, 345, 1045], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), blocks[0].D, device="cuda").to(dtype)
    first = torch.ones(blocks[0].D, device="cuda")
    norm = lambda r: ssd.block_norm_fwd(r, torch.zeros_like(r), first)[1]

    def whole():
        r, n = x, norm(x)
        for b in blocks:
            r, n = b.train(r, n, cu, max(lens))
        return r

    # training: the blocks learn to give back each token's predecessor
    target = torch.roll(x, 1, 0)
    opt = torch.optim.Adam([p for b in blocks for p in b.parameters], lr=2e-3)
    losses = []
    for _ in range(30):
        loss = (whole().float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"training loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    # serving: all but the last 5 tokens of each sequence as prompts, then token by token
    caches = [b.caches(4) for b in blocks]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        want = whole().float()
    keep = 5
    rows = [(int(cu[s]), lens[s]) for s in range(3)]
    part = torch.cat([torch.arange(a, a + L - keep, device="cuda") for a, L in rows])
    pcu = torch.tensor([0, 295, 335, 1030], dtype=torch.int32, device="cuda")
    r, n = x[part], norm(x[part])
    for b, cache in zip(blocks, caches):
        r, n = b.prompt(r, n, pcu, max(lens), *cache, slots)
    worst = (r.float() - want[part]).norm() / want[part].norm()
    for i in range(keep):
        at = torch.tensor([a + L - keep + i for a, L in rows], device="cuda")
        r, n = x[at], norm(x[at])
        for b, cache in zip(blocks, caches):
            r, n = b.step(r, n, *cache, slots)
        worst = max(worst, (r.float() - want[at]).norm() / want[at].norm())
    print(f"prompt and single tokens against one pass: {worst:.2e}")
    return losses, float(worst)


if __name__ == "__main__":
    main()
