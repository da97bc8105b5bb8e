"""A linear-attention block built from the library's operators, trained and served.

The residual stream r and its norm n go from block to block:

    q, k, v, z = n W_in                              (one projection, columns cut)
    y = linear attention(q, k, v) W_out
    r <- r + alpha gate(z) norm(y);  n <- norm(r)    (one call)

``Block.train`` runs it under autograd on packed sequences, ``Block.prompt`` and
``Block.step`` serve it: prompts of different lengths fill slots of a cache of
states, single tokens continue them.  Run it on a GPU:

    python examples/linear_attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_sequence_chunk_gb300 as ssd  # noqa: E402


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu_seqlens, max_seqlen):
        o, _ = ssd.linattn_fwd(q, k, v, log_decay, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen,
                               return_final_state=False)
        ctx.save_for_backward(q, k, v, log_decay, cu_seqlens)
        ctx.max_seqlen = max_seqlen
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, log_decay, cu = ctx.saved_tensors
        dq, dk, dv, _ = ssd.linattn_bwd(q, k, v, do.contiguous(), log_decay, cu_seqlens=cu,
                                        max_seqlen=ctx.max_seqlen)
        return dq, dk, dv, None, None, None


class BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, r, y, z, w_post, alpha, w_pre, heads):
        kw = dict(z=z, w_post=w_post, alpha=alpha, gate="silu", ngroups=heads)
        r_out, n, rstd = ssd.block_norm_fwd(r, y, w_pre, return_rstd=True, **kw)
        ctx.save_for_backward(r, y, z, w_post, alpha, w_pre, *rstd)
        ctx.heads = heads
        return r_out, n

    @staticmethod
    def backward(ctx, dr_out, dn):
        r, y, z, w_post, alpha, w_pre, *rstd = ctx.saved_tensors
        g = ssd.block_norm_bwd(r, y, w_pre, dr_out.contiguous(), dn.contiguous(), rstd, z=z,
                               w_post=w_post, alpha=alpha, gate="silu", ngroups=ctx.heads)
        return g["dr"], g["dy"], g["dz"], g["dw_post"], g["dalpha"], g["dw_pre"], None


class Block:
    """Width D, H heads of V values, G groups of K keys; bf16, residual stream fp32."""

    def __init__(self, D=512, H=8, G=4, K=64, V=64, device="cuda"):
        self.D, self.H, self.G, self.K, self.V = D, H, G, K, V
        p = lambda *s: (torch.randn(*s, device=device) * s[0] ** -0.5).bfloat16().requires_grad_()
        one = lambda: torch.ones(D, device=device, requires_grad=True)
        self.w_in, self.w_out = p(D, 2 * G * K + H * V + D), p(H * V, D)
        self.w_post, self.alpha, self.w_pre = one(), one(), one()
        self.log_decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=device) / H)
        self.parameters = [self.w_in, self.w_out, self.w_post, self.alpha, self.w_pre]

    def project(self, n):
        x = n @ self.w_in
        T, gk, hv = n.shape[0], self.G * self.K, self.H * self.V
        q, k, v, z = x.split([gk, gk, hv, self.D], 1)
        return q.view(T, self.G, self.K), k.view(T, self.G, self.K), v.view(T, self.H, self.V), z

    def train(self, r, n, cu_seqlens, max_seqlen):
        q, k, v, z = self.project(n)
        o = LinearAttention.apply(q, k, v, self.log_decay, cu_seqlens, max_seqlen)
        y = o.reshape(len(o), -1) @ self.w_out
        return BlockNorm.apply(r, y, z, self.w_post, self.alpha, self.w_pre, self.H)

    def close(self, r, o, z):
        return ssd.block_norm_fwd(r, o.reshape(len(o), -1) @ self.w_out, self.w_pre, z=z, w_post=self.w_post,
                                  alpha=self.alpha, gate="silu", ngroups=self.H)

    @torch.no_grad()
    def prompt(self, r, n, cu_seqlens, max_seqlen, cache, slots):
        """Runs the packed prompts from empty states and leaves theirs in cache[slots]."""
        q, k, v, z = self.project(n)
        o, states = ssd.linattn_fwd(q, k, v, self.log_decay, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
        cache[slots.long()] = states
        return self.close(r, o, z)

    @torch.no_grad()
    def step(self, r, n, cache, slots):
        """One more token for each of the streams in `slots`."""
        q, k, v, z = self.project(n)
        return self.close(r, ssd.linattn_step(q, k, v, self.log_decay, cache, slots=slots), z)


def main():
    torch.manual_seed(0)
    blocks = [Block(), Block()]
    lens = [300, 45, 700]
    cu = torch.tensor([0, 300, 345, 1045], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), blocks[0].D, device="cuda")
    first = torch.ones(blocks[0].D, device="cuda")
    norm = lambda r: ssd.block_norm_fwd(r, torch.zeros_like(r).bfloat16(), first)[1]

    # training: the blocks learn to give back each token's predecessor
    target = torch.roll(x, 1, 0)
    opt = torch.optim.Adam([p for b in blocks for p in b.parameters], lr=1e-2)
    losses = []
    for _ in range(30):
        r, n = x, norm(x)
        for b in blocks:
            r, n = b.train(r, n, cu, max(lens))
        loss = (r - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"training loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    # serving: all but the last 5 tokens of each sequence as prompts, then token by token
    caches = [torch.zeros(4, b.H, b.V, b.K, device="cuda") for b in blocks]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        r, n = x, norm(x)
        for b in blocks:
            r, n = b.train(r, n, cu, max(lens))
        whole = r
    keep = 5
    rows = [(int(cu[s]), lens[s]) for s in range(3)]
    part = torch.cat([torch.arange(a, a + L - keep, device="cuda") for a, L in rows])
    pcu = torch.tensor([0, 295, 335, 1030], dtype=torch.int32, device="cuda")
    r, n = x[part], norm(x[part])
    for b, cache in zip(blocks, caches):
        r, n = b.prompt(r, n, pcu, max(lens), cache, slots)
    worst = (r - whole[part]).norm() / whole[part].norm()
    for i in range(keep):
        at = torch.tensor([a + L - keep + i for a, L in rows], device="cuda")
        r, n = x[at], norm(x[at])
        for b, cache in zip(blocks, caches):
            r, n = b.step(r, n, cache, slots)
        worst = max(worst, (r - whole[at]).norm() / whole[at].norm())
    print(f"prompt and single tokens against one pass: {worst:.2e}")
    return losses, float(worst)


if __name__ == "__main__":
    main()
