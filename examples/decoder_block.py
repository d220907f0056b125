"""A decoder block on this library: attention over a paged cache, then the
activation-sparse FFN.

    python examples/decoder_block.py            # serve: prompts in chunks, then tokens
    python examples/decoder_block.py --train    # train: a few steps of the head norms

Serving runs sequences of different lengths together: each step appends the new
tokens' keys and values to the cache (heads normalised and rotated on the way),
attends, projects, and passes through the sparse FFN.  At the end the block is
computed once more for whole sequences, in plain float32, and compared.
Training fits the norm weights of q and k to a teacher's, with the library's
forward and backward behind torch's autograd.  The projections are torch
products; weights are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from activation_sparse_feed_amd import sffn  # noqa: E402

EPS = 1e-6


class Block:
    """Weights of one block, bf16."""

    def __init__(self, d_model=512, d_ff=1024, hq=8, hkv=2, dim=64, max_pos=512, beta=1.0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.d_model, self.d_ff, self.hq, self.hkv, self.dim, self.max_pos = \
            d_model, d_ff, hq, hkv, dim, max_pos
        self.qkv = w(d_model, (hq + 2 * hkv) * dim, scale=d_model ** -0.5)
        self.proj = w(hq * dim, d_model, scale=(hq * dim) ** -0.5)
        self.q_norm, self.k_norm = 1 + w(dim, scale=0.2), 1 + w(dim, scale=0.2)
        self.wg, self.wu = w(d_ff, d_model, scale=d_model ** -0.5), w(d_ff, d_model, scale=d_model ** -0.5)
        self.wd = w(d_ff, d_model, scale=d_ff ** -0.5)
        self.bg = torch.full((d_ff,), -beta, device="cuda")
        self.table = sffn.rotary_table(max_pos, dim)


def rms(x):
    """Norm of a token's activations, unit weights."""
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS)).to(x.dtype)


class Server:
    """The block's cache and its steps.  A step's shape (tokens, sequences) fixes
    its buffers; they are kept by shape."""

    def __init__(self, block: Block, lengths, page_size=16):
        self.b, self.page = block, page_size
        self.max_pages = max(-(-n // page_size) for n in lengths)
        n_pages = self.max_pages * len(lengths)
        # every sequence's pages, scattered over the cache
        self.pages = torch.randperm(n_pages, device="cuda").to(torch.int32).view(len(lengths), -1)
        shape = (n_pages, page_size, block.hkv, block.dim)
        self.k = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.done = [0] * len(lengths)
        self.shapes = {}

    def step(self, x, seqs, counts):
        """x: rows of the sequences `seqs`, counts[i] new tokens each, in order."""
        b, T = self.b, x.shape[0]
        key = (T, len(seqs), max(counts))
        if key not in self.shapes:
            attn = sffn.PagedAttention(
                T, len(seqs), b.hq, b.hkv, b.dim, torch.bfloat16, self.page, self.k.shape[0],
                self.max_pages, max(counts), self.max_pages * self.page, rot_dim=b.dim,
                max_pos=b.max_pos, norm=True, eps=EPS, k_cache=self.k, v_cache=self.v)
            self.shapes[key] = attn, sffn.SparseFFN(T, b.d_model, b.d_ff, 32, torch.bfloat16)
        attn, ffn = self.shapes[key]
        pos, seq, starts = [], [], [0]
        for s, n in zip(seqs, counts):
            pos += range(self.done[s], self.done[s] + n)
            seq += [s] * n
            starts.append(starts[-1] + n)
            self.done[s] += n
        pos, seq, starts, lens = (torch.tensor(t, dtype=torch.int32, device="cuda")
                                  for t in (pos, seq, starts, [self.done[s] for s in seqs]))
        bt = self.pages[torch.tensor(seqs, device="cuda")].contiguous()
        qkv = (rms(x) @ b.qkv).view(T, -1, b.dim)
        out = attn.forward(qkv[:, :b.hq], qkv[:, b.hq:b.hq + b.hkv], qkv[:, b.hq + b.hkv:], pos,
                           sffn.paged_slots(self.pages, seq, pos, self.page), starts, lens, bt,
                           b.table, b.q_norm, b.k_norm)
        x = x + out.view(T, -1) @ b.proj
        return x + ffn.forward(rms(x), b.wg, b.bg, b.wu, b.wd)


def plain(b: Block, x):
    """The block over one whole sequence, float32."""
    T = x.shape[0]
    qkv = (rms(x) @ b.qkv).float().view(T, -1, b.dim)

    def rotated(h, w):
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w.float()
        c, s = b.table[:T, None, :b.dim // 2], b.table[:T, None, b.dim // 2:]
        a, z = h[..., :b.dim // 2], h[..., b.dim // 2:]
        return torch.cat([a * c - z * s, z * c + a * s], -1)

    g = b.hq // b.hkv
    q = rotated(qkv[:, :b.hq], b.q_norm).permute(1, 0, 2)
    k = rotated(qkv[:, b.hq:b.hq + b.hkv], b.k_norm).permute(1, 2, 0).repeat_interleave(g, 0)
    v = qkv[:, b.hq + b.hkv:].permute(1, 0, 2).repeat_interleave(g, 0)
    p = q.contiguous() @ k.contiguous() * b.dim ** -0.5
    p = p.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -torch.inf).softmax(-1)
    x = x + ((p @ v.contiguous()).permute(1, 0, 2).reshape(T, -1) @ b.proj.float()).to(x.dtype)
    h = rms(x).float()
    h = torch.relu(h @ b.wg.float().T + b.bg) * (h @ b.wu.float().T)
    return x + (h @ b.wd.float()).to(x.dtype)


def serve(lengths=(150, 37, 90), chunk=48, tokens=6, seed=0):
    """Prompts of `lengths` in chunks, a sequence that is through its prompt taking
    single tokens meanwhile; returns the largest relative error of a sequence."""
    b = Block(seed=seed)
    total = [n + tokens for n in lengths]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    xs = [torch.randn((n, b.d_model), generator=g, device="cuda").to(torch.bfloat16) for n in total]
    srv = Server(b, total)
    ys = [[] for _ in total]
    while any(d < n for d, n in zip(srv.done, total)):
        seqs = [s for s, n in enumerate(total) if srv.done[s] < n]
        counts = [min(chunk, lengths[s] - srv.done[s]) if srv.done[s] < lengths[s] else 1 for s in seqs]
        x = torch.cat([xs[s][srv.done[s]:srv.done[s] + n] for s, n in zip(seqs, counts)])
        y = srv.step(x, seqs, counts)
        for s, part in zip(seqs, y.split(counts)):
            ys[s].append(part)
    worst = 0.0
    for x, y in zip(xs, ys):
        want, got = plain(b, x).float() - x.float(), torch.cat(y).float() - x.float()
        worst = max(worst, ((got - want).norm() / want.norm()).item())
    return worst


class RotatedHeads(torch.autograd.Function):
    """qk_norm_rope under autograd: q and k [T, heads, dim], float32 norm weights."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions):
        heads = sffn.make_heads(q.shape[0], q.shape[1], k.shape[1], q.shape[2], q.dtype,
                                table.shape[1], table.shape[0], True, EPS)
        wq, wk = q_weight.to(q.dtype), k_weight.to(q.dtype)
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        sffn.qk_norm_rope(heads, q, k, wq, wk, table, positions, q_out, k_out)
        ctx.heads = heads
        ctx.save_for_backward(q, k, wq, wk, table, positions)
        return q_out, k_out

    @staticmethod
    def backward(ctx, gq_out, gk_out):
        q, k, wq, wk, table, positions = ctx.saved_tensors
        gq, gk = torch.empty_like(gq_out), torch.empty_like(gk_out)
        gwq, gwk = (torch.empty(w.shape, dtype=torch.float32, device=w.device) for w in (wq, wk))
        sffn.qk_norm_rope_bwd(ctx.heads, q, k, wq, wk, table, positions, gq_out.contiguous(),
                              gk_out.contiguous(), gq, gk, gwq, gwk,
                              sffn.alloc_heads_workspace(ctx.heads))
        return gq, gk, gwq, gwk, None, None


def train(steps=60, T=256, lr=0.1, seed=0):
    """Fits norm weights to a teacher's; returns the first and the last loss."""
    b = Block(seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    wq = torch.ones(b.dim, device="cuda", requires_grad=True)
    wk = torch.ones(b.dim, device="cuda", requires_grad=True)
    losses = []
    for _ in range(steps):
        qkv = torch.randn((T, b.hq + b.hkv, b.dim), generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.randint(0, b.max_pos, (T,), generator=g, device="cuda").to(torch.int32)
        q, k = qkv[:, :b.hq], qkv[:, b.hq:]
        with torch.no_grad():
            tq, tk = RotatedHeads.apply(q, k, b.q_norm.float(), b.k_norm.float(), b.table, pos)
        yq, yk = RotatedHeads.apply(q, k, wq, wk, b.table, pos)
        loss = (yq.float() - tq.float()).square().mean() + (yk.float() - tk.float()).square().mean()
        gwq, gwk = torch.autograd.grad(loss, (wq, wk))
        with torch.no_grad():
            wq -= lr * b.dim / 2 * gwq
            wk -= lr * b.dim / 2 * gwk
        losses.append(loss.item())
    return losses[0], losses[-1]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--train", action="store_true")
    if p.parse_args().train:
        first, last = train()
        print(f"loss of the head norms: {first:.3e} -> {last:.3e}")
    else:
        print(f"served against whole sequences: relative error {serve():.2e}")


if __name__ == "__main__":
    main()
