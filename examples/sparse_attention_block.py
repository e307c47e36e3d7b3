"""One attention block of a decoder served with 2:4-sparse projections.

    python examples/sparse_attention_block.py [--hidden 4096] [--prompt 512] [--steps 16]

The fused Q/K/V projection and the output projection are pruned with a learned
channel permutation (a few optimisation steps on synthetic calibration tokens),
hardened and packed for the sparse matrix cores. A prompt is written into a
paged fp8 cache, read back for its own attention (plain torch), and new tokens
are then decoded for a batch of sequences that share the prompt:

    x -> deployed Q/K/V -> rotary positions + quantised cache write (one launch)
      -> attention over the pages -> deployed output projection

The last step is checked against plain torch on the values that the cache holds.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import learnable_channel_permutation_amd as lcp  # noqa: E402


class SparseLinear:
    """A linear layer pruned to 2:4 with a learned channel permutation and packed for deployment."""

    def __init__(self, W, X, steps, B=64):
        self.cout, self.cin = W.shape
        self.B = B
        nb, dev = self.cin // B, W.device
        s = lcp.LayerSession(W, X, B=B, iters=5, tau=1.0, N=2, M=4, harden=True)
        logits = 3.0 * torch.eye(B, device=dev).repeat(nb, 1, 1)
        if steps > 0:
            s.train(logits, steps=steps, lr=5e-3)
        bits = torch.empty((self.cout, self.cin // 32), dtype=torch.int32, device=dev)
        P = torch.empty((nb, B, B), device=dev)
        self.perm = torch.empty((nb, B), dtype=torch.int32, device=dev)
        self.error = s.forward(logits, P_out=P, bits_out=bits).item()
        lcp.lcp_harden(P, perm=self.perm)
        vb, mb = lcp.lcp_sparse_pack_bytes(self.cout, self.cin)
        self.vals = torch.empty(vb, dtype=torch.uint8, device=dev)
        self.meta = torch.empty(mb // 4, dtype=torch.int32, device=dev)
        lcp.lcp_sparse_pack(W, B, self.perm, bits, self.vals, self.meta)

    def __call__(self, x):
        xp, y = torch.empty_like(x), x.new_empty((x.shape[0], self.cout))
        lcp.lcp_deploy_forward(self.vals, self.meta, self.perm, self.B, x, self.cout, xp, y)
        return y


class AttentionBlock:
    """Rotary grouped-query attention over a paged cache between two sparse projections."""

    def __init__(self, hidden, heads, kv_heads, pages, page_size, max_pos, train_steps, calib, gen):
        self.hq, self.hk, self.D = heads, kv_heads, hidden // heads
        dev = calib.device

        def weight(n):
            return (0.02 * torch.randn(n, hidden, generator=gen, device=dev)).bfloat16()

        self.qkv = SparseLinear(weight((heads + 2 * kv_heads) * self.D), calib, train_steps)
        self.out = SparseLinear(weight(hidden), calib, train_steps)
        self.cache = lcp.PagedKVCache.empty(pages, page_size, kv_heads, self.D, device=dev)
        self.table = torch.empty((max_pos, self.D // 2, 2), device=dev)
        lcp.lcp_rope_table(lcp.make_rope_cfg(self.D, base=500000.0), self.table)

    def write(self, x, slots, pos):
        """Project tokens, rotate, and write their keys and values: the rotated queries."""
        n = [self.hq * self.D, self.hk * self.D, self.hk * self.D]
        q, k, v = (y.unflatten(1, (-1, self.D)) for y in self.qkv(x).split(n, 1))
        return self.cache.append(k, v, slots, q=q, q_out=torch.empty_like(q), table=self.table, pos=pos)

    def prompt(self, x, slots, pos):
        """A prompt's causal attention on the values the cache holds (plain torch, fp32)."""
        q = self.write(x, slots, pos).float().transpose(0, 1)
        k, v = (y.float().transpose(0, 1).repeat_interleave(self.hq // self.hk, 0) for y in self.cache.read(slots))
        z = torch.matmul(q, k.transpose(1, 2).contiguous()) * self.D ** -0.5
        z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(1), float("-inf"))
        return self.out(torch.matmul(z.softmax(-1), v).transpose(0, 1).flatten(1).bfloat16())

    def decode(self, x, slots, pos, pages, lens, max_len):
        """One new token of each sequence."""
        o, _ = self.cache.attend(self.write(x, slots, pos), pages, lens, max_len=max_len)
        return self.out(o.flatten(1)), o


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--page-size", type=int, default=64)
    ap.add_argument("--train-steps", type=int, default=10)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(7)
    ps, T = a.page_size, a.prompt
    shared, own = T // ps, -(-(T + a.steps) // ps) - T // ps      # whole pages of the prompt are shared
    calib = torch.randn(256, a.hidden, generator=gen, device=dev).bfloat16()
    blk = AttentionBlock(a.hidden, a.heads, a.kv_heads, shared + a.batch * own, ps, T + a.steps, a.train_steps, calib,
                         gen)
    pages = torch.cat([torch.arange(shared, device=dev).expand(a.batch, -1),
                       shared + torch.arange(a.batch * own, device=dev).view(a.batch, own)], 1).int().contiguous()

    def slots_of(b, t):
        return pages[b, t // ps] * ps + (t % ps).int()

    # the prompt: its last, partly filled page is written for every sequence
    x = torch.randn(T, a.hidden, generator=gen, device=dev).bfloat16()
    t = torch.arange(T, device=dev)
    blk.prompt(x, slots_of(0, t).contiguous(), t.int())
    tail = t[shared * ps:]
    for b in range(1, a.batch if len(tail) else 1):
        blk.write(x[shared * ps:], slots_of(b, tail).contiguous(), tail.int())

    rows = torch.arange(a.batch, device=dev)
    took = 0.0
    for i in range(a.steps):
        x = torch.randn(a.batch, a.hidden, generator=gen, device=dev).bfloat16()
        pos = torch.full((a.batch,), T + i, device=dev)
        slots, lens = slots_of(rows, pos).contiguous(), (pos + 1).int()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y, o = blk.decode(x, slots, pos.int(), pages, lens, T + i + 1)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    # the last step's attention in plain torch, on what the cache holds
    q = blk.write(x, slots, pos.int()).float()
    n, err = T + a.steps, 0.0
    for b in range(a.batch):
        k, v = (z.float().repeat_interleave(a.heads // a.kv_heads, 1)
                for z in blk.cache.read(slots_of(b, torch.arange(n, device=dev)).contiguous()))
        p = ((q[b] * k).sum(-1) * blk.D ** -0.5).softmax(0)
        ref = (p[..., None] * v).sum(0)
        err = max(err, float((o[b].float() - ref).norm() / ref.norm()))
    print("decoded %d steps of %d sequences after a prompt of %d: output %s, last step %.0f us, attention off plain "
          "torch by %.1e" % (a.steps, a.batch, T, tuple(y.shape), took * 1e6, err))
    return err, y


if __name__ == "__main__":
    main()
