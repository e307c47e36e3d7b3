"""The gated MLP of a decoder block with 2:4-sparse projections, between its norm and the next one.

    python examples/sparse_mlp_block.py [--hidden 4096] [--inner 11008] [--tokens 1] [--dtype bfloat16|float8_e4m3fn]

Gate and up are pruned as one layer with one learned channel permutation (a few optimisation steps on synthetic
calibration tokens), down with its own; both are hardened and packed for the sparse matrix cores, the rows of gate and
up in the order that down reads, so that no channel is moved between the products:

    h = x + r,  n = norm(h) in gate's and up's channel order (and 8-bit codes)     one launch
      -> up(n) -> silu(gate(n)) * up  [-> 8-bit codes] -> down + h                 a launch each

The result is checked against plain torch in fp32 on the pruned weights, and the norm's gradient against torch's.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import learnable_channel_permutation_amd as lcp  # noqa: E402


def prune(W, X, steps, B=64):
    """(perm [cin / B, B], mask bits [cout, cin / 32]) of a learned channel permutation."""
    nb, dev = W.shape[1] // B, W.device
    s = lcp.LayerSession(W, X, B=B, iters=5, tau=1.0, N=2, M=4, harden=True)
    logits = 3.0 * torch.eye(B, device=dev).repeat(nb, 1, 1)
    if steps > 0:
        s.train(logits, steps=steps, lr=5e-3)
    bits = torch.empty((W.shape[0], W.shape[1] // 32), dtype=torch.int32, device=dev)
    P = torch.empty((nb, B, B), device=dev)
    perm = torch.empty((nb, B), dtype=torch.int32, device=dev)
    s.forward(logits, P_out=P, bits_out=bits)
    lcp.lcp_harden(P, perm=perm)
    return perm, bits


def order(perm):
    """Source channel of every position."""
    return (torch.arange(perm.shape[0], device=perm.device)[:, None] * perm.shape[1] + perm).view(-1).long()


def dense(W, perm, bits):
    """The pruned weight in natural channel order, fp32."""
    keep = ((bits[:, :, None] >> torch.arange(32, device=W.device)) & 1).view(W.shape).bool()
    src = order(perm)
    out = torch.zeros(W.shape, device=W.device)
    out[:, src] = torch.where(keep, W.float()[:, src], 0.0)
    return out


class MlpBlock:
    def __init__(self, hidden, inner, dtype, train_steps, calib, gen):
        dev = calib.device
        self.dtype = dtype
        w = [(k ** -0.5 * torch.randn(n, k, generator=gen, device=dev)).bfloat16()
             for n, k in ((2 * inner, hidden), (hidden, inner))]
        self.weight = (1 + 0.1 * torch.randn(hidden, generator=gen, device=dev)).bfloat16()
        perm, bits = prune(w[0], calib, train_steps)
        gate, up = dense(w[0], perm, bits).split(inner)
        n = lcp.RMSNorm(self.weight)(calib)[0].float()
        acts = (torch.nn.functional.silu(n @ gate.T) * (n @ up.T)).bfloat16()        # what down reads
        perm_down, bits_down = prune(w[1], acts, train_steps)
        self.plain = gate, up, dense(w[1], perm_down, bits_down)
        rows = order(perm_down)
        self.gate, self.up = (lcp.SparseLinear.pack(w[0][i][rows].contiguous(), perm, bits[i][rows].contiguous(), dtype)
                              for i in (slice(inner), slice(inner, None)))
        self.down = lcp.SparseLinear.pack(w[1], perm_down, bits_down, dtype)
        self.norm = lcp.RMSNorm(self.weight, perm=perm, dtype=dtype)

    def __call__(self, x, r):
        """(x + r + MLP(norm(x + r)), the sum x + r) for x, r [T, hidden] bfloat16."""
        n, scale, h = self.norm(x, residual=r)
        a = self.gate(n, scale=scale, act="silu", gate=self.up(n, scale=scale))
        scale = None
        if self.dtype == torch.float8_e4m3fn:
            a, scale = codes(a)
        return self.down(a, scale=scale, residual=h), h


def codes(a):
    """Rows as e4m3 codes and scales by the rule of the operators (include/lcp.h, E4M3 rows), in plain torch: a product's
    epilogue does not see the maximum of a whole row."""
    a = a.float()
    top = a.abs().amax(-1)
    finite = torch.isfinite(top)
    m, e = torch.frexp(torch.where(finite, top, 1.0))
    power = torch.where(top > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    scale = torch.where(finite, torch.ldexp(torch.ones_like(top), power), torch.nan)
    return torch.where(finite[:, None], a / scale[:, None], 0.0).to(torch.float8_e4m3fn), scale


def reference(blk, x, r):
    h = x.float() + r.float()
    n = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * blk.weight.float()
    gate, up, down = blk.plain
    return (torch.nn.functional.silu(n @ gate.T) * (n @ up.T)) @ down.T + h


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=11008)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--dtype", choices=("bfloat16", "float8_e4m3fn"), default="bfloat16")
    ap.add_argument("--train-steps", type=int, default=10)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(7)
    calib = torch.randn(256, a.hidden, generator=gen, device=dev).bfloat16()
    blk = MlpBlock(a.hidden, a.inner, getattr(torch, a.dtype), a.train_steps, calib, gen)
    x, r = (torch.randn(a.tokens, a.hidden, generator=gen, device=dev).bfloat16() for _ in range(2))
    for _ in range(3):
        y, h = blk(x, r)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        blk(x, r)
    torch.cuda.synchronize()
    took = (time.perf_counter() - t0) / 20
    ref = reference(blk, x, r)
    err = float((y.float() - ref).norm() / ref.norm())
    # training: the norm's gradient, with the gradient that the residual stream brings
    dy, dh = (torch.randn(a.tokens, a.hidden, generator=gen, device=dev).bfloat16() for _ in range(2))
    dx, dw = lcp.RMSNorm(blk.weight).backward(h, dy, dsum=dh)
    hp, wp = h.float().requires_grad_(), blk.weight.float().requires_grad_()
    n = hp * (hp.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wp
    gx, gw = torch.autograd.grad((n * dy.float()).sum() + (hp * dh.float()).sum(), (hp, wp))
    grad = max(float((p.float() - q).norm() / q.norm()) for p, q in ((dx, gx), (dw, gw)))
    print("%d tokens, %s: %.0f us a block, off plain torch by %.1e, the norm's gradients by %.1e"
          % (a.tokens, a.dtype, took * 1e6, err, grad))
    return err, grad, y


if __name__ == "__main__":
    main()
