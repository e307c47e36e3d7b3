"""The 2:4 product in every way it is cut (tests/block_cuts.py), with all of its epilogue, against 64-bit sums on the GPU."""
import pytest
import torch

from tests import serve_ref as R
from tests.block_cuts import CUTS
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


@pytest.mark.parametrize("cut,yt", [(c, t) for c in CUTS for t in ((BF, F32) if c[0] < 2 else (BF,))],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, tuple) else str(v)[6:])
def test_every_cut(cut, yt):
    mode, (T, cout, cin) = cut[0], CUTS[cut]
    say("cut", cut, T, cout, cin, yt)
    g = torch.Generator(device=DEV).manual_seed(T + cout)
    W = (0.05 * torch.randn(cout, cin, generator=g, device=DEV)).to(BF)
    perm = torch.rand(cin // 32, 32, generator=g, device=DEV).argsort(-1).int().contiguous()
    nib = torch.tensor([3, 5, 9, 6, 10, 12], device=DEV)[torch.randint(0, 6, (cout, cin // 32, 8), generator=g, device=DEV)]
    word = (nib << (4 * torch.arange(8, device=DEV))).sum(-1)
    bits = torch.where(word >= 1 << 31, word - (1 << 32), word).int().contiguous()
    lin = lcp.SparseLinear.pack(W, perm, bits, dtype=F8 if mode else BF, fast=mode == 2)
    assert lcp.lcp_sparse_linear_cut(lin.p, T) == cut
    keep = ((nib[..., None] >> torch.arange(4, device=DEV)) & 1).view(cout, cin).bool()
    Ws = W[:, (torch.arange(cin // 32, device=DEV)[:, None] * 32 + perm).view(-1)].double() * keep
    del W, nib, word, bits, keep
    x, xs = torch.randn(T, cin, generator=g, device=DEV).to(BF), None
    xv = x.double()
    if mode:
        x, xs, _ = lcp.RMSNorm(torch.ones(cin, device=DEV), dtype=F8)(x)
        xv = x.double() * xs.double()[:, None]
        s = lin.scale.double()[:, None]
        Ws = (Ws / s).to(F32).to(F8).double() * s        # scales are powers of two, codes round to nearest even
    bias = torch.randn(cout, generator=g, device=DEV).to(BF)
    gate = torch.randn(T, 2 * cout, generator=g, device=DEV).to(BF)[:, cout:]
    res = torch.randn(T, cout, generator=g, device=DEV).to(yt)
    buf = torch.full((T + 2, cout + 32), 3.0, device=DEV).to(yt)
    y = buf[1:T + 1, 16:16 + cout]
    need = lcp.lcp_sparse_linear_workspace_bytes(lin.p, T)
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device=DEV)
    lcp.lcp_sparse_linear(lin.p, x, y, x_scale=xs, bias=bias, act="silu", gate=gate, residual=res,
                          ws=ws[:need] if need else None)
    assert bool((ws[need:] == 7).all())                  # nothing behind what was asked for
    # half of cin additions one after the other at most, joins of waves and parts, scales
    v = xv @ Ws.T + bias.double()
    tol = (cin / 2 + 64) * R.U32 * (xv.abs() @ Ws.abs().T) + R.U32 * v.abs()
    if mode == 2:                                        # sixteen products lose less than 2^-13 of their largest each
        top = [torch.nn.functional.pad(a, (0, -cin % 32)).abs().view(len(a), -1, 32).amax(-1) for a in (xv, Ws)]
        tol += 16 * 2.0 ** -13 * (top[0] @ top[1].T)
    # silu: a slope of 1.1 at most, its value good to 12 roundings (fp32) or 2^-15
    tol = 1.1 * tol + (12 * R.U32 if yt == F32 else 2.0 ** -15) * (v * torch.sigmoid(v)).abs()
    v = v * torch.sigmoid(v) * gate.double()
    tol = tol * gate.double().abs() + R.U32 * v.abs()
    v = v + res.double()
    tol += R.U32 * v.abs()
    half = torch.finfo(yt).eps / 2
    assert bool(((y.double() - v).abs() <= tol + half * (v.abs() + tol)).all())
    assert bool((buf[0] == 3).all() and (buf[-1] == 3).all() and (buf[:, :16] == 3).all() and (buf[:, 16 + cout:] == 3).all())
    again = lin(x, scale=xs, bias=bias, act="silu", gate=gate, residual=res, dtype=yt)
    assert torch.equal(again, y)
