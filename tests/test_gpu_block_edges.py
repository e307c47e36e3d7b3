"""Values and calls at the edges of what the documents of a decoder block's operators allow (root-mean-square norm, its
gradient, the 2:4 product with an epilogue), against their 64-bit definitions."""
import pytest
import torch

from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def straight(W, dtype, fast=False):
    """W [cout, cin] packed in its own order, the first two positions of every four kept."""
    cout, cin = W.shape
    perm = torch.arange(32, dtype=torch.int32, device=DEV).repeat(cin // 32, 1)
    bits = torch.full((cout, cin // 32), 0x33333333, dtype=torch.int32, device=DEV)
    return lcp.SparseLinear.pack(W.to(BF), perm, bits, dtype=dtype, fast=fast)


def cancelling(T, cout, cin):
    """W, x and their sums: of every 32 positions two kept products are 2^14 and -2^14, fourteen are 1. Sums are whole
    numbers of at most 256, partial sums below 2^24: exact in fp32 and in a bfloat16 output, in any order."""
    W, x = torch.ones(cout, cin, device=DEV), torch.ones(T, cin, device=DEV)
    W[:, 0::32], W[:, 17::32] = 128.0, -128.0
    x[:, 0::32] = x[:, 17::32] = 128.0
    return W, x, 14 * cin // 32


# ---- the product ----------------------------------------------------------------------
@pytest.mark.parametrize("yt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 16, 64, 65, 129, 333, 700])
@pytest.mark.parametrize("cout,cin", [(64, 512), (288, 96), (4128, 512)])
def test_sums_that_cancel(cout, cin, T, dtype, yt):
    """Small products beside large ones that cancel, whatever the number of tokens."""
    say("cancel", T, cout, cin, dtype, yt)
    W, x, want = cancelling(T, cout, cin)
    y = straight(W, dtype)(x.to(dtype), scale=torch.ones(T, device=DEV) if dtype == F8 else None, dtype=yt)
    assert bool((y == want).all())


@pytest.mark.parametrize("T", [1, 64, 65, 400])
def test_fast_layers(T):
    """fast: fp32 outputs and few tokens stay exact; each of the sixteen products of a lane loses less than 2^-13 of the
    largest of them, so that a group of 32 positions is off by less than 16 * 2^-13 * 2^14 = 32."""
    W, x, want = cancelling(T, 288, 512)
    lin, s = straight(W, F8, fast=True), torch.ones(T, device=DEV)
    assert lin.fast and not straight(W, F8).fast
    assert bool((lin(x.to(F8), scale=s, dtype=F32) == want).all())
    y = lin(x.to(F8), scale=s)
    if T <= 64:
        assert bool((y == want).all())
    else:
        assert bool(((y.float() - want).abs() < 32 * 512 / 32).all())
        g = torch.Generator(device=DEV).manual_seed(T)
        x, W = torch.randn(T, 512, generator=g, device=DEV).to(F8), torch.randn(288, 512, generator=g, device=DEV)
        a, b = straight(W, F8, fast=True), straight(W, F8)
        assert torch.equal(a.vals, b.vals) and torch.equal(a.meta, b.meta) and torch.equal(a.scale, b.scale)
        y, z = a(x, scale=s).double(), b(x, scale=s, dtype=F32).double()
        # the weights' values: one-hot tokens read them back
        eye = b(torch.eye(512, device=DEV).to(F8), scale=torch.ones(512, device=DEV), dtype=F32).double().T
        top = [t.double().abs().view(len(t), -1, 32).amax(-1) for t in (x.float(), eye)]
        tol = 16 * 2.0 ** -13 * (top[0] @ top[1].T) + 2 * (256 + 64) * 2.0 ** -24 * (x.double().abs() @ eye.abs().T)
        assert bool(((y - z).abs() <= tol + 2.0 ** -8 * (z.abs() + tol)).all())
