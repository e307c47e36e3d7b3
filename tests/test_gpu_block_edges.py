"""Values and calls at the edges of what the documents of a decoder block's operators allow (root-mean-square norm, its
gradient, the 2:4 product with an epilogue), against their 64-bit definitions."""
import math
import warnings

import numpy as np
import pytest
import torch

from tests import block_ref as B
from tests import serve_ref as R
from tests.gpu_util import DEV, down, say

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


# ---- the norm and its gradient ----------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [33, 640, 4097, 20000])
def test_small_elements_beside_large_ones(C, dtype):
    """Rows whose squares pass fp32's range, with elements 2^-140 of the largest and weights that bring them back."""
    say("small beside large", C, dtype)
    g = torch.Generator().manual_seed(5)
    x = 1e-12 * torch.randn(4, C, generator=g)
    x[0, 7], x[1, 9], x[2, 0], x[3, C - 1] = 1e30, -3e37, 2e20, 1.0
    x, w = x.to(dtype), torch.full((C,), 1e20)
    y, _, _ = lcp.RMSNorm(w.to(DEV), 1e-6, dtype=F32)(x.to(DEV))
    ref, _, tol = B.rms_norm(x.double().numpy(), None, w.double().numpy(), 1e-6)
    # an element whose normalised value n is subnormal is off by half of fp32's least number, times the weight
    low = 2.0 ** -150 * w.double().numpy()
    assert np.all(np.abs(down(y) - ref) <= tol + R.U32 * np.abs(ref) + low)
    dy = 1e-25 * torch.randn(4, C, generator=g)
    dy[:, 5] = 1e15
    dx, dw = lcp.RMSNorm(torch.ones(C, device=DEV), 1e-6).backward(x.float().to(DEV), dy.to(DEV))
    rx, rw, tx, tw = B.rms_norm_bwd(x.double().numpy(), dy.double().numpy(), None, np.ones(C), 1e-6)
    assert np.all(np.abs(down(dx) - rx) <= tx + R.U32 * np.abs(rx) + 2.0 ** -148)
    assert np.all(np.abs(down(dw) - rw) <= tw + R.U32 * np.abs(rw) + 2.0 ** -149 * np.abs(dy.double().numpy()).sum(0))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [33, 4097, 8192, 11008, 28672])
def test_rows_of_the_largest_numbers(C, dt):
    """Every element near fp32's largest: the factor is 2^-127 or less and keeps 21 bits, off by 2^-22 at most."""
    say("largest numbers", C, dt)
    g = torch.Generator().manual_seed(9)
    h = 3.3e38 * (1 - 0.2 * torch.rand(3, C, generator=g)) * torch.sign(torch.randn(3, C, generator=g))
    h[1] *= 0.3
    h, dy = h.to(dt), torch.randn(3, C, generator=g).to(dt)
    w = torch.rand(C, generator=g) + 0.5
    norm = lcp.RMSNorm(w.to(DEV), 1e-6, dtype=F32)
    ref, _, tol = B.rms_norm(h.double().numpy(), None, w.double().numpy(), 1e-6)
    y = down(norm(h.to(DEV))[0])
    assert np.all(np.abs(y - ref) <= tol + (R.U32 + 2.0 ** -22) * np.abs(ref))
    dx, dw = norm.backward(h.to(DEV), dy.to(DEV))
    rx, rw, tx, tw = B.rms_norm_bwd(h.double().numpy(), dy.double().numpy(), None, w.double().numpy(), 1e-6)
    # dx is about 1e-38: its rounding is half a step, eps / 2 of a normal number and half of the least of a subnormal one
    half, least = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert np.all(np.abs(down(dx) - rx) <= tx + (2.0 ** -20 + half) * np.abs(rx) + least)
    assert np.all(np.abs(down(dw) - rw) <= tw + R.U32 * np.abs(rw) + 2.0 ** -22 * 3 * np.abs(dy.double().numpy()).sum(0))


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-40, 3e-43, 1.5e-45])
def test_subnormal_eps(eps):
    """Any eps above 0, beside rows whose mean square is as small, or whose squares are no fp32 numbers at all."""
    say("subnormal eps", eps)
    C, e = 640, float(np.float32(eps))
    g = torch.Generator().manual_seed(6)
    x, dy = torch.randn(9, C, generator=g), torch.randn(9, C, generator=g)
    x *= torch.tensor([1.0, 1e25, 1e-12, 1e-19, 1e-20, 3e-21, 1e-22, 1e-30, 1e-41])[:, None]
    x[3, 5] = 0
    w = torch.rand(C, generator=g) + 0.5
    norm = lcp.RMSNorm(w.to(DEV), eps)
    y = down(norm(x.to(DEV))[0])
    ref, _, tol = B.rms_norm(x.double().numpy(), None, w.double().numpy(), e)
    assert np.all(np.abs(y - ref) <= tol + R.U32 * np.abs(ref))
    dy[6:] *= 1e-5                                       # the factor is 1e22 there
    dx, dw = norm.backward(x.to(DEV), dy.to(DEV))
    rx, rw, tx, tw = B.rms_norm_bwd(x.double().numpy(), dy.double().numpy(), None, w.double().numpy(), e)
    assert np.all(np.abs(down(dx) - rx) <= tx + R.U32 * np.abs(rx))
    assert np.all(np.abs(down(dw) - rw) <= tw + R.U32 * np.abs(rw))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [256, 4097, 20000])
def test_gradient_of_large_elements_and_large_gradients(C, dt):
    """Sums of dy h past fp32's range whose means with the normalised h are ordinary numbers."""
    say("large gradient", C, dt)
    g = torch.Generator().manual_seed(8)
    h, dy = torch.randn(6, C, generator=g), torch.randn(6, C, generator=g)
    h *= torch.tensor([3e16, 1e28, 1e-15, 1e17, 1.0, 1e30])[:, None]
    dy *= torch.tensor([3e25, 1e35, 1e15, 1e30, 1e36, 1.0])[:, None]
    h[3] = h[3].abs()
    dy[3] = dy[3].abs()                                  # the sum does not cancel
    h, dy, w = h.to(dt), dy.to(dt), torch.rand(C, generator=g) + 0.5
    dx, dw = lcp.RMSNorm(w.to(DEV), 1e-6).backward(h.to(DEV), dy.to(DEV))
    rx, rw, tx, tw = B.rms_norm_bwd(h.double().numpy(), dy.double().numpy(), None, w.double().numpy(), 1e-6)
    half = torch.finfo(dt).eps / 2
    assert np.isfinite(rx).all() and np.isfinite(rw).all()
    assert np.all(np.abs(down(dx) - rx) <= tx + half * (np.abs(rx) + tx))
    assert np.all(np.abs(down(dw) - rw) <= tw + R.U32 * np.abs(rw))
    dy[1, 3] = float("inf")                              # and what is not finite stays so, in its row alone
    dx2, _ = lcp.RMSNorm(w.to(DEV), 1e-6).backward(h.to(DEV), dy.to(DEV))
    assert not bool(torch.isfinite(dx2[1]).any())
    assert torch.equal(dx2[[0, 2, 3, 4, 5]], dx[[0, 2, 3, 4, 5]])


def guarded(n, dtype):
    """(the whole buffer, n elements inside it): what lies around them is 7 in every byte."""
    size = torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n * size + 512,), 7, dtype=torch.uint8, device=DEV)
    return buf, buf[256:256 + n * size].view(dtype)


def untouched(buf):
    return bool((buf[:256] == 7).all() and (buf[-256:] == 7).all())


@pytest.mark.parametrize("dt,wt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bf16", "bf16-f32", "f32", "f32-bf16"])
@pytest.mark.parametrize("T,C", [(1, 1), (1, 3), (2, 33), (65, 1025), (300, 521), (1100, 322), (9, 4097), (3, 8190), (3, 11007),
                                 (2, 28670), (2, 32767), (2, 32768)])
def test_nothing_around_the_gradients_outputs(T, C, dt, wt):
    """What lies around dx, dweight and the workspace, also where rows end inside the last thread's elements; and the
    results, to tolerances of the sums as they are made: a thread adds 32 of 32768 elements (1024 threads), then six steps
    of its wave and at most sixteen waves."""
    say("gradient guards", T, C, dt, wt)
    g = torch.Generator().manual_seed(C)
    h, dy = (torch.randn(T, C, generator=g).to(dt) for _ in range(2))
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(wt)
    need = lcp.lcp_rms_norm_bwd_workspace_bytes(T, C)
    (bx, dx), (bw, dw), (bs, ws) = guarded(T * C, dt), guarded(C, wt), guarded(need, torch.uint8)
    lcp.lcp_rms_norm_bwd(h.to(DEV), w.to(DEV), dy.to(DEV), dx.view(T, C), dw, ws, eps=1e-5)
    assert untouched(bx) and untouched(bw) and untouched(bs)
    h, dy, w = (t.double().numpy() for t in (h, dy, w))
    s = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-5)
    n, gw = h * s, dy * w
    rx, rw = s * (gw - n * (gw * n).mean(-1, keepdims=True)), (dy * n).sum(0)
    adds, part = 32 + 6 + 16, np.abs(gw * n).mean(-1, keepdims=True)
    # s: half of its sum's roundings, a mean, a root, a division; the mean of g n: its sum's and five products'; three more
    tx = R.U32 * s * ((adds / 2 + 8) * np.abs(gw) + (1.5 * adds + 20) * np.abs(n) * part)
    # terms by s and three products; a workgroup's rows one after the other, then 32 shares of the workgroups and their join
    rows = -(-T // min(T, 256)) + 1024 // 32 + 32
    tw = (adds / 2 + 10 + rows) * R.U32 * np.abs(dy * n).sum(0)
    for got, want, tol, t in ((down(dx).reshape(T, C), rx, tx, dt), (down(dw), rw, tw, wt)):
        half = torch.finfo(t).eps / 2
        assert np.all(np.abs(got - want) <= tol + half * (np.abs(want) + tol) + 2.0 ** -140)


@pytest.mark.parametrize("xt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,C,Bs", [(1, 1, 0), (3, 33, 0), (70, 1025, 0), (5, 4096, 64), (5, 4097, 0), (3, 13824, 128), (2, 32767, 0),
                                    (2, 32768, 64), (5000, 96, 32)])
def test_nothing_around_the_norms_outputs(T, C, Bs, xt):
    """What lies around the codes, their scales and the sum; and fp32 outputs to a tolerance of the sums as they are made."""
    say("norm guards", T, C, Bs, xt)
    g = torch.Generator().manual_seed(C)
    x, r = (torch.randn(T, C, generator=g).to(xt) for _ in range(2))
    w = 1 + 0.3 * torch.randn(C, generator=g)
    perm = torch.stack([torch.randperm(Bs, generator=g) for _ in range(C // Bs)]).int() if Bs else None
    p = None if perm is None else perm.to(DEV)
    (by, y), (bc, scale), (bs, total) = guarded(T * C, torch.uint8), guarded(T, F32), guarded(T * C, xt)
    lcp.lcp_rms_norm(x.to(DEV), w.to(DEV), y.view(F8).view(T, C), scale=scale, residual=r.to(DEV), sum_out=total.view(T, C),
                     perm=p, eps=1e-5)
    assert untouched(by) and untouched(bc) and untouched(bs)
    b32, y32 = guarded(T * C, F32)
    lcp.lcp_rms_norm(x.to(DEV), w.to(DEV), y32.view(T, C), residual=r.to(DEV), perm=p, eps=1e-5)
    assert untouched(b32)
    ref, h, _ = B.rms_norm(x.double().numpy(), r.double().numpy(), w.double().numpy(), 1e-5, None if perm is None else perm.numpy())
    y32 = down(y32).reshape(T, C)
    # half of the sum's roundings (54 additions, as above, of squares of h rounded once), the factor's four, h's and two products'
    tol = ((32 + 6 + 16) / 2 + 9) * R.U32 * np.abs(ref) + 2.0 ** -140
    assert np.all(np.abs(y32 - ref) <= tol)
    half = torch.finfo(xt).eps / 2
    assert np.all(np.abs(down(total).reshape(T, C) - h) <= (R.U32 + half) * (1 + R.U32) * np.abs(h))
    codes, s = R.quantise(y32.astype(np.float32), "fp8")               # of the very numbers that the kernel rounds
    assert np.array_equal(y.view(T, C).cpu().numpy(), codes) and np.array_equal(scale.cpu().numpy(), s)


def test_inputs_that_ask_for_a_gradient():
    """Results have no graph, and the caller is told so where the call stands; not under no_grad, nor of plain inputs."""
    x, w = torch.randn(3, 64, device=DEV), torch.ones(64, device=DEV)
    lin, y = straight(torch.randn(32, 64, device=DEV), BF), torch.empty(3, 64, device=DEV)
    xb, bias = x.to(BF), torch.zeros(32, device=DEV).to(BF)

    def ask(t):
        return t.detach().clone().requires_grad_()

    calls = [lambda f: lcp.RMSNorm(w)(f(x)), lambda f: lcp.RMSNorm(f(w))(x), lambda f: lcp.RMSNorm(w)(x, residual=f(x)),
             lambda f: lcp.lcp_rms_norm(f(x), w, y), lambda f: lin(f(xb)), lambda f: lin(xb, bias=f(bias)),
             lambda f: lin(xb, gate=f(bias.expand(3, 32).contiguous())), lambda f: lin(xb, residual=f(x[:, :32].contiguous()))]
    for call in calls:
        with pytest.warns(UserWarning, match="autograd") as seen:
            call(ask)
        assert seen[0].filename == __file__
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(lambda t: t)
            with torch.no_grad():
                call(ask)
            with pytest.raises(UserWarning):
                call(ask)


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


@pytest.mark.parametrize("T,yt", [(1, F32), (1, BF), (40, F32), (70, BF), (70, F32), (300, BF), (300, F32), (2000, BF)])
def test_scales_whose_product_passes_fp32(T, yt):
    """A row's scale 2^110 and tokens' of 2^30 and 2^-126: sums of 0 and of 2^-18 (the smallest codes' product). And
    2^-126 for both, where nothing is left of a sum."""
    say("scales", T, yt)
    W = torch.zeros(64, 512, device=DEV)
    W[:, 0], W[:, 1] = 1.75 * 2.0 ** 118, 2.0 ** 101
    W[32:] *= 2.0 ** -118                                # their scale: 2^-8
    lin = straight(W, F8)
    assert bool((lin.scale[:32] == 2.0 ** 110).all()) and bool((lin.scale[32:] == 2.0 ** -8).all())
    x, s = torch.zeros(T, 512, device=DEV), torch.full((T,), 2.0 ** 30, device=DEV)
    x[::2, 1] = 2.0 ** -9                                # W's code there is 2^-9, too
    s[4::4] = 2.0 ** -126
    y = lin(x.to(F8), scale=s, dtype=yt)
    want = torch.where(x[:, 1:2] > 0, 2.0 ** -18 * s[:, None], torch.zeros((), device=DEV)).expand(T, 64).double()
    want = want * lin.scale.double()
    want[:, 32:][s == 2.0 ** -126] = 0                   # 2^-18 2^-126 2^-8: nothing of it in fp32
    assert bool(torch.isfinite(want).all()) and float(want.max()) == 2.0 ** 122
    assert torch.equal(y.double(), want)
    lin = straight(torch.zeros(64, 512, device=DEV), F8)
    y = lin(torch.full((T, 512), 448.0, device=DEV).to(F8), scale=torch.full((T,), 2.0 ** -126, device=DEV), dtype=yt)
    assert bool((y == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 0.0])
@pytest.mark.parametrize("T", [3, 70, 300])
def test_token_scales_that_are_no_powers_of_two(T, bad):
    """Any number is a scale: the product of two fractions is rounded once, and NaN, infinity and 0 are what they are."""
    g = torch.Generator(device=DEV).manual_seed(T)
    lin = straight(torch.randn(64, 96, generator=g, device=DEV), F8)
    x = torch.randn(T, 96, generator=g, device=DEV).to(F8)
    s = torch.rand(T, generator=g, device=DEV) + 0.3
    one = lin(x, scale=torch.ones(T, device=DEV), dtype=F32)
    y = lin(x, scale=s, dtype=F32).double()
    want = one.double() * s.double()[:, None]
    assert bool(((y - want).abs() <= 2.0 ** -24 * 1.01 * 2 * want.abs()).all())      # the fractions' product and the sum's
    s[T // 2] = bad
    z = lin(x, scale=s, dtype=F32)[T // 2]
    row = one[T // 2] * bad
    assert torch.equal(z.isnan(), row.isnan()) and torch.equal(z[~row.isnan()], row[~row.isnan()])


@pytest.mark.parametrize("yt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_relative_to_their_values(act, yt):
    """From -86 to 40, tails and all. fp32: one unit in the last place (two roundings) each of the exponential and the
    reciprocal, one of its correction, at most three of a polynomial of fitted error 0.3 * 2^-24 and three products: 12.
    bf16: 2^-15 of an exponent that is rounded, and the output's rounding."""
    say("activation", act, yt)
    T = 2048
    g = torch.Generator().manual_seed(7)
    v = torch.cat([torch.linspace(-86, 40, T * 3), torch.linspace(-14, 14, T * 4), 0.01 * torch.randn(T, generator=g)])
    hi = v.view(8, T).T.to(BF)
    lo = (v.view(8, T).T - hi.float()).to(BF)            # two products that are added exactly: 16 bits of v
    x, W = torch.zeros(T, 32, dtype=BF), torch.zeros(32, 32)
    x[:, 0::4], x[:, 1::4] = hi, lo
    for i in range(8):
        W[i, 4 * i:4 * i + 2] = 1
    z = hi.double().numpy() + lo.double().numpy()
    if act == "silu":
        ref = np.where(z < 0, z * np.exp(z) / (1 + np.exp(z)), z / (1 + np.exp(-np.abs(z))))
    elif act == "gelu":
        ref = 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2))
    else:
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        ref = np.where(z < 0, z * np.exp(np.minimum(u, 0)) / (1 + np.exp(np.minimum(u, 0))), z / (1 + np.exp(-np.abs(u))))
    tol = 12 * 2.0 ** -24 if yt == F32 else 2.0 ** -15 * (1 + 2.0 ** -8) + 2.0 ** -8
    lin = straight(W.to(DEV), BF)
    for n in (1, 40, T):
        rows = torch.arange(0, T, max(1, T // n))[:n]
        y = down(lin(x[rows].to(DEV), act=act, dtype=yt))[:, :8]
        r = ref[rows.numpy()]
        assert np.all(np.abs(y - r) <= tol * np.abs(r) + 2.0 ** -118)


def operands(T, cout, cin, dtype, seed):
    """(layer, x, scale) of random numbers, in the weights' own order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    W, x, s = 0.1 * torch.randn(cout, cin, generator=g, device=DEV), torch.randn(T, cin, generator=g, device=DEV), None
    lin = straight(W, dtype)
    if dtype == F8:
        x, s, _ = lcp.RMSNorm(torch.ones(cin, device=DEV), dtype=F8)(x)
    else:
        x = x.to(BF)
    return lin, x, s


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [2, 17, 64, 100, 400, 1300])
def test_rows_that_share_memory(T, dtype):
    """One row for all tokens (stride 0) as x, gate and residual gives what T copies of it give."""
    lin, x, s = operands(1, 544, 352, dtype, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    gate, res = (torch.randn(1, 544, generator=g, device=DEV).to(BF) for _ in range(2))
    s = None if s is None else s.expand(T).contiguous()
    for yt in (BF, F32):
        kw = dict(scale=s, act="silu", dtype=yt)
        want = lin(x.repeat(T, 1), gate=gate.repeat(T, 1), residual=res.repeat(T, 1), **kw)
        assert torch.equal(lin(x.expand(T, -1), gate=gate.expand(T, -1), residual=res.expand(T, -1), **kw), want)


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 40, 300, 1000])
def test_position_words_at_any_word(T, dtype):
    """meta begins at a multiple of 4 bytes, as it may."""
    lin, x, s = operands(T, 544, 1056, dtype, 5)
    for yt in (BF, F32):
        want = lin(x, scale=s, dtype=yt)
        for off in (1, 2, 3):
            m = torch.empty(lin.meta.numel() + 4, dtype=torch.int32, device=DEV)[off:off + lin.meta.numel()]
            m.copy_(lin.meta)
            assert torch.equal(lcp.SparseLinear(lin.vals, m, 544, 1056, lin.scale)(x, scale=s, dtype=yt), want)


@pytest.mark.parametrize("fast", [False, True], ids=["exact", "fast"])
@pytest.mark.parametrize("yt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 19, 70, 400])
def test_nan_codes(T, yt, fast):
    """A NaN code at a kept position makes its token's outputs NaN where the weight is kept (0 times NaN, too), and no other's;
    at a pruned one it is not read."""
    W = torch.randn(64, 288, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    lin = straight(W, F8, fast=fast)
    _, x, s = operands(T, 32, 288, F8, 7)
    clean = lin(x, scale=s, dtype=yt)
    bad = x.clone()
    bad.view(torch.uint8)[T // 2, 161] = 0x7f            # position 1 of its group: kept
    bad.view(torch.uint8)[0, 6] = 0xff                   # position 2: pruned
    y = lin(bad, scale=s, dtype=yt)
    assert bool(torch.isnan(y[T // 2]).all())
    rest = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(y[rest], clean[rest]) and bool(torch.isfinite(clean).all())


def test_one_token_of_any_stride():
    """The stride of a single row is no address: it may be anything, also where more rows would have to be aligned."""
    for dtype in (BF, F8):
        lin, x, s = operands(1, 96, 64, dtype, 8)
        want = lin(x, scale=s)
        for stride in (0, 1, 67, 1 << 39):
            out = torch.zeros(1, 96, dtype=BF, device=DEV)
            got = lin(x.as_strided((1, 64), (stride, 1)), scale=s, residual=out.as_strided((1, 96), (stride, 1)),
                      out=out.as_strided((1, 96), (stride, 1)))
            assert torch.equal(got, want) and torch.equal(out, want)
    x, w = torch.randn(1, 77, device=DEV), torch.ones(77, device=DEV)
    want, _, _ = lcp.RMSNorm(w)(x)
    dx, dw = lcp.RMSNorm(w).backward(x, x)
    for stride in (0, 1, 1 << 39):
        v = x.as_strided((1, 77), (stride, 1))
        y = torch.empty(77, device=DEV).as_strided((1, 77), (stride, 1))
        assert torch.equal(lcp.RMSNorm(w)(v, out=y)[0], want)
        a, b = lcp.RMSNorm(w).backward(v, v, dx=y)
        assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("Bs", [32, 64, 128])
def test_orders_are_read_modulo_their_blocks(Bs):
    """Entries beyond a block or below 0, in the norm and in both packings."""
    C = 384
    g = torch.Generator().manual_seed(Bs)
    perm = torch.stack([torch.randperm(Bs, generator=g) for _ in range(C // Bs)])
    other = perm + Bs * torch.randint(-3, 4, perm.shape, generator=g)
    other[0, 0] = perm[0, 0] - (1 << 31)
    perm, other = perm.int().to(DEV), other.int().to(DEV)
    x, w = torch.randn(5, C, generator=g).to(BF).to(DEV), torch.rand(C, generator=g).to(DEV)
    W, bits = torch.randn(64, C, generator=g).to(BF).to(DEV), torch.full((64, C // 32), 0x66666666, dtype=torch.int32, device=DEV)
    for dtype in (BF, F8):
        a, b = (lcp.RMSNorm(w, perm=p, dtype=dtype)(x) for p in (perm, other))
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and (a[1] is None or torch.equal(a[1], b[1]))
        a, b = (lcp.SparseLinear.pack(W, p, bits, dtype=dtype) for p in (perm, other))
        assert torch.equal(a.vals, b.vals) and torch.equal(a.meta, b.meta)
