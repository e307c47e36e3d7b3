"""Serving operators (rotary positions, paged key/value cache, one-token
attention) against their 64-bit definitions, at the sizes, strides and masks
where they can go wrong. Tolerances follow from the roundings each operator
makes (U32: the unit roundoff of fp32); bfloat16 outputs have to be the rounding
of a number within the fp32 tolerance."""
import math

import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.gpu_util import DEV, down, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")

FMT = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def dev_f32(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)


# ---- rotary positions ---------------------------------------------------------
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_parts"])
@pytest.mark.parametrize("rot", [2, 20, 128])
def test_rope_table(scaling, rot):
    if scaling == "base" and rot == 2:
        pytest.skip("the raised base needs more than one pair")
    say("rope table", scaling, rot)
    kw = dict(base=50000.0, scaling=scaling, factor=4.0, orig_len=2048)
    n = 9001
    t = torch.full((n, rot // 2, 2), 7.0, device=DEV)
    lcp.lcp_rope_table(lcp.make_rope_cfg(rot, magnitude=1.25, **kw), t)
    ref = R.rope_table(n, R.rope_theta(rot, **kw), 1.25)
    # one rounding to fp32 of a value up to 1.25, and the 64-bit angle's error (9001 * 2^-50) far below it
    assert np.abs(down(t) - ref).max() <= 1.25 * R.U32 + 1e-10


def rope_case(T, H, D, layout, dtype, seed):
    """Rows [T][H][D] in a memory layout: their own tensor, a slice of a wider
    row, head-major, an odd offset and stride, or one token broadcast."""
    g = torch.Generator().manual_seed(seed)
    if layout == "own":
        x = torch.randn(T, H, D, generator=g).to(dtype).to(DEV)
    elif layout == "packed":
        x = torch.randn(T, (H + 3) * D, generator=g).to(dtype).to(DEV)[:, D:(H + 1) * D].view(T, H, D)
    elif layout == "head-major":
        x = torch.randn(H, T, D, generator=g).to(dtype).to(DEV).transpose(0, 1)
    elif layout == "odd":
        x = torch.randn(T * (H * D + 5) + 1, generator=g).to(dtype).to(DEV)[1:].view(T, H * D + 5)[:, :H * D]
        x = x.unflatten(1, (H, D))
    else:
        x = torch.randn(1, H, D, generator=g).to(dtype).to(DEV).expand(T, H, D)
    return x


ROPE = [  # T, hq, hk, D, rot, layout
    (1, 1, 0, 2, 2, "own"), (1, 3, 1, 64, 64, "own"), (7, 5, 0, 6, 4, "own"), (3, 32, 8, 128, 128, "packed"),
    (65, 4, 2, 128, 64, "head-major"), (33, 6, 6, 80, 32, "own"), (17, 3, 1, 80, 80, "packed"),
    (9, 7, 2, 80, 40, "packed"), (19, 5, 5, 256, 256, "packed"), (6, 2, 1, 256, 32, "head-major"),
    (11, 4, 1, 128, 128, "odd"), (5, 3, 2, 64, 48, "broadcast"), (4, 2, 2, 512, 512, "own"), (2, 3, 1, 1024, 1000, "own"),
    (3, 2, 1, 96, 96, "own"), (129, 16, 4, 128, 32, "own"), (5, 3, 2, 130, 130, "own"), (300, 40, 40, 64, 64, "packed"),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("T,hq,hk,D,rot,layout", ROPE)
def test_rope(T, hq, hk, D, rot, layout, interleaved, dtype):
    say("rope", T, hq, hk, D, rot, layout, interleaved, dtype)
    table = R.rope_table(500, R.rope_theta(rot), 1.1).astype(np.float32)
    rng = np.random.default_rng(T * 7 + D)
    pos = rng.integers(0, 500, T)
    pos[0] = 499
    if T > 4:
        pos[1], pos[2], pos[3] = -5, 500, 2 ** 31 - 1        # held to the table
    dt, dp = dev_f32(table), dev_i32(pos)
    q, k = rope_case(T, hq, D, layout, dtype, 1), rope_case(T, hk, D, layout, dtype, 2) if hk else None
    for inverse in (False, True):
        qo = torch.full((T, hq, D), 9.0, dtype=dtype, device=DEV)
        ko = torch.full((T, hk, D), 9.0, dtype=dtype, device=DEV) if hk else None
        lcp.lcp_rope(q, qo, dt, dp, k=k, k_out=ko, interleaved=interleaved, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                continue
            ref = R.rope(down(x), table, pos, interleaved, inverse)
            # two products and their sum, each rounded (the sum's share again where the terms cancel)
            mag = R.rope_abs(down(x), table, pos, interleaved)
            tol = 1.01 * R.U32 * (mag + np.abs(ref))
            if dtype == torch.bfloat16:
                assert R.bf16_within(down(y), ref, tol)
            else:
                assert np.all(np.abs(down(y) - ref) <= tol)
            assert torch.equal(y[..., rot:], x[..., rot:])      # passed through unrounded


@pytest.mark.parametrize("layout", ["own", "packed", "head-major", "odd"])
def test_rope_in_place_and_output_strides(layout):
    say("rope in place", layout)
    T, H, D, rot = 37, 5, 128, 96
    dt = dev_f32(R.rope_table(64, R.rope_theta(rot)))
    pos = dev_i32(np.arange(T))
    x = rope_case(T, H, D, layout, torch.bfloat16, 3)
    want = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    lcp.lcp_rope(x, want, dt, pos)
    out = torch.zeros(H, T, D + 24, dtype=torch.bfloat16, device=DEV)
    lcp.lcp_rope(x, out[..., 8:D + 8].transpose(0, 1), dt, pos)
    assert torch.equal(out[..., 8:D + 8].transpose(0, 1), want)
    assert not out[..., :8].any() and not out[..., D + 8:].any()
    lcp.lcp_rope(x, x, dt, pos)
    assert torch.equal(x, want)


def test_rope_gradient_is_the_transpose_and_matches_differences():
    """<g, R x> = <R' g, x>, and a difference quotient of <g, R x> along a direction."""
    say("rope gradient")
    T, H, D, rot = 9, 3, 80, 48
    table = dev_f32(R.rope_table(100, R.rope_theta(rot), 1.3))
    pos = dev_i32(np.arange(T) * 11)
    g = torch.Generator().manual_seed(5)
    x, w, u = (torch.randn(T, H, D, generator=g).to(DEV) for _ in range(3))
    for inter in (False, True):
        def f(z):
            y = torch.empty_like(z)
            lcp.lcp_rope(z, y, table, pos, interleaved=inter)
            return (y.double() * w.double()).sum().item()
        grad = torch.empty_like(w)
        lcp.lcp_rope(w, grad, table, pos, interleaved=inter, inverse=True)
        n = float(w.double().norm() * x.double().norm()) * 1.3
        assert abs(f(x) - float((grad.double() * x.double()).sum())) <= 6 * R.U32 * n
        h = 0.5      # linear: any step is exact up to rounding
        d = (f(x + h * u) - f(x - h * u)) / (2 * h)
        n = float(w.double().norm() * (x.double().norm() + u.double().norm())) * 1.3
        assert abs(d - float((grad.double() * u.double()).sum())) <= 12 * R.U32 * n


# ---- cache ------------------------------------------------------------------------
def new_cache(fmt, pages, ps, heads, D, poison=True):
    """A cache whose every bit pattern is hostile: NaN values or NaN scales."""
    c = lcp.PagedKVCache.empty(pages, ps, heads, D, FMT[fmt])
    if poison:
        for t in (c.k, c.v):
            t.view(torch.uint8).fill_(0xFF)
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.fill_(math.nan)
    return c


def held(c, side, fmt):
    """(codes, scales) of the whole cache on the host; bf16: (values, None)."""
    t = c.k if side == "k" else c.v
    if fmt == "bf16":
        return t.float().cpu().numpy(), None
    s = (c.k_scale if side == "k" else c.v_scale).cpu().numpy()
    return (t.view(torch.uint8).cpu().numpy() if fmt == "fp8" else t.cpu().numpy()), s


@pytest.mark.parametrize("rot,interleaved", [(0, False), (1, False), (1, True), (2, False), (2, True), (16, True)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("T,hq,hk,D,ps", [(1, 4, 1, 64, 16), (5, 8, 2, 128, 48), (131, 6, 6, 256, 64),
                                          (257, 40, 8, 128, 16), (70, 5, 5, 64, 128)])
def test_kv_append_and_read(T, hq, hk, D, ps, fmt, rot, interleaved):
    """Codes and scales equal to the fp32 definition bit for bit; slots outside
    the cache write nothing and read as zeros; the rest of the cache is untouched."""
    rot = D // rot if rot in (1, 2) else rot
    say("kv append", T, hq, hk, D, ps, fmt, rot, interleaved)
    rng = np.random.default_rng(T + D)
    pages = T // ps + 3
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if T > 4:
        slots[1], slots[2], slots[3] = -1, pages * ps, 2 ** 31 - 1
    gain = 10.0 ** rng.uniform(-3, 3, (T, 1, 1))
    qkv = [R.bf16(rng.normal(size=(T, h, D)) * gain) for h in (hq, hk, hk)]
    if T > 20:
        qkv[1][7] = 0
        qkv[2][8] = 0
        qkv[1][9, 0, 3], qkv[2][10, hk - 1, 5], qkv[2][11, 0, 0] = np.nan, np.inf, -np.inf
        qkv[2][12, 0] = R.bf16(np.full(D, 448.0 / 3))
        qkv[2][13, 0] = 1e-38
    packed = dev_f32(np.concatenate([x.reshape(T, -1) for x in qkv], 1), torch.bfloat16)
    q, k, v = (x.view(T, -1, D) for x in packed.split([hq * D, hk * D, hk * D], 1))
    c = new_cache(fmt, pages, ps, hk, D)
    before = {s: held(c, s, fmt) for s in "kv"}
    if rot:
        pos = rng.integers(0, 300, T)
        table = R.rope_table(300, R.rope_theta(rot)).astype(np.float32)
        qo = torch.full((T, hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        c.append(k, v, dev_i32(slots), q=q, q_out=qo, table=dev_f32(table), pos=dev_i32(pos), interleaved=interleaved)
        kr = R.rope_f32(qkv[1], table, pos, interleaved)
        assert np.array_equal(down(qo), R.bf16(R.rope_f32(qkv[0], table, pos, interleaved)).astype(np.float64))
    else:
        c.append(k, v, dev_i32(slots))
        kr = qkv[1]
    good = (slots >= 0) & (slots < pages * ps)
    pg, off = slots[good] // ps, slots[good] % ps
    expect = {}
    for side, x in (("k", kr), ("v", qkv[2])):
        got, sc = held(c, side, fmt)
        if fmt == "bf16":
            ref = R.bf16(x)
            assert np.array_equal(got[pg, :, off], ref[good], equal_nan=True)
        else:
            ref, s = R.quantise(x, fmt)
            assert np.array_equal(sc[pg, :, off], s[good], equal_nan=True)
            assert np.array_equal(got[pg, :, off], ref[good])
            ref = R.dequantise(ref, s, fmt)
        untouched = np.ones((pages, ps), dtype=bool)
        untouched[pg, off] = False
        assert np.array_equal(got.transpose(0, 2, 1, 3)[untouched], before[side][0].transpose(0, 2, 1, 3)[untouched],
                              equal_nan=fmt == "bf16")
        expect[side] = np.where(good[:, None, None], ref, np.float32(0))
    for odt in (torch.bfloat16, torch.float32):
        ko, vo = (torch.full((T, hk, D), 5.0, dtype=odt, device=DEV) for _ in range(2))
        c.read(dev_i32(slots), ko, vo)
        for got, side in ((ko, "k"), (vo, "v")):
            want = expect[side] if odt == torch.float32 else R.bf16(expect[side])
            bad = np.isnan(expect[side])
            assert np.array_equal(np.isnan(down(got)), bad)
            assert np.array_equal(down(got)[~bad], want.astype(np.float64)[~bad])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kv_append_rows_of_any_alignment(fmt, D):
    """Odd offsets and strides, head-major rows and broadcast values give the bits of aligned rows."""
    say("kv append alignment", fmt, D)
    T, hq, hk, ps = 21, 4, 2, 16
    rows = {lay: [rope_case(T, h, D, lay, torch.bfloat16, 7 + i) for i, h in enumerate((hq, hk, hk))]
            for lay in ("own", "odd", "head-major", "broadcast")}
    table, pos = dev_f32(R.rope_table(64, R.rope_theta(D // 2))), dev_i32(np.arange(T))
    slots = dev_i32(np.random.default_rng(1).permutation(3 * ps)[:T])
    for lay, (q, k, v) in rows.items():
        for inter in (False, True):
            got = []
            for a, b, c in ((q, k, v), [x.contiguous() for x in (q, k, v)]):
                cache = new_cache(fmt, 3, ps, hk, D)
                qo = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV)
                cache.append(b, c, slots, q=a, q_out=qo, table=table, pos=pos, interleaved=inter)
                got.append([qo] + [x.view(torch.uint8) for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)
                                   if x is not None])
            assert all(torch.equal(x, y) for x, y in zip(*got)), (lay, inter)


def test_kv_offsets_beyond_32_bits():
    """Pages whose byte offset passes 2^32 (bf16: elements too), written, read and attended."""
    say("kv offsets beyond 32 bits")
    ps, hk, D = 128, 16, 256
    pages = (1 << 32) // (ps * hk * D) + 4
    c = lcp.PagedKVCache.empty(pages, ps, hk, D, torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(150, hk, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    t = np.arange(150)
    table = np.array([pages - 1, pages - 3])
    slots = table[t // ps] * ps + t % ps
    c.append(k, v, dev_i32(slots))
    ko, vo = c.read(dev_i32(slots))
    assert torch.equal(ko, k) and torch.equal(vo, v)
    q = torch.randn(1, hk, D, generator=g).bfloat16().to(DEV)
    out, lse = c.attend(q, dev_i32(table[None]), dev_i32([150]))
    ref, rl, _ = R.attend(down(q)[0], down(k), down(v), D ** -0.5)
    assert np.abs(down(out)[0] - ref).max() < 2.0 ** -8 * np.abs(ref).max() and np.abs(down(lse)[0] - rl).max() < 1e-5
    del c
    torch.cuda.empty_cache()


# ---- attention ------------------------------------------------------------------------
def filled(fmt, pages, ps, hk, D, need, seed, gain=1.0):
    """A hostile cache with `need` slots of each listed page valid, and the
    fp32 values it holds: [pages][ps][hk][D]."""
    rng = np.random.default_rng(seed)
    c = new_cache(fmt, pages, ps, hk, D)
    vals = {}
    for side, t, s in (("k", c.k, c.k_scale), ("v", c.v, c.v_scale)):
        x = (rng.normal(size=(pages, hk, ps, D)) * gain).astype(np.float32)
        host = t.cpu()
        if fmt == "bf16":
            x = R.bf16(x)
            new = torch.from_numpy(x).bfloat16()
        else:
            codes, sc = R.quantise(x, fmt)
            x = R.dequantise(codes, sc, fmt)
            new = torch.from_numpy(codes)
            new = new.view(torch.float8_e4m3fn) if fmt == "fp8" else new
            sh = s.cpu()
            for p, n in need.items():
                sh[p, :, :n] = torch.from_numpy(sc)[p, :, :n]
            s.copy_(sh)
        hb, nb = host.view(torch.uint8), new.view(torch.uint8)
        for p, n in need.items():
            hb[p, :, :n] = nb[p, :, :n]
        t.copy_(host)
        vals[side] = x.transpose(0, 2, 1, 3)
    return c, vals


def check_attend(fmt, lens, hq, hk, D, ps, window=0, gain=1.0, odt=torch.float32, scale=None, seed=0, spare=0,
                 holes=(), q_pad=0):
    rng = np.random.default_rng(seed + 1000)
    B = len(lens)
    npg = [-(-n // ps) for n in lens]
    P = max(max(npg), 1) + spare
    pages = sum(npg) + 2
    order = rng.permutation(pages)
    table = np.full((B, P), -1, dtype=np.int64)
    table[:, 1::2] = 2 ** 31 - 1                       # entries that must not be used
    need, at = {}, 0
    for b, n in enumerate(lens):
        table[b, :npg[b]] = order[at:at + npg[b]]
        at += npg[b]
        for i in range(npg[b]):
            need[int(table[b, i])] = min(ps, n - i * ps)
    c, vals = filled(fmt, pages, ps, hk, D, need, seed, gain)
    real = table.copy()
    for b, i in holes:                                 # page numbers outside the cache
        table[b, i] = pages if (b + i) % 2 else -7
    qh = R.bf16(rng.normal(size=(B, hq, D)))
    buf = torch.full((B, hq * D + q_pad), math.nan, dtype=torch.bfloat16, device=DEV)
    q = buf[:, :hq * D].unflatten(1, (hq, D))
    q.copy_(dev_f32(qh, torch.bfloat16))
    out = torch.full((B, hq, D), math.nan, dtype=odt, device=DEV)
    lse = torch.full((B, hq), math.nan, device=DEV)
    args = (q, dev_i32(table), dev_i32(lens))
    kw = dict(max_len=max(max(lens), 0), scale=scale, window=window)
    c.attend(*args, out=out, lse=lse, **kw)
    scale = D ** -0.5 if scale is None else scale
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        t = np.array([i for i in range(lo, n) if (b, i // ps) not in holes], dtype=np.int64)
        k, v = (vals[s][real[b, t // ps], t % ps].astype(np.float64) for s in "kv")
        ref, rl, (zmag, vmag) = R.attend(qh[b].astype(np.float64), k, v, scale)
        # a score: D + 6 roundings of sums and products up to zmag (scale and code scale among them);
        # p: exp of that, its own roundings and its split into two bfloat16 (2^-17 each); sums of n terms
        dz = (D + 6) * R.U32 * zmag + 4 * R.U32 * (1 + zmag)
        dp = 2 * dz + (len(t) + 64) * R.U32 + 2.0 ** -16
        tol = dp[:, None] * vmag * (1 + dp[:, None]) + 1e-30
        got, gl = down(out)[b], down(lse)[b]
        if odt == torch.bfloat16:
            assert R.bf16_within(got, ref, tol), (b, n)
        else:
            assert np.all(np.abs(got - ref) <= tol), (b, n, float(np.abs(got - ref).max()))
        if len(t) == 0:
            assert np.all(gl == -np.inf)
        else:
            assert np.all(np.abs(gl - rl) <= dp + 2 * R.U32 * np.abs(rl)), (b, n)
    again, lse2 = c.attend(*args, out=torch.empty_like(out), **kw)
    assert torch.equal(again, out) and torch.equal(lse2, lse)      # the same bits
    return c, args, out


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 200, 255, 257, 511, 513, 777, 1000, 1]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("hq,hk,D,ps", [(8, 8, 64, 16), (8, 2, 128, 16), (16, 1, 128, 48), (6, 2, 256, 32),
                                        (20, 1, 64, 64), (40, 1, 128, 128), (10, 2, 128, 64), (33, 1, 256, 16)])
def test_attend_lengths(fmt, hq, hk, D, ps):
    say("attend lengths", fmt, hq, hk, D, ps)
    check_attend(fmt, LENS, hq, hk, D, ps, spare=2)


@pytest.mark.parametrize("window", [1, 7, 16, 33, 100, 600, 5000])
def test_attend_window(window):
    say("attend window", window)
    check_attend("fp8", LENS, 8, 2, 128, 48, window=window)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("n", [4095, 4097, 9000, 20011])
def test_attend_long_few_rows(fmt, n):
    say("attend long", fmt, n)
    check_attend(fmt, [n, 5], 4, 1, 128, 64)


@pytest.mark.parametrize("D", [64, 256])
def test_attend_long_other_heads(D):
    say("attend long", D)
    check_attend("bf16", [6001], 6, 2, D, 32)
    check_attend("int8", [6001, 0, 3], 17, 1, D, 16, window=5000)


@pytest.mark.parametrize("B,n,hq,hk,D", [(300, 700, 2, 2, 64), (70, 1500, 16, 8, 64), (9, 4000, 34, 1, 64),
                                          (530, 530, 1, 1, 64), (40, 1000, 32, 16, 64)])
def test_attend_many_sequences(B, n, hq, hk, D):
    """Batches whose rounds are dealt over the workgroups: units cut anywhere, several to a workgroup, empty ones among them."""
    say("attend many", B, n, hq, hk, D)
    rng = np.random.default_rng(B)
    lens = rng.integers(0, n + 1, B)
    lens[rng.integers(0, B, B // 5)] = 0
    lens[rng.integers(0, B)] = n
    check_attend("int8", [int(x) for x in lens], hq, hk, D, 32)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("hq,hk,D", [(17, 1, 64), (80, 2, 64), (32, 1, 128), (47, 1, 128), (49, 1, 128)])
def test_attend_groups_of_more_than_16_heads(fmt, hq, hk, D):
    """Enough work that two tiles of 16 heads share a wave's loads: dealt (long sequences) and direct (many short ones)."""
    say("attend large groups", fmt, hq, hk, D)
    rng = np.random.default_rng(hq)
    lens = [int(x) for x in rng.integers(0, 4000, 30)] + [0, 1, 31, 32, 33, 4000]
    check_attend(fmt, lens, hq, hk, D, 48, window=3500)
    lens = [int(x) for x in rng.integers(0, 70, 140)] + [0, 1, 127, 128, 129]
    check_attend(fmt, lens, hq, hk, D, 16, holes={(142, 2), (0, 0)})


@pytest.mark.parametrize("fmt,B,n,hq,hk,D", [("fp8", 100, 4000, 4, 2, 128), ("int8", 70, 6000, 4, 2, 64),
                                             ("bf16", 70, 3000, 2, 2, 128), ("int8", 30, 9000, 3, 1, 256)])
def test_attend_more_work_than_one_part_a_compute_unit(fmt, B, n, hq, hk, D):
    say("attend much work", fmt, B, n, hq, hk, D)
    rng = np.random.default_rng(B + D)
    check_attend(fmt, [int(x) for x in rng.integers(0, n + 1, B - 2)] + [0, n], hq, hk, D, 64)


def test_attend_empty_batch_rows_and_zero_max_len():
    say("attend empty")
    check_attend("fp8", [0, 0, 0], 8, 2, 128, 16)
    check_attend("bf16", [0], 2, 2, 64, 16)


def test_attend_pages_left_out():
    """Tokens of a page number outside the cache count for nothing, also where that leaves none."""
    say("attend holes")
    check_attend("fp8", [100, 16, 64, 300], 8, 2, 128, 16,
                 holes={(0, 0), (0, 3), (1, 0), (2, 1), (2, 2), (3, 18), (3, 7)})
    check_attend("bf16", [1000], 4, 4, 64, 64, holes={(0, i) for i in range(0, 16, 2)})


def test_attend_bf16_out_strides_scale_and_peaked_scores():
    say("attend bf16 out")
    check_attend("int8", [5, 70, 333], 12, 4, 128, 32, odt=torch.bfloat16, q_pad=24)
    check_attend("bf16", [5, 70, 333], 12, 4, 128, 32, gain=30.0, scale=0.5)      # scores of hundreds
    check_attend("fp8", [5, 70, 333], 12, 4, 64, 32, scale=-0.3)
    check_attend("fp8", [33], 4, 4, 64, 32, scale=0.0)


def test_attend_lengths_past_the_bound_are_held_to_it():
    say("attend held lengths")
    c, (q, table, lens), out = check_attend("bf16", [64, 64], 4, 2, 64, 16)
    o, _ = c.attend(q, table, dev_i32([2 ** 31 - 1, 64]), max_len=64, out=torch.empty_like(out))
    assert torch.equal(o, out)
    o, l = c.attend(q, table, dev_i32([-3, 64]), max_len=64, out=torch.empty_like(out))
    assert not o[0].any() and torch.all(l[0] == -math.inf) and torch.equal(o[1], out[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attend_non_finite_counted_tokens_show(fmt):
    """A NaN among the counted keys or values reaches the rows that read it and no other."""
    say("attend non-finite", fmt)
    c, (q, table, lens), out = check_attend(fmt, [40, 70, 9], 4, 2, 128, 16)
    page = int(table[1, 2])
    if fmt == "bf16":
        c.k[page, 1, 5, 3] = math.nan
        c.v[int(table[2, 0]), 0, 8, 1] = math.inf
    else:
        c.k_scale[page, 1, 5] = math.nan
        c.v_scale[int(table[2, 0]), 0, 8] = math.nan
    o, l = c.attend(q, table, lens, out=torch.empty_like(out))
    assert torch.equal(o[0], out[0])
    assert torch.isnan(o[1, 2:]).all() and torch.isnan(l[1, 2:]).all()
    assert torch.equal(o[1, :2], out[1, :2]) and torch.equal(o[2, 2:], out[2, 2:])
    assert not torch.isfinite(o[2, :2, 1]).any()


def test_step_on_another_stream_and_in_a_graph():
    """append + attend on a stream of their own, and captured: every replay on
    new contents equals the eager result, with eager work between."""
    say("serve stream and graph")
    hq, hk, D, ps, B = 8, 2, 128, 16, 3
    lens = np.array([20, 33, 1])
    c, vals = filled("fp8", 12, ps, hk, D, {p: ps for p in range(12)}, 5)
    pt = np.arange(12).reshape(B, 4)
    table = dev_f32(R.rope_table(64, R.rope_theta(D)))
    slots = dev_i32(pt[np.arange(B), (lens - 1) // ps] * ps + (lens - 1) % ps)
    pos, dl, dp = dev_i32(lens - 1), dev_i32(lens), dev_i32(pt)
    g = torch.Generator().manual_seed(9)
    qkv = torch.empty(B, (hq + 2 * hk) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (x.view(B, -1, D) for x in qkv.split([hq * D, hk * D, hk * D], 1))
    qo, out = (torch.empty(B, hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lse = torch.empty(B, hq, device=DEV)
    ws = torch.empty(lcp.lcp_attn_decode_workspace_bytes(c.c, B, hq, 64), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        c.append(k, v, slots, q=q, q_out=qo, table=table, pos=pos, stream=stream)
        c.attend(qo, dp, dl, max_len=64, out=out, lse=lse, ws=ws, stream=stream)

    inputs = [torch.randn(qkv.shape, generator=g).bfloat16().to(DEV) for _ in range(4)]
    want = []
    for x in inputs:
        qkv.copy_(x)
        step()
        want.append((out.clone(), lse.clone(), c.k.view(torch.uint8).clone()))
    assert not torch.equal(want[0][0], want[1][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qkv.copy_(inputs[2])
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want[2][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 3, 1, 2, 0):
        qkv.copy_(inputs[i])
        out.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
        assert torch.equal(c.k.view(torch.uint8), want[i][2])
        c.attend(qo, dp, dl, max_len=64)                # eager work in between


def test_example_decodes_through_the_deployed_layers():
    """The attention block of examples/: deployed 2:4 projections, rotary cache write, attention over shared pages."""
    import importlib.util
    import os
    say("example block")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "sparse_attention_block.py")
    spec = importlib.util.spec_from_file_location("sparse_attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for prompt in (200, 256):
        err, y = mod.main(["--hidden", "512", "--heads", "8", "--kv-heads", "2", "--prompt", str(prompt), "--steps", "5",
                           "--batch", "3", "--train-steps", "2"])
        # bfloat16 output (2^-8) against fp32 on the same bfloat16 reads of fp8 codes, which are exact
        assert err < 2.0 ** -8 and torch.isfinite(y.float()).all() and y.shape == (3, 512)


def test_tensors_on_the_cpu_are_refused():
    """Also where only the cache is: its pointers would reach the kernels."""
    say("cpu tensors")
    host = lcp.PagedKVCache.empty(2, 16, 2, 64, device="cpu")
    dev = lcp.PagedKVCache.empty(2, 16, 2, 64, device=DEV)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    i, p = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    for call in (lambda: host.append(x, x, i), lambda: host.read(i), lambda: host.attend(x, p, i),
                 lambda: dev.append(x, x.cpu(), i), lambda: dev.read(i.cpu()), lambda: dev.attend(x, p, i.cpu())):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
