"""One-token attention where its work is cut over the workgroups and joined by a
second kernel: many sequences, windows, pages left out, lengths out of range,
NaN and infinities, another stream and replayed graphs; and what an append
leaves untouched beside the codes."""
import math

import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.gpu_util import DEV, say
from tests.test_gpu_serve import FMT, check_attend, dev_f32, dev_i32, filled, new_cache

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")


def assert_cut(fmt, B, hq, hk, D, max_len, window=0):
    """Units of more than 192 KB of K are cut whatever their number is; the workspace query says that they can be."""
    span = min(max_len, window + 31) if window else max_len
    assert span * D * (2 if fmt == "bf16" else 1) > 192 << 10
    k = torch.empty(1, hk, 16, D, dtype=FMT[fmt])
    s = None if fmt == "bf16" else torch.empty(1, hk, 16)
    c = lcp._lib.make_kv_cache(k, torch.empty_like(k), s, None if s is None else torch.empty_like(s))
    assert lcp.lcp_attn_decode_workspace_bytes(c, B, hq, max_len, window) > 0


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("B,hq,hk,D", [(300, 2, 2, 64), (530, 1, 1, 64), (700, 20, 1, 64), (520, 2, 1, 256)])
def test_cut_work_of_many_sequences(B, hq, hk, D, fmt):
    """More sequences than a workgroup has threads: several to a thread in the scan of the lengths, units cut anywhere
    and several to a workgroup, many of them empty, the first and last ones among them."""
    say("cut many", fmt, B, hq, hk, D)
    n = (193 << 10) // (D * (2 if fmt == "bf16" else 1)) + 40
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, 150, B)
    lens[rng.integers(0, B, B // 3)] = 0
    lens[rng.integers(0, B, 5)] = n - rng.integers(0, 70, 5)
    lens[B // 2], lens[0], lens[-1] = n, 0, 0
    assert_cut(fmt, B, hq, hk, D, n)
    check_attend(fmt, [int(x) for x in lens], hq, hk, D, 32)


@pytest.mark.parametrize("fmt,hq,hk,D,window", [("fp8", 8, 2, 128, 1700), ("bf16", 6, 2, 256, 450), ("int8", 34, 1, 64, 3301),
                                                ("bf16", 48, 1, 128, 1001)])
def test_cut_windows(fmt, hq, hk, D, window):
    """Windows that begin anywhere in a step, sequences shorter and longer than the window."""
    say("cut windows", fmt, hq, hk, D, window)
    lens = [0, 1, 33, window - 1, window, window + 1, window + 16, window + 31, window + 32, 2 * window + 5, 5000, 0]
    assert_cut(fmt, len(lens), hq, hk, D, max(lens), window)
    check_attend(fmt, lens, hq, hk, D, 48, window=window)


@pytest.mark.parametrize("fmt,hq,hk,D", [("bf16", 3, 1, 64), ("fp8", 20, 1, 128), ("int8", 4, 2, 256)])
def test_cut_pieces_without_a_counted_token(fmt, hq, hk, D):
    """Pages outside the cache over whole pieces of a unit: their maximum is that of no token and their sum 0."""
    say("cut holes", fmt, hq, hk, D)
    n, ps = 9000, 64
    P = -(-n // ps)
    assert_cut(fmt, 1, hq, hk, D, n)
    # 64 KB of K and V a part and a step more here: 288 tokens at most
    for gone in (range(0, 40), range(50, 100), range(100, P), [i for i in range(P) if i % 47 > 2], range(P)):
        check_attend(fmt, [n], hq, hk, D, ps, holes={(0, i) for i in gone})
    check_attend(fmt, [n, 17, 0, 5000], hq, hk, D, ps, holes={(0, i) for i in range(P)} | {(3, 2)})


def test_cut_lengths_past_the_bound_and_none():
    say("cut held lengths")
    n = 3500
    assert_cut("bf16", 3, 4, 2, 64, n)
    c, (q, table, lens), out = check_attend("bf16", [n, 40, n], 4, 2, 64, 16)
    o, _ = c.attend(q, table, dev_i32([2 ** 31 - 1, 40, n + 1]), max_len=n, out=torch.empty_like(out))
    assert torch.equal(o, out)
    o, l = c.attend(q, table, dev_i32([-3, 40, -2 ** 31]), max_len=n, out=torch.empty_like(out))
    assert not o[::2].any() and torch.all(l[::2] == -math.inf)
    ref, _ = c.attend(q[1:2], table[1:2], dev_i32([40]), max_len=n, out=torch.empty_like(out[1:2]))
    assert torch.allclose(o[1:2], ref, rtol=0, atol=2.0 ** -14 * float(ref.abs().max()))        # cut elsewhere
    o, l = c.attend(q, table, dev_i32([0, 0, 0]), max_len=n, out=torch.full_like(out, 3.0), lse=torch.zeros(3, 4, device=DEV))
    assert not o.any() and torch.all(l == -math.inf)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_cut_non_finite_counted_tokens_show(fmt):
    """A NaN among the counted keys or values reaches the rows that read it and no other, through the join."""
    say("cut non-finite", fmt)
    n = 4000
    assert_cut(fmt, 3, 4, 2, 128, n)
    c, (q, table, lens), out = check_attend(fmt, [n, n - 900, 2000], 4, 2, 128, 16)
    page = int(table[1, 100])
    if fmt == "bf16":
        c.k[page, 1, 5, 3] = math.nan
        c.v[int(table[2, 60]), 0, 8, 1] = math.inf
    else:
        c.k_scale[page, 1, 5] = math.nan
        c.v_scale[int(table[2, 60]), 0, 8] = math.nan
    o, l = c.attend(q, table, lens, max_len=n, out=torch.empty_like(out))
    assert torch.equal(o[0], out[0])
    assert torch.isnan(o[1, 2:]).all() and torch.isnan(l[1, 2:]).all()
    assert torch.equal(o[1, :2], out[1, :2]) and torch.equal(o[2, 2:], out[2, 2:])
    assert not torch.isfinite(o[2, :2, 1]).any()


@pytest.mark.parametrize("hq,hk", [(8, 2), (34, 2)])
def test_cut_step_on_another_stream_and_in_a_graph(hq, hk):
    """append + attend with a caller's workspace on a stream of their own, and captured: every replay, with lengths that
    move the cut and leave sequences empty, equals the eager result, with eager work between."""
    say("cut stream and graph", hq, hk)
    D, ps, B, P = 128, 16, 5, 250
    most = P * ps
    assert_cut("fp8", B, hq, hk, D, most)
    c, _ = filled("fp8", B * P, ps, hk, D, {p: ps for p in range(B * P)}, 5)
    pt = np.random.default_rng(1).permutation(B * P).reshape(B, P)
    table = dev_f32(R.rope_table(most, R.rope_theta(D)))
    g = torch.Generator().manual_seed(9)
    qkv = torch.empty(B, (hq + 2 * hk) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (x.view(B, -1, D) for x in qkv.split([hq * D, hk * D, hk * D], 1))
    qo, out = (torch.empty(B, hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lse = torch.empty(B, hq, device=DEV)
    slots, pos, dl = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(3))
    dp = dev_i32(pt)
    need = lcp.lcp_attn_decode_workspace_bytes(c.c, B, hq, most)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def step(stream=None):
        c.append(k, v, slots, q=q, q_out=qo, table=table, pos=pos, stream=stream)
        c.attend(qo, dp, dl, max_len=most, out=out, lse=lse, ws=ws, stream=stream)

    def load(i):
        lens = np.array(LENS[i])
        at = np.maximum(lens - 1, 0)
        s = pt[np.arange(B), at // ps] * ps + at % ps
        slots.copy_(dev_i32(np.where(lens > 0, s, -1)))
        pos.copy_(dev_i32(at))
        dl.copy_(dev_i32(lens))
        qkv.copy_(inputs[i])

    LENS = [[4000, 3999, 1, 700, 2222], [0, 4000, 0, 0, 31], [17, 0, 3000, 4000, 0], [0, 0, 0, 0, 0], [4000] * 5]
    inputs = [torch.randn(qkv.shape, generator=g).bfloat16().to(DEV) for _ in LENS]
    first = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]

    def restart():
        for t, f in zip((c.k, c.v, c.k_scale, c.v_scale), first):
            t.copy_(f)

    want = []
    for i in range(len(LENS)):
        restart()
        load(i)
        ws.fill_(0xFF)
        step()
        want.append((out.clone(), lse.clone(), c.k.view(torch.uint8).clone()))
    assert not torch.equal(want[0][0], want[4][0]) and not want[3][0].any() and torch.all(want[3][1] == -math.inf)
    side = torch.cuda.Stream()
    for i in (0, 2):
        restart()
        load(i)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 4, 3, 2, 0, 3, 4):
        restart()
        load(i)
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
        assert torch.equal(c.k.view(torch.uint8), want[i][2])
        c.attend(qo, dp, dl, max_len=most)              # eager work in between


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_append_writes_no_scale_but_its_own(fmt):
    say("append scales", fmt)
    T, hk, D, ps, pages = 70, 3, 128, 48, 5
    rng = np.random.default_rng(2)
    slots = rng.permutation(pages * ps)[:T]
    slots[1], slots[2], slots[3] = -1, pages * ps, 2 ** 31 - 1
    x = dev_f32(rng.normal(size=(T, hk, D)), torch.bfloat16)
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape).copy_(x)
    good = (slots >= 0) & (slots < pages * ps)
    rest = np.ones((pages, ps), dtype=bool)
    rest[slots[good] // ps, slots[good] % ps] = False
    for rows in (x, odd):
        c = new_cache(fmt, pages, ps, hk, D)
        for s in (c.k_scale, c.v_scale):
            s.copy_(torch.arange(s.numel(), device=DEV).view(s.shape))
        before = [s.clone() for s in (c.k_scale, c.v_scale)]
        c.append(rows, rows, dev_i32(slots))
        for s, b in zip((c.k_scale, c.v_scale), before):
            s, b = (t.cpu().numpy().transpose(0, 2, 1) for t in (s, b))
            assert np.array_equal(s[rest], b[rest]) and not np.any(s[~rest] == b[~rest])


@pytest.mark.parametrize("ps", [16, 80, 112, 496, 1008, 4080, 4096])
def test_page_sizes(ps):
    """Pages of any multiple of 16 tokens, cut and direct: the page of a tile and its place there."""
    say("page sizes", ps)
    assert_cut("int8", 3, 6, 2, 128, 9001)
    check_attend("int8", [9001, 0, 4097], 6, 2, 128, ps)
    check_attend("bf16", [490, 1, 479, 33], 6, 2, 128, ps, spare=1)
