"""Which way a call of lcp_sparse_linear is cut (host only), and that the sizes of tests/block_cuts.py reach every one of
them: a change of the estimates that takes a way out of the tests fails here."""
import ctypes
import math
import random

import pytest

from learnable_channel_permutation_amd import _lib as L
from tests.block_cuts import CUTS

P = 0x100000
LAYERS = ((4096, 4096), (4096, 11008), (11008, 4096), (5120, 13824), (13824, 5120), (8192, 28672), (28672, 8192))


def packed(mode, cout, cin):
    return L.lcp_packed(P, 2 * P, 3 * P, L.LCP_E4M3 if mode else L.LCP_BF16, cout, cin, int(mode == 2))


def cut(mode, T, cout, cin):
    return L.lcp_sparse_linear_cut(packed(mode, cout, cin), T)


def steps(mode, cin):
    return -(-cin * (1 if mode else 2) // 128)


@pytest.mark.parametrize("want", list(CUTS), ids=str)
def test_sizes_reach_their_cut(want):
    T, cout, cin = CUTS[want]
    mode, rt, _, waves, parts = want
    n = steps(mode, cin)
    assert cut(mode, T, cout, cin) == want
    assert cin % 128 and T % 16
    if rt:                                               # steps beyond a wave's first, dealt unevenly
        assert n > waves and n % waves
    else:
        assert cout > 256 and T > 128 and cout % 256 and T % 128
        assert n // parts >= 8 and (parts == 1 or n % parts)


def test_every_cut_of_a_call_has_a_size():
    rng = random.Random(5)
    seen = set()
    for _ in range(60000):
        cout, cin = rng.choice(LAYERS)
        if rng.random() < 0.5:
            cout, cin = (32 * max(1, round(math.exp(rng.uniform(0, math.log(900))))) for _ in range(2))
        T = max(1, round(math.exp(rng.uniform(0, math.log(5000)))))
        mode = rng.randrange(3)
        seen.add(cut(mode, T, cout, cin))
    assert seen == set(CUTS)


def test_the_parts_fit_the_workspace():
    n = ctypes.c_size_t(0)
    for mode in range(3):
        for cout, cin in LAYERS + ((288, 28672), (64, 1 << 20)):
            for T in (65, 100, 128, 333, 700, 2048, 5000, 30000):
                p = packed(mode, cout, cin)
                assert L.LIB.lcp_sparse_linear_workspace_bytes(ctypes.byref(p), T, ctypes.byref(n)) == L.LCP_OK
                _, rt, _, _, parts = L.lcp_sparse_linear_cut(p, T)
                assert 1 <= parts <= min(8, steps(mode, cin)) and (rt == 0 or parts == 1)
                assert parts == 1 or parts * T * cout * 4 <= n.value
                each = -(-steps(mode, cin) // parts)
                assert (parts - 1) * each < steps(mode, cin)           # the last part has steps


def test_operands():
    """fp32 outputs, few tokens and every layer that is not fast: exact products."""
    assert [cut(0, T, 64, 64)[0] for T in (1, 64, 65, 4096)] == [0] * 4
    assert [cut(1, T, 64, 64)[0] for T in (1, 64, 65, 4096)] == [1] * 4
    assert [cut(2, T, 64, 64)[0] for T in (1, 64, 65, 4096)] == [1, 1, 2, 2]
    assert [L.lcp_sparse_linear_cut(packed(2, 64, 64), T, L.LCP_F32)[0] for T in (1, 64, 65, 4096)] == [1] * 4


def test_refusals():
    out = (ctypes.c_int32 * 5)()

    def call(p, T=5, dt=L.LCP_BF16, out=out):
        return L.LIB.lcp_sparse_linear_cut(None if p is None else ctypes.byref(p), T, dt, out)

    p = packed(1, 64, 128)
    assert call(p) == L.LCP_OK
    for bad in (call(None), call(p, 0), call(p, -1), call(p, out=None), call(packed(1, 48, 128)), call(packed(1, 64, 0))):
        assert bad == L.LCP_E_INVAL
    assert call(p, dt=L.LCP_E4M3) == L.LCP_E_UNSUPPORTED
    with pytest.raises(L.LcpError):
        L.lcp_sparse_linear_cut(p, 0)
