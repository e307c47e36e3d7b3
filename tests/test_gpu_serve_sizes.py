"""Serving calls of sizes that stand near the limits of a launch."""
import ctypes

import torch
import pytest

from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")


def test_kv_read_of_many_slots():
    """More than 2^26 rows (17 GB of outputs): read, with offsets past 32 bits, not refused."""
    say("kv read many")
    T, hk, D, ps = (1 << 23) + 77, 8, 64, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    c = lcp.PagedKVCache.empty(8, ps, hk, D, torch.bfloat16)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    slots = torch.randint(-1, 8 * ps, (T,), generator=g, device=DEV, dtype=torch.int32)
    k, v = c.read(slots)
    for got, t in ((k, c.k), (v, c.v)):
        rows = torch.cat((t.transpose(1, 2).reshape(8 * ps, hk, D), torch.zeros_like(t[:1, :, 0])))   # -1: the zeros
        for i in range(0, T, 1 << 20):
            assert torch.equal(got[i:i + (1 << 20)], rows[slots[i:i + (1 << 20)].long()]), i
    del k, v, got
    torch.cuda.empty_cache()


def test_append_does_not_look_at_the_outputs_of_k_and_v():
    """Whatever stands in those fields: the aligned kernel runs (the other one cannot launch 2^26 rows and refuses)."""
    say("append unused outputs")
    L = lcp._lib
    T, hk, D, ps = (1 << 22) + 1, 8, 64, 16
    c = lcp.PagedKVCache.empty(2, ps, hk, D, torch.bfloat16)
    for t in (c.k, c.v):
        t.fill_(3.0)
    x = torch.ones(hk, D, dtype=torch.bfloat16, device=DEV)
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    slots[T - 1] = 17
    for y, stride in ((None, 0), (0x1001, 3)):
        h = L.lcp_heads(x.data_ptr(), y, hk, 0, D, stride, stride)           # one row for all tokens
        assert L.LIB.lcp_kv_append(ctypes.byref(c.c), None, ctypes.byref(h), ctypes.byref(h), T, slots.data_ptr(), None,
                                   0, None, 0, 0, L._stream()) == L.LCP_OK
    k, v = c.read(torch.arange(2 * ps, dtype=torch.int32, device=DEV))
    for t in (k, v):
        assert (t[17] == 1).all() and (t[:17] == 3).all() and (t[18:] == 3).all()
