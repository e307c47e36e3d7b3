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
