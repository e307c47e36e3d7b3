"""Serving calls on a stream of their own that make their outputs and workspace
themselves, next to queued work of the current stream."""
import math

import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.gpu_util import DEV, down, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")


@pytest.mark.parametrize("what", ["read", "attend"])
def test_what_a_call_makes_does_not_touch_the_current_streams_memory(what):
    """A buffer freed while queued work still reads it may be given to the current stream only, whose order protects
    it: a call on another stream must neither overwrite it nor be overwritten."""
    say("serve allocations", what)
    hq, hk, D, ps, n = 8, 2, 128, 64, 6000
    pages = -(-n // ps)
    g = torch.Generator().manual_seed(3)
    c = lcp.PagedKVCache.empty(pages, ps, hk, D, torch.bfloat16)
    k, v = (torch.randn(n, hk, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    c.append(k, v, slots)
    q = torch.randn(1, hq, D, generator=g).bfloat16().to(DEV)
    table, lens = torch.arange(pages, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV)
    need = lcp.lcp_attn_decode_workspace_bytes(c.c, 1, hq, n)
    assert need > 0                                    # cut over the workgroups: the call makes a workspace, too
    sizes = [k.nbytes, v.nbytes] if what == "read" else [need, q.nbytes, hq * 4]
    a = torch.randn(4096, 4096, device=DEV).bfloat16()
    want = R.attend(down(q)[0], down(k), down(v), D ** -0.5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full((x,), 5, dtype=torch.uint8, device=DEV) for x in sizes]
        torch.cuda.synchronize()
        for _ in range(40):                            # some milliseconds of queued work ahead of the readers
            a = (a @ a).clamp_(-1, 1)
        seen = [x.clone() for x in held]
        del held
        got = c.read(slots, stream=side) if what == "read" else c.attend(q, table, lens, stream=side)
        for x in seen:
            x += 1                                     # the current stream goes on allocating and writing
        torch.cuda.current_stream().wait_stream(side)
        if what == "read":
            assert torch.equal(got[0], k) and torch.equal(got[1], v)
        else:
            assert np.abs(down(got[0])[0] - want[0]).max() < 2.0 ** -8 * np.abs(want[0]).max()
            assert np.abs(down(got[1])[0] - want[1]).max() < 1e-5 and math.isfinite(want[1].max())
        assert all(bool((x == 6).all()) for x in seen)
        del got
