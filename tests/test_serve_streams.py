"""Serving calls on a stream of their own (no GPU: allocations are watched, the
native calls are stood in for)."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import learnable_channel_permutation_amd as lcp


class Allocations(TorchDispatchMode):
    """Which stream was current at each allocation."""

    def __init__(self, current):
        super().__init__()
        self.current, self.seen = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "empty" in func.name():
            self.seen.append(self.current[-1])
        return func(*args, **(kwargs or {}))


class Native:
    """Makes what is missing, as the native module does on the current stream."""

    @staticmethod
    def read(c, slots, k_out, v_out, stream):
        made = [torch.empty(slots.shape[0], c.heads, c.D) if t is None else t for t in (k_out, v_out)]
        return (0, *made)

    @staticmethod
    def attend(c, q, pages, lens, max_len, out, lse, ws, scale, window, make, stream):
        torch.empty(16 if ws is None else 0)
        return 0, torch.empty_like(q) if out is None else out, torch.empty(q.shape[:2]) if lse is None else lse


@pytest.mark.parametrize("call", ["read", "read one", "attend", "attend workspace"])
def test_allocations_belong_to_the_stream_that_uses_them(call, monkeypatch):
    """Memory of another stream's pool may still be in use there: the given stream does not wait for it."""
    class Side:
        device = torch.device("cuda", 0)
        cuda_stream = 7

    side, current = Side(), ["caller's"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16)
    cache = lcp.PagedKVCache(k, k.clone(), s, s.clone())
    slots = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pages, lens = torch.zeros(3, 900, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    given = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(3, 4)
    kept = []
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append(s))
    monkeypatch.setattr(lcp._lib, "_serve", Native)
    with Allocations(current) as watched:
        if call == "read":
            cache.read(slots, stream=side)
        elif call == "read one":
            assert cache.read(slots, v_out=given, stream=side)[1] is given
        elif call == "attend":
            cache.attend(q, pages, lens, stream=side)
        else:
            cache.attend(q, pages, lens, out=out, lse=lse, stream=side)
    assert watched.seen and all(x is side for x in watched.seen)
    # results that were made are used by the caller's stream next: kept until it is done with them
    assert kept == ["caller's"] * {"read": 2, "read one": 1, "attend": 2, "attend workspace": 0}[call]


@pytest.mark.parametrize("max_len", [None, 64])
def test_a_call_that_makes_nothing_passes_its_stream_on(max_len, monkeypatch):
    """Outputs given and no workspace needed: no change of the current stream, which costs more than the call."""
    class Handle:
        cuda_stream = 7

    got = []
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: pytest.fail("the current stream was changed"))
    monkeypatch.setattr(Native, "attend", staticmethod(lambda *a: (got.append(a[-1]), (0, a[5], a[6]))[1]))
    monkeypatch.setattr(lcp._lib, "_serve", Native)
    cache = lcp.PagedKVCache.__new__(lcp.PagedKVCache)
    cache._c = lcp._lib.lcp_kv_cache(4096, 8192, 4096, 4096, lcp._lib.LCP_KV_INT8, 4, 16, 2, 64)
    q, h = torch.zeros(3, 4, 64, dtype=torch.bfloat16), Handle()
    out, lse = torch.zeros_like(q), torch.zeros(3, 4)
    assert cache.attend(q, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), max_len=max_len, out=out,
                        lse=lse, stream=h)[0] is out
    assert got == [h]
