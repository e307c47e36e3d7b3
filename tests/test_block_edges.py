"""What a decoder block's operators refuse at the edges of what their documents allow, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

import learnable_channel_permutation_amd as lcp
from learnable_channel_permutation_amd import _lib as L

P = 0x100000


def test_fast_belongs_to_8_bit_layers():
    n = ctypes.c_size_t(0)
    for dt, fast, want in ((L.LCP_E4M3, 0, L.LCP_OK), (L.LCP_E4M3, 1, L.LCP_OK), (L.LCP_BF16, 0, L.LCP_OK),
                           (L.LCP_BF16, 1, L.LCP_E_INVAL), (L.LCP_E4M3, 2, L.LCP_E_INVAL), (L.LCP_E4M3, -1, L.LCP_E_INVAL)):
        p = L.lcp_packed(P, 2 * P, 3 * P, dt, 64, 128, fast)
        assert L.LIB.lcp_sparse_linear_workspace_bytes(ctypes.byref(p), 80, ctypes.byref(n)) == want, (dt, fast)
    assert ctypes.sizeof(L.lcp_packed) == 40
    vb, mb = lcp.lcp_sparse_pack_bytes(96, 64)
    bf = torch.zeros(vb, dtype=torch.uint8), torch.zeros(mb // 4, dtype=torch.int32)
    assert lcp.SparseLinear(*bf, 96, 64).fast is False
    vb, mb = lcp.lcp_sparse_pack_e4m3_bytes(96, 64)
    f8 = torch.zeros(vb, dtype=torch.uint8), torch.zeros(mb // 4, dtype=torch.int32)
    assert lcp.SparseLinear(*f8, 96, 64, torch.ones(96)).fast is False
    assert lcp.SparseLinear(*f8, 96, 64, torch.ones(96), fast=True).fast is True
    for bad in (lambda: lcp.SparseLinear(*bf, 96, 64, fast=True), lambda: lcp.make_packed(*bf, 96, 64, None, True)):
        with pytest.raises(ValueError):
            bad()


def _kernel(file, name):
    """The source of a kernel, from its name to the end of its body."""
    path = os.path.join(os.path.dirname(os.path.abspath(lcp.__file__)), "csrc", file)
    text = open(path).read()
    at = text.index(name + "(")
    return text[at:text.index("\n}\n", at)]


def test_lanes_that_exchange_through_lds_are_fenced():
    """What a lane reads of a wave's LDS may come from another lane: no run shows a compiler that swaps the two, so the
    fences between writes and reads, and between reads and the next step's writes, are held in the source."""
    body = _kernel("linear.hip", "linear_thin_kernel")
    loop = body[body.index("while (s < KS) {"):body.index("// a round of tiles")]
    events = [m.group(0) for m in re.finditer(r"mine\[[^;]*\] = |wave_fence\(\)|mine\[n", loop)]
    kinds = ["write" if " = " in e else "fence" if "fence" in e else "read" for e in events]
    assert kinds == ["write", "fence", "read", "read", "fence"], events
    body = _kernel("norm.hip", "norm_kernel")
    kinds = re.findall(r"to_order<|wave_fence\(\)|in_order<", body)
    assert kinds == ["to_order<", "wave_fence()", "in_order<", "wave_fence()"]
