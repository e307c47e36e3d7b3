"""Serving calls that have to agree with each other to the last bit."""
import numpy as np
import pytest
import torch

from tests import serve_ref as R
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

lcp = pytest.importorskip("learnable_channel_permutation_amd")


def put(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def shifted(x):
    """The same numbers, one element off alignment."""
    y = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
    return y.copy_(x)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 48), (256, 64)])
def test_every_rotation_gives_the_bits_of_the_fp32_definition(D, rot, interleaved):
    """lcp_rope from aligned and odd addresses, both types and directions, and the queries that append rotates."""
    say("rotation bits", D, rot, interleaved)
    T, H, hk, ps = 700, 16, 2, 64
    rng = np.random.default_rng(D + rot)
    table = R.rope_table(900, R.rope_theta(rot), 1.1).astype(np.float32)
    pos = rng.integers(0, 900, T)
    x = rng.normal(size=(T, H, D)).astype(np.float32)
    xb = R.bf16(x)
    dt, dp = put(table), put(pos.astype(np.int32), torch.int32)
    back = table * np.array([1, -1], dtype=np.float32)
    for inverse in (False, True):
        for a, dtype in ((x, torch.float32), (xb, torch.bfloat16)):
            want = put(R.rope_f32(a, back if inverse else table, pos, interleaved)).to(dtype)
            q = put(a, dtype)
            for inp in (q, shifted(q)):
                out = torch.empty_like(q)
                lcp.lcp_rope(inp, out, dt, dp, interleaved=interleaved, inverse=inverse)
                assert torch.equal(out, want), (inverse, dtype, inp.data_ptr() % 16)
    cache = lcp.PagedKVCache.empty(-(-T // ps), ps, hk, D)
    kv = torch.zeros(T, hk, D, dtype=torch.bfloat16, device=DEV)
    q, slots = put(xb, torch.bfloat16), torch.arange(T, dtype=torch.int32, device=DEV)
    want = torch.empty_like(q)
    lcp.lcp_rope(q, want, dt, dp, interleaved=interleaved)
    for inp in (q, shifted(q)):
        out = torch.empty_like(q)
        cache.append(kv, kv, slots, q=inp, q_out=out, table=dt, pos=dp, interleaved=interleaved)
        assert torch.equal(out, want)


def test_a_flag_without_a_truth_value_is_its_own_error():
    say("flags")
    x, t = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(9, 32, 2, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    for kw in (dict(interleaved=torch.ones(2)), dict(inverse=torch.ones(2))):
        with pytest.raises(RuntimeError, match="ambiguous"):
            lcp.lcp_rope(x, torch.empty_like(x), t, pos, **kw)
