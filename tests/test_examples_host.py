"""Parts of the examples that need no GPU."""
import importlib.util
import os

import numpy as np
import torch

from tests import serve_ref as R

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def _example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_codes_are_those_of_the_operators():
    """The 8-bit rows between two products: the least power of two, not under 2^-126, that brings a row to 448 or less;
    zeros, rows of fp32's smallest numbers, maxima at the rule's border, rows that are not finite."""
    g = torch.Generator().manual_seed(3)
    a = torch.randn(12, 96, generator=g)
    a *= torch.tensor([1.0, 1e-3, 1e30, 1e-33, 1e-38, 0.0, 1.0, 1.0, 1.0, 1.0, 2.0 ** -126, 1e-20])[:, None]
    a[1] = torch.clamp(a[1], -1, 1)
    a[6, 5], a[7, 9] = 448.0, 448.0 + 2.0
    a[8, 3], a[9, 1] = float("inf"), float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        x = a.to(dtype)
        codes, scale = _example("sparse_mlp_block").codes(x)
        want, s = R.quantise(x.float().numpy(), "fp8")
        assert codes.dtype == torch.float8_e4m3fn and scale.dtype == torch.float32
        assert np.array_equal(scale.numpy(), s, equal_nan=True)
        assert np.array_equal(codes.view(torch.uint8).numpy(), want)
