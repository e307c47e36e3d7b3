"""The references of the serving operators against independent facts (no GPU):
codes against a search over all values, the rotation's gradient against
differences, the softmax against its shift invariance."""
import math

import numpy as np
import pytest

from tests import serve_ref as R


def test_e4m3_nearest_of_all_codes():
    vals = R.e4m3_values()
    finite = np.where(np.isnan(vals))[0]
    assert list(finite) == [127, 255] and np.nanmax(vals) == 448 and vals[1] == 2.0 ** -9
    rng = np.random.default_rng(1)
    x = np.concatenate((rng.uniform(-448, 448, 2000), rng.normal(0, 0.02, 2000), vals[:127],
                        (vals[:126] + vals[1:127]) / 2))        # values and exact ties
    got = vals[R.e4m3_encode(x)]
    err = np.abs(got - x)
    best = np.abs(vals[None, :127] - np.abs(x)[:, None]).min(1)
    assert np.array_equal(err, best)
    ties = R.e4m3_encode((vals[:126] + vals[1:127]) / 2)
    assert np.all(ties % 2 == 0)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_quantised_values_within_half_a_step(fmt):
    rng = np.random.default_rng(2)
    x = (rng.normal(size=(64, 128)) * 10.0 ** rng.uniform(-6, 6, (64, 1))).astype(np.float32)
    x[5] = 0
    x[6] = 448.0 / 3
    codes, s = R.quantise(x, fmt)
    y = R.dequantise(codes, s, fmt).astype(np.float64)
    a = np.abs(x).max(-1, keepdims=True).astype(np.float64)
    if fmt == "int8":
        step = a / 127
    else:
        # a / s in (224, 448]: half a step of the value's own binade, at least the smallest step
        assert np.all((a / s[:, None] <= 448) & ((a / s[:, None] > 224) | (a == 0)))
        step = np.maximum(np.abs(x) * 2.0 ** -3, s[:, None] * 2.0 ** -9)
    assert np.all(np.abs(y - x) <= step / 2 * (1 + 1e-6) + 1e-300)
    bad = x.copy()
    bad[3, 7] = np.nan
    bad[4, 9] = np.inf
    _, s = R.quantise(bad, fmt)
    assert np.isnan(s[3]) and np.isnan(s[4]) and np.isfinite(np.delete(s, [3, 4])).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_against_differences_and_inverse(interleaved):
    rng = np.random.default_rng(3)
    table = R.rope_table(50, R.rope_theta(12), magnitude=1.25)
    pos = np.array([0, 7, 49])
    x, g = rng.normal(size=(3, 2, 16)), rng.normal(size=(3, 2, 16))
    f = lambda z: float((R.rope(z, table, pos, interleaved) * g).sum())    # noqa: E731
    grad = R.rope(g, table, pos, interleaved, inverse=True)
    h = 1e-6
    for idx in [(0, 0, 0), (1, 1, 5), (2, 0, 11), (1, 0, 13), (2, 1, 15)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((f(x + e) - f(x - e)) / (2 * h) - grad[idx]) < 1e-7
    unit = R.rope_table(50, R.rope_theta(12))
    back = R.rope(R.rope(x, unit, pos, interleaved), unit, pos, interleaved, inverse=True)
    assert np.abs(back - x).max() < 1e-14
    # relative positions: q.k depends on the distance alone
    q, k = rng.normal(size=(1, 1, 12)), rng.normal(size=(1, 1, 12))
    dot = [float((R.rope(q, unit, [a], interleaved) * R.rope(k, unit, [b], interleaved)).sum())
           for a, b in ((9, 4), (45, 40))]
    assert abs(dot[0] - dot[1]) < 1e-12


def test_rope_f32_sequence_close_to_definition():
    rng = np.random.default_rng(4)
    table = R.rope_table(40, R.rope_theta(32)).astype(np.float32)
    pos = rng.integers(0, 40, 9)
    x = rng.normal(size=(9, 3, 64)).astype(np.float32)
    for inter in (False, True):
        d = R.rope_f32(x, table, pos, inter) - R.rope(x, table, pos, inter)
        assert np.abs(d).max() < 4 * 2 * R.U32 * np.abs(x).max()


def test_rope_scalings():
    plain = R.rope_theta(64, base=10000.0)
    assert np.allclose(R.rope_theta(64, scaling="linear", factor=4.0), plain / 4)
    b = R.rope_theta(64, scaling="base", factor=4.0)
    assert np.isclose(b[0], plain[0]) and np.isclose(b[-1], plain[-1] / 4)
    p = R.rope_theta(64, scaling="by_parts", factor=4.0, orig_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(p[turns >= 32], plain[turns >= 32]) and np.allclose(p[turns <= 1], plain[turns <= 1] / 4)
    assert np.all(p <= plain) and np.all(p >= plain / 4)


def test_attention_by_parts_joins():
    """Attention of two halves joined by their lse equals the whole."""
    rng = np.random.default_rng(5)
    q, k, v = rng.normal(size=(4, 8)), rng.normal(size=(21, 2, 8)), rng.normal(size=(21, 2, 8))
    o, lse, _ = R.attend(q, k, v, 0.3)
    a, b = R.attend(q, k[:8], v[:8], 0.3), R.attend(q, k[8:], v[8:], 0.3)
    wa, wb = np.exp(a[1] - lse)[:, None], np.exp(b[1] - lse)[:, None]
    assert np.abs(wa * a[0] + wb * b[0] - o).max() < 1e-12
    e = R.attend(q, k[:0], v[:0], 0.3)
    assert np.all(e[0] == 0) and np.all(e[1] == -np.inf)
