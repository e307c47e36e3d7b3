"""Rotary positions, the paged key/value cache and one-token attention from
their definitions, in NumPy (64 bits, or the stated fp32 sequence where codes
have to be equal to the last bit). Nothing here uses the package."""
import math

import numpy as np

U32 = 2.0 ** -24      # unit roundoff of fp32


def bf16(x):
    """Round float32 numbers to bfloat16 (nearest even), as float32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32)


def bf16_within(got, ref, tol):
    """Whether bfloat16 numbers are the rounding of something within tol of ref (rounding is monotone)."""
    return np.all((got >= bf16(np.nextafter((ref - tol).astype(np.float32), np.float32(-np.inf)))) &
                  (got <= bf16(np.nextafter((ref + tol).astype(np.float32), np.float32(np.inf)))))


# ---- rotary positions ---------------------------------------------------------
def rope_theta(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, low_turns=1.0, high_turns=32.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "by_parts":
        g = np.clip((orig_len * theta / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0, 1)
        theta = theta * (g + (1 - g) / factor)
    return theta


def rope_table(max_pos, theta, magnitude=1.0):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * theta
    return magnitude * np.stack((np.cos(a), np.sin(a)), -1)


def rope_matrix(cs, D, interleaved):
    """The D x D rotation of one token from its table row [rot / 2][2]."""
    R = np.eye(D)
    half = cs.shape[0]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cs[i]
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def rope(x, table, pos, interleaved, inverse=False):
    """x [T][H][D] -> rotated, 64 bits, one matrix a token."""
    x = np.asarray(x, dtype=np.float64)
    y = np.empty_like(x)
    for t in range(x.shape[0]):
        p = min(max(int(pos[t]), 0), table.shape[0] - 1)
        R = rope_matrix(np.asarray(table[p], dtype=np.float64), x.shape[2], interleaved)
        y[t] = x[t] @ (R if inverse else R.T)
    return y


def rope_abs(x, table, pos, interleaved):
    """Sum of the magnitudes of the products that each output is made of."""
    y = np.empty(x.shape)
    for t in range(x.shape[0]):
        p = min(max(int(pos[t]), 0), table.shape[0] - 1)
        R = rope_matrix(np.asarray(table[p], dtype=np.float64), x.shape[2], interleaved)
        y[t] = np.abs(x[t]) @ np.abs(R.T)
    return y


def rope_f32(x, table, pos, interleaved):
    """The same in fp32, every product and sum rounded by itself."""
    x = np.asarray(x, dtype=np.float32)
    cs = np.asarray(table, dtype=np.float32)[np.clip(pos, 0, table.shape[0] - 1)][:, None]
    c, s = cs[..., 0], cs[..., 1]
    half = c.shape[-1]
    y = x.copy()
    a = x[..., 0:2 * half:2] if interleaved else x[..., :half]
    b = x[..., 1:2 * half:2] if interleaved else x[..., half:2 * half]
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, v
    else:
        y[..., :half], y[..., half:2 * half] = u, v
    return y


# ---- cache formats --------------------------------------------------------------
def e4m3_values():
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 mantissa bits; S.1111.111 is NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7)
        v[c] = math.nan if e == 15 and m == 7 else x
        if c & 128:
            v[c] = -v[c]
    return v


def e4m3_encode(x):
    """Nearest code of each |x| <= 448, ties to the even code."""
    pos = e4m3_values()[:127]
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(pos[hi] == a, hi, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x, fmt):
    """fp32 rows [..., D] -> (codes uint8 / int8, scales fp32) by the definitions, in fp32."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x).max(-1)
    ok = np.isfinite(x).all(-1)
    a = np.where(ok, a, np.float32(1))
    if fmt == "fp8":
        m, e = np.frexp(a.astype(np.float64))       # a = m 2^e, 1/2 <= m < 1
        k = np.where(a > 0, e - 9 + (m > 0.875), -126)
        s = np.ldexp(1.0, np.maximum(k, -126)).astype(np.float32)
    else:
        s = np.maximum(a / np.float32(127), np.float32(2.0 ** -126))
    y = np.where(ok[..., None], x, np.float32(0)) / s[..., None]
    codes = e4m3_encode(y) if fmt == "fp8" else np.clip(np.rint(y), -127, 127).astype(np.int8)
    if fmt == "fp8":
        codes = np.where(ok[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(ok, s, np.float32(np.nan))


def dequantise(codes, scales, fmt):
    v = e4m3_values()[codes] if fmt == "fp8" else codes.astype(np.float64)
    return (v.astype(np.float32) * scales[..., None]).astype(np.float32)


# ---- attention ------------------------------------------------------------------
def attend(q, k, v, scale):
    """q [H][D], k and v [n][Hk][D] of the counted tokens: (out [H][D], lse [H],
    bounds) in 64 bits; bounds = (sum of |q k| scale, sum of p |v|) for tolerances."""
    H, D = q.shape
    n, Hk = k.shape[:2]
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    zmag, vmag = np.zeros(H), np.zeros((H, D))
    if n == 0:
        return out, lse, (zmag, vmag)
    for h in range(H):
        kh, vh = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        z = scale * (kh @ q[h])
        m = z.max()
        p = np.exp(z - m)
        out[h], lse[h] = p @ vh / p.sum(), m + np.log(p.sum())
        zmag[h] = abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
        vmag[h] = p @ np.abs(vh) / p.sum()
    return out, lse, (zmag, vmag)
