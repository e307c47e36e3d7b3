"""Cases of the serving operators that stand between the deployed sparse
projections of an attention block: rotary positions, the quantised paged
key/value cache (written and read back) and the attention of one new token
over it.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, with ``own`` set, through the package's operators; ``exact``
evaluates the definitions in 64 bits.

A case is one of three kinds:

  rope    rotary positions on the queries and keys of T tokens (``bwd``: the
          gradient, the transposed rotation)
  cache   T new tokens rotated, quantised and written into the pages, then
          ``ctx`` earlier tokens and the new ones read back for a prompt's
          attention (``ctx`` 0: one token of each of T sequences, read back)
  attend  one new token of each of B sequences over its pages

Head counts follow the widths of this repository's layers (4096, 5120 and
8192 channels) divided by the head size.
"""
import math

import torch

own = False

WIDTHS = (4096, 5120, 8192)
MAX_POS = 1 << 17


def listed():
    return [
        # a decode step of a few sequences: the rotation's latency
        dict(name="rope decode 5", kind="rope", T=5, hq=32, hk=8, D=128, rot=128, inter=False, bwd=False,
             dtype="bf16", packed=True),
        # a long prompt of a multi-head layer of 5120 channels
        dict(name="rope prompt 16384", kind="rope", T=16384, hq=40, hk=40, D=128, rot=128, inter=True, bwd=False,
             dtype="bf16", packed=True),
        # the gradient in training, bf16, grouped heads of a layer of 8192 channels
        dict(name="rope grad 8191", kind="rope", T=8191, hq=64, hk=8, D=128, rot=128, inter=False, bwd=True,
             dtype="bf16", packed=False),
        # the gradient in fp32 with part of an 80-wide head rotated, an odd number of tokens
        dict(name="rope grad part fp32", kind="rope", T=2051, hq=64, hk=64, D=80, rot=32, inter=False, bwd=True,
             dtype="f32", packed=False),
        # one new token of each of 33 sequences into an fp8 cache
        dict(name="cache decode 33 fp8", kind="cache", T=33, ctx=0, hq=32, hk=8, D=128, rot=128, inter=False,
             fmt="fp8", page=64),
        # a prompt's second chunk, int8, everything so far read back
        dict(name="cache chunk 2048 int8", kind="cache", T=2048, ctx=6000, hq=64, hk=8, D=128, rot=64, inter=True,
             fmt="int8", page=16),
        # a long prompt of a multi-head layer of 4096 channels in one chunk, fp8, odd length
        dict(name="cache prompt 16001 fp8", kind="cache", T=16001, ctx=4096, hq=32, hk=32, D=128, rot=128,
             inter=False, fmt="fp8", page=48),
        # one sequence, short context, multi-head, unquantised: the attention's latency
        dict(name="attend 1 x 333", kind="attend", B=1, maxlen=333, hq=32, hk=32, D=128, fmt="bf16", page=16, window=0),
        # an ordinary batch of ragged sequences over an fp8 cache
        dict(name="attend 48 x 4096 fp8", kind="attend", B=48, maxlen=4096, hq=64, hk=8, D=128, fmt="fp8", page=64,
             window=0),
        # few rows, a long context: the split over the length carries it
        dict(name="attend 2 x 131071 int8", kind="attend", B=2, maxlen=131071, hq=32, hk=8, D=128, fmt="int8",
             page=64, window=0),
        # a sliding window over wide heads
        dict(name="attend 24 window 4096", kind="attend", B=24, maxlen=16384, hq=16, hk=4, D=256, fmt="bf16", page=32,
             window=4096),
        # a large serving batch, unquantised
        dict(name="attend 128 x 8192 bf16", kind="attend", B=128, maxlen=8192, hq=64, hk=8, D=128, fmt="bf16",
             page=128, window=0),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "attend", "attend"])
    width = rng.choice(WIDTHS)
    if kind == "rope":
        D = rng.choice([64, 80, 128, 128, 256])
        hq = (5120 if width % D else width) // D
        hk = hq // rng.choice([g for g in (1, 2, 4, 8) if hq % g == 0])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rot = rng.choice([D, D, D // 2, 32])
        most = 16384 * 80 * 128 // ((hq + hk) * D * (2 if dtype == "f32" else 1))
        return dict(kind=kind, T=_log(rng, 1, most), hq=hq, hk=hk, D=D, rot=rot, inter=rng.random() < 0.5,
                    bwd=rng.random() < 0.5, dtype=dtype, packed=rng.random() < 0.5)
    D = rng.choice([64, 128, 128, 256])
    hq = width // D
    hk = hq // rng.choice([g for g in (1, 2, 4, 5, 8, 16) if hq % g == 0])
    fmt = rng.choice(["bf16", "fp8", "fp8", "int8"])
    page = rng.choice([16, 32, 48, 64, 128])
    if kind == "cache":
        ctx = rng.randint(0, 8192)
        most = (1100000000 - 6 * ctx * hk * D) // (D * (4 * hq + 12 * hk))
        T = _log(rng, 1, min(16001, most))
        if T <= 256 and rng.random() < 0.5:
            ctx = 0
        return dict(kind=kind, T=T, ctx=ctx, hq=hq, hk=hk, D=D, rot=rng.choice([D, D, D // 2]),
                    inter=rng.random() < 0.5, fmt=fmt, page=page)
    B = _log(rng, 1, 128)
    most = 128 * 8192 * 8 * 128 // (B * hk * D * (1 if fmt == "bf16" else 2))
    maxlen = _log(rng, 16, max(16, min(131071, most)))
    window = rng.choice([0, 0, 0, max(1, maxlen // 3)])
    return dict(kind=kind, B=B, maxlen=maxlen, hq=hq, hk=hk, D=D, fmt=fmt, page=page, window=window)


def _lengths(case):
    """Cached tokens of each sequence: the longest first, the others spread
    over the range; an empty one in larger batches."""
    B, n = case["B"], case["maxlen"]
    lens = [n] + [1 + int(n * ((i * 0.6180339887) % 1.0)) for i in range(1, B)]
    lens = [min(n, x) for x in lens]
    if B >= 16:
        lens[B // 2] = 0
    return lens


def _esize(fmt):
    return 2 if fmt == "bf16" else 1


def work(case):
    if case["kind"] == "rope":
        e = 4 if case["dtype"] == "f32" else 2
        n = case["T"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * n * case["D"] * e + case["T"] * (case["rot"] * 4 + 4), "flops": 3 * n * case["rot"]}
    D, hk, e = case["D"], case["hk"], _esize(case["fmt"])
    scale = 0 if case["fmt"] == "bf16" else 4
    if case["kind"] == "cache":
        T, R = case["T"], case["T"] + case["ctx"]
        q = T * case["hq"] * D
        kv = 2 * T * hk
        back = 2 * R * hk
        new = 2 * q * 2 + kv * (D * (2 + e) + scale) + T * (case["rot"] * 4 + 8)
        return {"bytes": new + back * (D * (2 + e) + scale) + 4 * R,
                "flops": 3 * T * (case["hq"] + hk) * case["rot"] + 3 * kv * D + back * D}
    w = case["window"]
    tokens = sum(min(n, w) if w else n for n in _lengths(case))
    rows = case["B"] * case["hq"]
    return {"bytes": 2 * tokens * hk * (D * e + scale) + rows * (4 * D + 4) + 4 * (case["B"] + tokens // case["page"]),
            "flops": 4 * tokens * case["hq"] * D}


def _table(rot, dev):
    """cos and sin of every position and pair, [MAX_POS][rot/2][2] fp32: base
    500000, low frequencies stretched 8 times for contexts beyond 16384, high
    ones kept, a linear ramp between 1 and 32 turns of the original context."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    theta = 500000.0 ** (-2.0 * i / rot)
    turns = 16384 * theta / (2 * math.pi)
    g = ((turns - 1.0) / 31.0).clamp(0, 1)
    theta = theta * (g + (1 - g) / 8.0)
    a = torch.arange(MAX_POS, dtype=torch.float64, device=dev)[:, None] * theta
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


def _power_scale(a):
    """The power of two that brings fp32 maxima a into e4m3's range of 448."""
    bits = a.view(torch.int32)
    k = (bits >> 23) - 127
    e = (k - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=-126)
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x, fmt):
    """fp32 rows -> (codes, scales)."""
    a = x.abs().amax(-1)
    if fmt == "fp8":
        s = _power_scale(a)
        return (x / s[..., None]).to(torch.float8_e4m3fn), s
    s = (a / 127).clamp(min=2.0 ** -126)
    return (x / s[..., None]).round().clamp(-127, 127).to(torch.int8), s


def _rows(codes):
    """Codes in a type that indexing takes."""
    return codes.view(torch.uint8) if codes.dtype == torch.float8_e4m3fn else codes


def _values(codes, like):
    """Indexed codes -> fp32."""
    return (codes.view(like) if like == torch.float8_e4m3fn else codes).float()


def _pages(pages, case, gen, dev):
    """Pages filled with keys (a few channels several times larger) and values."""
    hk, ps, D, fmt = case["hk"], case["page"], case["D"], case["fmt"]
    dt = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    gain = torch.exp(0.5 * torch.randn(hk, 1, D, generator=gen, device=dev))
    out = []
    for side in range(2):
        codes = torch.empty(pages, hk, ps, D, dtype=dt, device=dev)
        scales = None if fmt == "bf16" else torch.empty(pages, hk, ps, dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (hk * ps * D))
        for i in range(0, pages, step):
            x = torch.randn(min(step, pages - i), hk, ps, D, generator=gen, device=dev)
            if side == 0:
                x *= gain
            if fmt == "bf16":
                codes[i:i + step] = x.bfloat16()
            else:
                c, s = _quantise(x, fmt)
                _rows(codes)[i:i + step] = _rows(c)
                scales[i:i + step] = s
        out += [codes, scales]
    return {"k_pages": out[0], "k_scale": out[1], "v_pages": out[2], "v_scale": out[3]}


def _heads(T, counts, D, packed, dtype, gen, dev):
    """Head rows [T][h][D] of a projection's output: views of one row per
    token when packed, else tensors of their own."""
    if packed:
        x = torch.randn(T, sum(counts) * D, generator=gen, device=dev).to(dtype)
        return [y.view(T, -1, D) for y in x.split([c * D for c in counts], dim=1)]
    return [torch.randn(T, c, D, generator=gen, device=dev).to(dtype) for c in counts]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    D, hq, hk = case["D"], case["hq"], case["hk"]
    if case["kind"] == "rope":
        T = case["T"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        q, k, _ = _heads(T, (hq, hk, hk), D, case["packed"], dtype, gen, dev)
        if T <= 64:   # decode: each token at its own sequence's position
            pos = torch.randint(0, MAX_POS, (T,), generator=gen, device=dev)
        else:         # a run of tokens from some place on
            pos = torch.arange(T, device=dev) + int(torch.randint(0, MAX_POS - T, (1,), generator=gen, device=dev))
        s.update(q=q, k=k, pos=pos.int(), table=_table(case["rot"], dev))
        return s
    ps = case["page"]
    if case["kind"] == "cache":
        T, ctx = case["T"], case["ctx"]
        n = T if ctx == 0 and T <= 256 else -(-(ctx + T) // ps)
        s.update(_pages(n + 3, case, gen, dev))
        order = torch.randperm(n + 3, generator=gen, device=dev)
        if ctx == 0 and T <= 256:
            off = torch.randint(0, ps, (T,), generator=gen, device=dev)
            slots, pos = order[:T] * ps + off, torch.randint(0, MAX_POS, (T,), generator=gen, device=dev)
        else:
            t = torch.arange(ctx + T, device=dev)
            slots, pos = order[t // ps] * ps + t % ps, t[ctx:]
        q, k, v = _heads(T, (hq, hk, hk), D, True, torch.bfloat16, gen, dev)
        s.update(q=q, k=k, v=v, pos=pos.int().contiguous(), read=slots.int().contiguous(),
                 slots=slots[-T:].int().contiguous(), table=_table(case["rot"], dev))
        return s
    lens = _lengths(case)
    need = [-(-n // ps) for n in lens]
    total = sum(need) + 2
    s.update(_pages(total, case, gen, dev))
    order = torch.randperm(total, generator=gen, device=dev).tolist()
    P = max(need)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (P - n))
        at += n
    s.update(table=torch.tensor(table, dtype=torch.int32).to(dev), lens=torch.tensor(lens, dtype=torch.int32).to(dev),
             q=torch.randn(case["B"], hq, D, generator=gen, device=dev).bfloat16())
    return s


def _rotate(x, cs, case, bwd=False):
    """The rotation of fp32 rows [T][h][D] by cs [T][1][rot/2][2]."""
    r = case["rot"]
    c, s = cs[..., 0], cs[..., 1]
    if bwd:
        s = -s
    if case["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return y if r == x.shape[-1] else torch.cat((y, x[..., r:]), dim=-1)


def _plain_rope(s):
    case = s["case"]
    cs = s["table"][s["pos"]][:, None]
    return {n: _rotate(s[n].float(), cs, case, case["bwd"]).to(s[n].dtype) for n in ("q", "k")}


def _plain_cache(s):
    case = s["case"]
    ps = case["page"]
    cs = s["table"][s["pos"]][:, None]
    out = {"q": _rotate(s["q"].float(), cs, case).bfloat16()}
    page, off = s["slots"] // ps, s["slots"] % ps
    rpage, roff = s["read"] // ps, s["read"] % ps
    k, v = _rotate(s["k"].float(), cs, case), s["v"].float()
    if case["fmt"] == "bf16":
        s["k_pages"][page, :, off], s["v_pages"][page, :, off] = k.bfloat16(), v.bfloat16()
        out["k"], out["v"] = s["k_pages"][rpage, :, roff], s["v_pages"][rpage, :, roff]
        return out
    (kc, ksc), (vc, vsc) = _quantise(k, case["fmt"]), _quantise(v, case["fmt"])
    _rows(s["k_pages"])[page, :, off], s["k_scale"][page, :, off] = _rows(kc), ksc
    _rows(s["v_pages"])[page, :, off], s["v_scale"][page, :, off] = _rows(vc), vsc
    like = s["k_pages"].dtype
    out["k"] = (_values(_rows(s["k_pages"])[rpage, :, roff], like) * s["k_scale"][rpage, :, roff, None]).bfloat16()
    out["v"] = (_values(_rows(s["v_pages"])[rpage, :, roff], like) * s["v_scale"][rpage, :, roff, None]).bfloat16()
    return out


def _gathered(s, side, table):
    """The pages of every sequence as fp32 [B][hk][P * page][D]."""
    codes = s[side + "_pages"]
    B, P = table.shape
    x = _values(_rows(codes)[table], codes.dtype)
    if s[side + "_scale"] is not None:
        x = x * s[side + "_scale"][table][..., None]
    return x.transpose(1, 2).reshape(B, codes.shape[1], P * codes.shape[2], codes.shape[3])


def _plain_attend(s):
    case = s["case"]
    B, hq, hk, D = case["B"], case["hq"], case["hk"], case["D"]
    table, lens = s["table"].clamp(min=0), s["lens"][:, None]
    t = torch.arange(table.shape[1] * case["page"], device=lens.device)[None]
    masked = t >= lens
    if case["window"]:
        masked = masked | (t < lens - case["window"])
    z = torch.matmul(s["q"].float().view(B, hk, hq // hk, D), _gathered(s, "k", table).transpose(-1, -2)) * D ** -0.5
    z = z.masked_fill(masked[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(s, "v", table)) / total.clamp(min=1e-30)
    return {"out": o.view(B, hq, D).bfloat16(), "lse": (m + total.log()).view(B, hq)}


def run(state):
    s = state
    case = s["case"]
    kind = case["kind"]
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "attend": _plain_attend}[kind](s)
    import learnable_channel_permutation_amd as lcp
    if kind == "rope":
        q, k = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        lcp.lcp_rope(s["q"], q, s["table"], s["pos"], k=s["k"], k_out=k, interleaved=case["inter"],
                     inverse=case["bwd"])
        return {"q": q, "k": k}
    cache = lcp.PagedKVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if kind == "cache":
        q = torch.empty_like(s["q"])
        cache.append(s["k"], s["v"], s["slots"], q=s["q"], q_out=q, table=s["table"], pos=s["pos"],
                     interleaved=case["inter"])
        k, v = cache.read(s["read"])
        return {"q": q, "k": k, "v": v}
    out, lse = cache.attend(s["q"], s["table"], s["lens"], max_len=case["maxlen"], window=case["window"])
    return {"out": out, "lse": lse}


def _exact_rotate(x, cs, case, bwd=False):
    """A rotation of each pair as a complex number, in 64 bits."""
    r = case["rot"]
    w = torch.complex(cs[..., 0].double(), cs[..., 1].double())[:, None]
    w = w.conj() if bwd else w
    x = x.double()
    y = x.clone()
    if case["inter"]:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * w
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * w
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _exact_stored(x, fmt):
    """The value that the cache holds for each entry of 64-bit rows."""
    if fmt == "bf16":
        return x
    a = x.abs().amax(-1, keepdim=True)
    if fmt == "int8":
        s = (a / 127).clamp(min=2.0 ** -126)
        return torch.round(x / s) * s
    m, e = torch.frexp(a)                       # a = m 2^e, m in [1/2, 1)
    shift = (e - 9 + (m > 0.875).int()).clamp(min=-126).double()
    s = torch.exp2(shift)
    x = x / s
    _, e = torch.frexp(x)                       # three mantissa bits, exponents from 2^-6 on
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step * s


def _exact_held(s, side, page, off):
    """What the pages hold, [n][hk][D] in 64 bits."""
    codes = s[side + "_pages"]
    x = _values(_rows(codes)[page, :, off], codes.dtype).double()
    return x if s[side + "_scale"] is None else x * s[side + "_scale"][page, :, off, None].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        cs = s["table"][s["pos"].long()]
        return {n: _exact_rotate(s[n], cs, case, case["bwd"]) for n in ("q", "k")}
    ps = case["page"]
    if case["kind"] == "cache":
        cs = s["table"][s["pos"].long()]
        out = {"q": _exact_rotate(s["q"], cs, case)}
        new = {"k": _exact_rotate(s["k"], cs, case), "v": s["v"].double()}
        old = s["read"][:s["read"].shape[0] - case["T"]].long()
        for side in ("k", "v"):
            held = _exact_held(s, side, old // ps, old % ps)
            out[side] = torch.cat((held, _exact_stored(new[side], case["fmt"])))
        return out
    B, hq, hk, D, w = case["B"], case["hq"], case["hk"], case["D"], case["window"]
    out = torch.zeros(B, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        t = torch.arange(max(0, n - w) if w else 0, n, device="cuda")
        page, off = s["table"][b].long()[t // ps], t % ps
        k, v = (_exact_held(s, side, page, off).transpose(0, 1).contiguous() for side in ("k", "v"))
        z = torch.matmul(s["q"][b].double().view(hk, hq // hk, D), k.transpose(1, 2).contiguous()) / math.sqrt(D)
        lse[b] = torch.logsumexp(z, -1).view(hq)
        out[b] = torch.matmul(torch.softmax(z, -1), v).view(hq, D)
    return {"out": out, "lse": lse}
