"""Refusals of the serving entry points (no GPU: every call is rejected before
any HIP call) and the argument checks of their Python forms."""
import ctypes
import math

import pytest
import torch

P = 0x100000


def _lib():
    from learnable_channel_permutation_amd import _lib as L
    return L


def _rows(L, heads=4, x=P, y=2 * P, xt=512, xh=128, yt=512, yh=128):
    return L.lcp_heads(x, y, heads, xt, xh, yt, yh)


def test_rope_table_refusals():
    L = _lib()

    def call(n=10, table=P, **kw):
        return L.LIB.lcp_rope_table(ctypes.byref(L.make_rope_cfg(**{"rot_dim": 64, **kw})), n, table, None)

    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=math.nan), dict(magnitude=0.0),
                dict(magnitude=math.inf), dict(n=0), dict(table=None), dict(table=P + 4), dict(n=1 << 27),
                dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.inf),
                dict(scaling="base", factor=2.0, rot_dim=2), dict(scaling="by_parts", factor=2.0),
                dict(scaling="by_parts", factor=2.0, orig_len=10.0, low_turns=4.0, high_turns=4.0)):
        assert call(**bad) == L.LCP_E_INVAL, bad
    assert call(rot_dim=1026) == L.LCP_E_UNSUPPORTED
    c = L.make_rope_cfg(64)
    c.scaling = 9
    assert L.LIB.lcp_rope_table(ctypes.byref(c), 10, P, None) == L.LCP_E_UNSUPPORTED
    assert L.LIB.lcp_rope_table(None, 10, P, None) == L.LCP_E_INVAL


def test_rope_refusals():
    L = _lib()

    def call(q=None, k=None, dt=L.LCP_BF16, T=5, D=128, table=P, n=10, pos=P, rot=128, inter=0, inv=0):
        q = _rows(L) if q is None else q
        return L.LIB.lcp_rope(ctypes.byref(q), None if k is None else ctypes.byref(k), dt, T, D, table, n, pos, rot,
                              inter, inv, None)

    for bad in (dict(T=0), dict(T=-1), dict(table=None), dict(table=P + 8), dict(pos=None), dict(n=0), dict(rot=0),
                dict(rot=63), dict(rot=130), dict(D=1, rot=1), dict(inter=2), dict(inv=-1),
                dict(q=_rows(L, heads=0)), dict(q=_rows(L, x=0)), dict(q=_rows(L, y=0)), dict(q=_rows(L, x=P + 1)),
                dict(q=_rows(L, xt=-512)), dict(q=_rows(L, yt=500)), dict(q=_rows(L, yh=127)), dict(q=_rows(L, yt=0)),
                dict(q=_rows(L, x=P, y=P, xt=1024)), dict(k=_rows(L, x=0)), dict(k=_rows(L, yt=100)),
                dict(dt=L.LCP_F32, q=_rows(L, x=P + 2)), dict(q=_rows(L, xt=1 << 50)), dict(pos=P + 2)):
        assert call(**bad) == L.LCP_E_INVAL, bad
    assert call(dt=7) == L.LCP_E_UNSUPPORTED
    assert call(D=1026, rot=64, q=_rows(L, yt=1 << 20, yh=1 << 11)) == L.LCP_E_UNSUPPORTED
    assert L.LIB.lcp_rope(None, None, L.LCP_BF16, 1, 64, P, 1, P, 64, 0, 0, None) == L.LCP_E_INVAL


def _cache(L, **kw):
    f = dict(k=P, v=2 * P, k_scale=3 * P, v_scale=4 * P, format=L.LCP_KV_E4M3, pages=10, page_size=16, heads=4, D=128)
    f.update(kw)
    return L.lcp_kv_cache(*[f[n] for n, _ in L.lcp_kv_cache._fields_])


BAD_CACHE = [(dict(k=None), -1), (dict(v=None), -1), (dict(v=P), -1), (dict(k=P + 8), -1), (dict(k_scale=None), -1),
             (dict(v_scale=P + 4), -1), (dict(pages=0), -1), (dict(heads=0), -1), (dict(D=-64), -1),
             (dict(page_size=0), -1), (dict(pages=1 << 27), -1), (dict(format=3), -2), (dict(format=-1), -2),
             (dict(D=96), -2), (dict(page_size=24), -2), (dict(page_size=8192), -2)]


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_cache_refusals(bad, code):
    L = _lib()
    c = ctypes.byref(_cache(L, **bad))
    r = _rows(L)
    assert L.LIB.lcp_kv_append(c, None, ctypes.byref(r), ctypes.byref(r), 3, P, None, 0, None, 0, 0, None) == code
    assert L.LIB.lcp_kv_read(c, P, 3, P, 2 * P, L.LCP_BF16, None) == code
    n = ctypes.c_size_t(0)
    assert L.LIB.lcp_attn_decode_workspace_bytes(c, 1, 4, 100, 0, ctypes.byref(n)) == code
    assert L.LIB.lcp_attn_decode(c, P, 512, 1, 4, P, 10, P, 100, 0.1, 0, P, L.LCP_BF16, None, P, 1 << 30, None) == code


def test_append_and_read_refusals():
    L = _lib()

    def app(q=None, k="d", v="d", T=3, slots=P, table=P, n=10, pos=P, rot=128, inter=0, c=None):
        k, v = (_rows(L) if x == "d" else x for x in (k, v))
        r = lambda x: None if x is None else ctypes.byref(x)       # noqa: E731
        return L.LIB.lcp_kv_append(r(c or _cache(L)), r(q), r(k), r(v), T, slots, table, n, pos, rot, inter, None)

    for bad in (dict(k=None), dict(v=None), dict(T=0), dict(slots=None), dict(slots=P + 2), dict(pos=P + 1), dict(k=_rows(L, heads=3)),
                dict(v=_rows(L, heads=5)), dict(k=_rows(L, x=P + 1)), dict(v=_rows(L, x=0)), dict(pos=None), dict(n=0),
                dict(rot=0), dict(rot=144), dict(inter=3), dict(table=P + 4), dict(q=_rows(L, y=0)),
                dict(q=_rows(L), table=None), dict(q=_rows(L, yt=100))):
        assert app(**bad) == L.LCP_E_INVAL, bad
    assert app(rot=24) == L.LCP_E_UNSUPPORTED
    c = ctypes.byref(_cache(L))
    rd = L.LIB.lcp_kv_read
    assert rd(c, None, 3, P, 2 * P, 1, None) == L.LCP_E_INVAL
    assert rd(c, P, 0, P, 2 * P, 1, None) == L.LCP_E_INVAL
    assert rd(c, P, 3, None, 2 * P, 1, None) == L.LCP_E_INVAL
    assert rd(c, P, 3, P, P, 1, None) == L.LCP_E_INVAL
    assert rd(c, P, 3, P + 8, 2 * P, 1, None) == L.LCP_E_INVAL
    assert rd(c, P, 3, P, 2 * P, 5, None) == L.LCP_E_UNSUPPORTED


def test_attend_refusals():
    L = _lib()

    def call(q=P, row=512, B=2, hq=4, pages=P, mp=10, lens=P, ml=100, scale=0.1, window=0, out=P, odt=1, lse=None,
             ws=P, n=1 << 30):
        return L.LIB.lcp_attn_decode(ctypes.byref(_cache(L)), q, row, B, hq, pages, mp, lens, ml, scale, window, out,
                                     odt, lse, ws, n, None)

    for bad in (dict(q=None), dict(q=P + 8), dict(row=504), dict(row=516), dict(B=0), dict(hq=0), dict(hq=6),
                dict(pages=None), dict(mp=0), dict(lens=None), dict(ml=-1), dict(ml=161), dict(scale=math.nan),
                dict(scale=math.inf), dict(window=-1), dict(out=None), dict(out=P + 4), dict(lse=P + 2),
                dict(pages=P + 1), dict(lens=P + 2), dict(B=1 << 23), dict(ml=16000, mp=1000, ws=None)):
        assert call(**bad) == L.LCP_E_INVAL, bad
    assert call(odt=4) == L.LCP_E_UNSUPPORTED
    c = _cache(L)
    need = L.lcp_attn_decode_workspace_bytes(c, 2, 4, 16000)       # long enough to be split
    assert need > 0 and need % 256 == 0
    for bad in (dict(ws=P + 128), dict(n=0), dict(n=need - 1)):
        assert call(ml=16000, mp=1000, **bad) == L.LCP_E_WORKSPACE, bad
    with pytest.raises(L.LcpError) as e:
        L.lcp_attn_decode_workspace_bytes(c, 0, 4, 160)
    assert e.value.code == L.LCP_E_INVAL
    assert L.LIB.lcp_attn_decode_workspace_bytes(ctypes.byref(c), 2, 4, 160, 0, None) == L.LCP_E_INVAL


def test_python_forms_check_shapes_and_types():
    """Wrong dtypes, shapes and layouts are errors in Python, not reads of something else."""
    import learnable_channel_permutation_amd as lcp
    OTHER = "^(?!tensors must be on the GPU)"        # the device is looked at last
    bf = torch.bfloat16
    x, t = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(9, 32, 2)
    pos = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(pos=pos.long()), dict(pos=pos[:2]), dict(table=t.double()), dict(table=t[:, ::2]),
               dict(q=x.transpose(1, 2)), dict(q_out=x[:2]), dict(q_out=x.float()), dict(k=x),
               dict(k=x[:2], k_out=x[:2]), dict(k=x.float(), k_out=x.float())):
        a = {**dict(q=x, q_out=torch.empty_like(x), table=t, pos=pos), **kw}
        with pytest.raises(ValueError, match=OTHER):
            lcp.lcp_rope(**a)
    with pytest.raises(TypeError):
        h = x.half()
        lcp.lcp_rope(h, torch.empty_like(h), t, pos)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(4, 2, 16)
    with pytest.raises(TypeError):
        lcp.PagedKVCache(k.half(), k.half())
    for a in ((k, k, None, s), (k, k, s, s.double()), (k, k[:2], s, s), (k.transpose(1, 2), k.transpose(1, 2), s, s)):
        with pytest.raises(ValueError, match=OTHER):
            lcp.PagedKVCache(*a)
    c = lcp.PagedKVCache(k, k.clone(), s, s.clone())
    with pytest.raises(ValueError, match=OTHER):
        c.append(x, x[:2], pos)
    with pytest.raises(ValueError, match=OTHER):
        c.append(x, x, pos.long())
    with pytest.raises(ValueError, match=OTHER):
        c.append(x, x, pos, q=x)
    with pytest.raises(ValueError, match=OTHER):
        c.read(pos, torch.empty(3, 2, 65), torch.empty(3, 2, 65))
    pt, ln = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for a, kw in (((x.float(), pt, ln), {}), ((x, pt[:2], ln), {}), ((x, pt, ln.long()), {}),
                  ((x, pt, ln), dict(out=torch.empty(3, 2, 32))), ((x, pt, ln), dict(lse=torch.empty(3, 2).double())),
                  ((torch.zeros(3, 64, 2, dtype=bf).transpose(1, 2), pt, ln), {})):
        with pytest.raises(ValueError, match=OTHER):
            c.attend(*a, **kw)
    with pytest.raises(lcp.LcpError):       # heads of q not a multiple of the cache's
        c.attend(torch.zeros(3, 3, 64, dtype=bf), pt, ln)
    for call in (lambda: lcp.lcp_rope(x, torch.empty_like(x), t, pos), lambda: c.append(x, x, pos),
                 lambda: c.read(pos), lambda: c.attend(x, pt, ln)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match=OTHER):
        lcp.lcp_rope(x, None, t, pos)


def test_workspace_of_the_largest_call_serves_the_smaller():
    """The query grows with the batch and the length, whatever way of working the sizes lead to."""
    L = _lib()
    for D in (64, 128, 256):
        k, s = torch.empty(4, 2, 16, D, dtype=torch.int8), torch.empty(4, 2, 16)
        c = L.make_kv_cache(k, k.clone(), s, s.clone())
        for G in (1, 16, 17, 31, 32, 40):
            sizes = [[L.lcp_attn_decode_workspace_bytes(c, B, 2 * G, n) for n in (1, 700, 3000, 20000, 200000)]
                     for B in (1, 5, 40, 300)]
            for row, below in zip(sizes, sizes[1:] + [sizes[-1]]):
                assert row == sorted(row)
                assert all(x <= y for x, y in zip(row, below))


def test_sizes_past_a_grid_are_refused():
    """More threads than a grid counts: refused before the launch, in either form of the kernels."""
    L = _lib()
    big = _rows(L, heads=65536, xt=0, xh=0, yt=65536 * 128, yh=128)
    odd = _rows(L, heads=65536, x=P + 2, xt=0, xh=0, yt=65536 * 128, yh=128)
    for q, T in ((big, 1 << 14), (odd, 1 << 11)):
        assert L.LIB.lcp_rope(ctypes.byref(q), None, L.LCP_BF16, T, 128, P, 10, P, 128, 0, 0, None) == L.LCP_E_INVAL
        k = _rows(L, xt=0, xh=0)
        assert L.LIB.lcp_kv_append(ctypes.byref(_cache(L)), ctypes.byref(q), ctypes.byref(k), ctypes.byref(k), T, P, P,
                                   10, P, 128, 0, None) == L.LCP_E_INVAL
    n = ctypes.c_size_t(0)
    c = ctypes.byref(_cache(L, D=64, heads=1))
    assert L.LIB.lcp_attn_decode_workspace_bytes(c, 1 << 24, 1, 16, 0, ctypes.byref(n)) == L.LCP_E_INVAL


def test_cache_on_two_devices_is_refused():
    L = _lib()
    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16)
    m = [torch.empty_like(k, device="meta"), torch.empty_like(s, device="meta")]
    for a in ((k, m[0], s, s), (k, k.clone(), s, m[1])):
        with pytest.raises(ValueError, match="one device"):
            L.make_kv_cache(*a)
    assert L.make_kv_cache(k, k.clone(), s, s.clone()).gpu == -1


def test_table_on_the_cpu_is_refused():
    L = _lib()
    with pytest.raises(ValueError, match="on the GPU"):
        L.lcp_rope_table(L.make_rope_cfg(64), torch.zeros(9, 32, 2))


def test_cache_and_its_addresses_stay_together():
    """No call may use the address of a tensor that was replaced or freed."""
    import gc
    import weakref
    import learnable_channel_permutation_amd as lcp
    L = _lib()

    def tensors(pages):
        k, s = torch.zeros(pages, 2, 16, 64, dtype=torch.int8), torch.zeros(pages, 2, 16)
        return k, k.clone(), s, s.clone()

    c = lcp.PagedKVCache(*tensors(4))
    for name, t in zip(("k", "v", "k_scale", "v_scale"), tensors(9)):
        with pytest.raises(AttributeError):
            setattr(c, name, t)
        assert getattr(c.c, name) == getattr(c, name).data_ptr()
    with pytest.raises(AttributeError):
        c.c = L.make_kv_cache(*tensors(9))
    all4 = tensors(4)
    alive = [weakref.ref(t) for t in all4]
    s = L.make_kv_cache(*all4)
    del all4
    gc.collect()
    assert all(r() is not None and r().data_ptr() == getattr(s, n)
               for r, n in zip(alive, ("k", "v", "k_scale", "v_scale")))


def test_strides_whose_span_passes_64_bits_are_refused():
    """Sums of offsets that wrap would pass for rows that keep apart: token 2 and head 1 meet here."""
    L = _lib()
    T = (1 << 25) + 1
    for kw in (dict(yt=1 << 39, yh=1 << 40), dict(xt=1 << 39)):
        q = ctypes.byref(_rows(L, **kw))
        assert L.LIB.lcp_rope(q, None, L.LCP_BF16, T, 128, P, 10, P, 128, 0, 0, None) == L.LCP_E_INVAL
        k = ctypes.byref(_rows(L, xt=1 << 39))
        good = ctypes.byref(_rows(L))
        for a in ((q, good, good), (None, k, good), (None, good, k)):
            assert L.LIB.lcp_kv_append(ctypes.byref(_cache(L, heads=4)), *a, T >> 1, P, P, 10, P, 128, 0,
                                       None) == L.LCP_E_INVAL


def test_a_flag_without_a_truth_value_is_its_own_error():
    """As any Python call reports it; not a result with an error left behind."""
    import learnable_channel_permutation_amd as lcp
    x, t = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(9, 32, 2)
    pos, both = torch.zeros(3, dtype=torch.int32), torch.ones(2)
    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16)
    c = lcp.PagedKVCache(k, k.clone(), s, s.clone())
    for call in (lambda: lcp.lcp_rope(x, torch.empty_like(x), t, pos, interleaved=both),
                 lambda: lcp.lcp_rope(x, torch.empty_like(x), t, pos, inverse=both),
                 lambda: c.append(x, x, pos, table=t, pos=pos, interleaved=both)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()


def test_every_public_name_exists():
    import learnable_channel_permutation_amd as lcp
    names = {}
    exec("from learnable_channel_permutation_amd import *", names)
    assert set(lcp.__all__) <= set(names)
    # the two that have no Python form of their own: messages come with LcpError, the version is the library's
    assert set(_lib().EXPORTS) - set(lcp.__all__) == {"lcp_status_string", "lcp_version"}


def test_read_without_outputs_is_refused():
    """They would be made, on the current stream whatever the call's is, and lost."""
    import learnable_channel_permutation_amd as lcp
    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16)
    c, slots = lcp.PagedKVCache(k, k.clone(), s, s.clone()).c, torch.zeros(3, dtype=torch.int32)
    out = torch.zeros(3, 2, 64)
    for a in ((None, None), (out, None), (None, out)):
        with pytest.raises(ValueError, match="k_out and v_out must be tensors"):
            lcp.lcp_kv_read(c, slots, *a)
