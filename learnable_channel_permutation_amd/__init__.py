"""MI355X (gfx950) learnable channel permutation (LCP) step.

The computation lives in liblcp.so (HIP kernels behind the C ABI of
include/lcp.h); this package only binds it (``_lib``) and wraps the
per-layer buffers in a small session object. Importing fails if the library
has not been built.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import (LCP_BF16, LCP_F32, LcpError, lcp_colnorm, lcp_error,  # noqa: F401
                   lcp_error_workspace_bytes, lcp_harden, lcp_layer_init, lcp_nm_mask, lcp_permute,
                   lcp_sinkhorn, lcp_sinkhorn_bwd, lcp_step_bwd, lcp_step_fwd,
                   lcp_step_workspace_bytes, lcp_xt_pitch, make_cfg, make_layer, make_timing,
                   lcp_adamw, lcp_step_bwd_adamw, lcp_train, make_adamw_cfg, lcp_layer_outputs,
                   lcp_attn_decode, lcp_attn_decode_workspace_bytes, lcp_kv_append, lcp_kv_read, lcp_rope,
                   lcp_rope_table, make_kv_cache, make_rope_cfg, lcp_deploy_forward, lcp_gather_channels,
                   lcp_layer_outputs_noalloc, lcp_sparse_gemm, lcp_sparse_pack, lcp_sparse_pack_bytes,
                   lcp_rms_norm, lcp_rms_norm_bwd, lcp_rms_norm_bwd_workspace_bytes, lcp_sparse_linear,
                   lcp_sparse_linear_cut, lcp_sparse_linear_workspace_bytes, lcp_sparse_pack_e4m3,
                   lcp_sparse_pack_e4m3_bytes, make_packed)

__all__ = ["LayerSession", "LcpError", "PagedKVCache", "RMSNorm", "SparseLinear"] + [n for n in _lib.EXPORTS if n in globals()]


class LayerSession:
    """Device buffers for repeated LCP steps on one layer.

    Holds W and X (caller tensors on one GPU), the per-layer setup written by
    lcp_layer_init (column norms; X transposed for bf16 layers) and one step
    workspace sized by lcp_step_workspace_bytes. harden=True runs the
    hardened forward with the straight-through backward; loss="cosine"
    optimises the cosine objective (the dense outputs Y = W X^T and ||Y||^2
    are then computed once here by lcp_layer_outputs); mask_ste=True adds the
    straight-through gradient of the mask.
    """

    def __init__(self, W, X, B, iters, tau, N, M, stream=None, harden=False, loss="frobenius",
                 mask_ste=False):
        if W.device != X.device or W.dtype != X.dtype:
            raise ValueError("W and X must share device and dtype")
        self.W, self.X = W, X
        self.B, self.iters, self.tau, self.N, self.M = B, iters, tau, N, M
        cout, cin = W.shape
        T = X.shape[0]
        dev = W.device
        self.norms = torch.empty(cin, dtype=torch.float32, device=dev)
        self.Xt = None
        if W.dtype == torch.bfloat16:
            self.Xt = torch.empty((cin, lcp_xt_pitch(T)), dtype=torch.bfloat16, device=dev)
        nbytes = lcp_step_workspace_bytes(cout, cin, T, B, iters, _lib.dtype_code(W))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.err = torch.empty(1, dtype=torch.float32, device=dev)
        self.Y = self.y2 = None
        if loss == "cosine":
            self.Y = torch.empty((cout, lcp_xt_pitch(T)), dtype=W.dtype, device=dev)
            self.y2 = torch.empty(1, dtype=torch.float32, device=dev)
        self.layer = make_layer(W, X, self.norms, B, self.Xt, self.Y, self.y2)
        self.cfg = make_cfg(iters, tau, N, M, harden, loss, mask_ste)
        self.init(stream)

    def init(self, stream=None):
        """Per-layer setup (column norms, transposed X; dense outputs and
        their squared norm for the cosine objective)."""
        lcp_layer_init(self.X, self.norms, self.Xt, stream=stream)
        if self.Y is not None:
            cout, cin = self.W.shape
            ebytes = lcp_error_workspace_bytes(cout, cin, self.X.shape[0], _lib.dtype_code(self.W))
            if ebytes > self.ws.numel():
                raise RuntimeError("step workspace smaller than the layer-output workspace")
            lcp_layer_outputs(self.W, self.X, self.Y, self.y2, self.ws, stream=stream)

    def forward(self, logits, P_out=None, bits_out=None, timing=None, stream=None):
        lcp_step_fwd(self.layer, logits, self.cfg, self.ws, self.err, P_out, bits_out, timing, stream)
        return self.err

    def backward(self, logits, dlogits=None, timing=None, stream=None):
        if dlogits is None:
            dlogits = torch.empty_like(logits)
        lcp_step_bwd(self.layer, logits, self.cfg, self.ws, dlogits, timing, stream)
        return dlogits

    def capture_step(self, logits, dlogits, setup=True):
        """Capture one step on fixed buffers into a HIP graph
        (torch.cuda.CUDAGraph): the per-layer setup (when `setup`), the
        forward (E into self.err) and the backward (into `dlogits`). The
        library allocates nothing, synchronises nothing and issues no memset
        inside a step, so the captured kernels are exactly the eager ones;
        graph.replay() reruns them on the current contents of the buffers."""
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):           # one eager run before capture
            if setup:
                self.init()
            self.forward(logits)
            self.backward(logits, dlogits)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(g):
            if setup:
                self.init()
            self.forward(logits)
            self.backward(logits, dlogits)
        return g

    def train(self, logits, steps, lr, tau0=1.0, tau1=0.1, beta1=0.9, beta2=0.999, eps=1e-8,
              weight_decay=0.01, stream=None):
        """`steps` AdamW steps on `logits` (updated in place) with the
        temperature annealed linearly from tau0 to tau1 (lcp_train). Returns
        the per-step objective values as a device tensor."""
        m = torch.zeros_like(logits)
        v = torch.zeros_like(logits)
        errs = torch.empty(steps, dtype=torch.float32, device=logits.device)
        acfg = make_adamw_cfg(lr, beta1, beta2, eps, weight_decay)
        lcp_train(self.layer, logits, self.cfg, self.ws, m, v, steps, tau0, tau1, acfg, errs, stream)
        return errs


def _made_on(stream, given, call, *args):
    """call(*args, None) with `stream` as the current one, so that what it allocates belongs to that stream: a block
    of the caller's stream may still be in use by work queued there, which `stream` does not wait for. The tensors
    that it makes (results not among `given`) are kept from reuse until the caller's stream is done with them, too."""
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        results = call(*args, None)
    for t in results[1:]:
        if t is not None and not any(t is g for g in given):
            t.record_stream(caller)
    return results


class PagedKVCache:
    """A paged key/value cache on one GPU and the attention that reads it.

    k, v: pages [pages, heads, page_size, D] in bfloat16, float8_e4m3fn or
    int8 (the 8-bit formats with fp32 scales [pages, heads, page_size]); D 64,
    128 or 256, page_size a multiple of 16. Which pages belong to which
    sequence is the caller's: slots (page * page_size + offset) say where new
    tokens go, a page table [B, max_pages] and the lengths what a step reads.
    The tensors are the cache's for its life: k, v, k_scale and v_scale are read-only.
    Calls run on the current stream, or on a given one: inputs have to be ready there, and
    results are, in its order.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._c = make_kv_cache(k, v, k_scale, v_scale)

    # The tensors and the struct of their addresses are one: another tensor needs another cache.
    c = property(lambda self: self._c)
    k = property(lambda self: self._c.tensors[0])
    v = property(lambda self: self._c.tensors[1])
    k_scale = property(lambda self: self._c.tensors[2])
    v_scale = property(lambda self: self._c.tensors[3])

    @classmethod
    def empty(cls, pages, page_size, heads, D, dtype=torch.float8_e4m3fn, device="cuda"):
        """A cache with room for pages * page_size tokens (its contents are undefined until written)."""
        k, v = (torch.empty((pages, heads, page_size, D), dtype=dtype, device=device) for _ in range(2))
        ks = vs = None
        if dtype != torch.bfloat16:
            ks, vs = (torch.empty((pages, heads, page_size), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def append(self, k, v, slots, q=None, q_out=None, table=None, pos=None, interleaved=False, stream=None):
        """Write new tokens' k and v [T, heads, D] (k rotated by the table at pos first) and rotate q [T, hq, D]
        into q_out (lcp_kv_append)."""
        lcp_kv_append(self._c, k, v, slots, q, q_out, table, pos, interleaved, stream)
        return q_out

    def read(self, slots, k_out=None, v_out=None, stream=None):
        """The stored k and v of slots, [T, heads, D] bfloat16 unless outputs are given (lcp_kv_read)."""
        if stream is None or (k_out is not None and v_out is not None):
            code, k_out, v_out = _lib._serve.read(self._c, slots, k_out, v_out, stream)
        else:
            code, k_out, v_out = _made_on(stream, (k_out, v_out), _lib._serve.read, self._c, slots, k_out, v_out)
        _lib._check("lcp_kv_read", code)
        return k_out, v_out

    def attend(self, q, pages, lens, max_len=None, scale=None, window=0, out=None, lse=None, ws=None, stream=None):
        """Attention of one new token of each sequence, q [B, hq, D] bfloat16 (lcp_attn_decode): (out, lse). max_len,
        the host's bound on lens, defaults to what the page table can hold; scale to D^-1/2."""
        args = (self._c, q, pages, lens, max_len, out, lse, ws, scale, window, True)
        made = stream is not None and (out is None or lse is None)
        if stream is not None and not made and ws is None:
            n = pages.shape[1] * self._c.page_size if max_len is None else max_len
            made = lcp_attn_decode_workspace_bytes(self._c, q.shape[0], q.shape[1], n, window) > 0
        if made:
            code, out, lse = _made_on(stream, (out, lse), _lib._serve.attend, *args)
        else:
            code, out, lse = _lib._serve.attend(*args, stream)
        _lib._check("lcp_attn_decode", code)
        return out, lse


class RMSNorm:
    """The root-mean-square norm in front of a deployed layer (lcp_rms_norm).

    weight [C] float32 or bfloat16. perm [C / B, B] int32 (lcp_harden's): the output is in that layer's channel
    order. dtype: the output's, float32, bfloat16 or float8_e4m3fn (with a scale for each token), None for x's.
    Calls are no part of autograd's graph (they warn where an input asks for a gradient): backward() computes it.
    """

    def __init__(self, weight, eps=1e-6, perm=None, dtype=None):
        self.weight, self.eps, self.perm = weight, float(eps), perm
        self._y = _type_code(dtype, (torch.float32, torch.bfloat16, torch.float8_e4m3fn))

    def __call__(self, x, residual=None, out=None, scale=None, sum_out=None, stream=None):
        """(y, scale, sum) for x [T, C]: scale of an 8-bit y, else None; sum = x + residual where there is one."""
        args = (x, self.weight, residual, self.perm, out, scale, sum_out, self._y, self.eps, True)
        if stream is not None and (out is None or (scale is None and out.dtype == torch.float8_e4m3fn) or
                                   (sum_out is None and residual is not None)):
            code, out, scale, sum_out = _made_on(stream, (out, scale, sum_out), _lib._serve.rms_norm, *args)
        else:
            code, out, scale, sum_out = _lib._serve.rms_norm(*args, stream)
        _lib._check("lcp_rms_norm", code)
        return out, scale, sum_out

    def backward(self, h, dy, dsum=None, dx=None, dweight=None, ws=None, stream=None):
        """(dx, dweight) from the sum (or the x) that was normalised, dL/dy and, with a residual stream, the gradient
        dsum that arrives at the sum (lcp_rms_norm_bwd). In natural channel order: not with perm."""
        if self.perm is not None:
            raise ValueError("the gradient is in natural channel order: use an RMSNorm without perm")
        args = (h, self.weight, dy, dsum, dx, dweight, ws, self.eps, True)
        if stream is not None and (dx is None or dweight is None or ws is None):
            code, dx, dweight = _made_on(stream, (dx, dweight), _lib._serve.rms_norm_bwd, *args)
        else:
            code, dx, dweight = _lib._serve.rms_norm_bwd(*args, stream)
        _lib._check("lcp_rms_norm_bwd", code)
        return dx, dweight


class SparseLinear:
    """A deployed 2:4 layer with an epilogue (lcp_sparse_linear), for one token or many.

    vals, meta: the outputs of lcp_sparse_pack, or with scale [cout] those of lcp_sparse_pack_e4m3; pack() makes
    them. Inputs are in the layer's permuted channel order (RMSNorm with perm, lcp_gather_channels, or a layer whose
    rows were packed in that order). The tensors are the layer's for its life.
    Products are exact and sums float32. fast=True, for 8-bit layers, lets bfloat16 outputs of more than 64 tokens come
    from the e4m3 matrix instructions, up to a third faster; a sum far smaller than its terms may then be all error.
    """

    def __init__(self, vals, meta, cout, cin, scale=None, fast=False):
        self._p = make_packed(vals, meta, cout, cin, scale, fast)

    p = property(lambda self: self._p)
    cout = property(lambda self: self._p.cout)
    cin = property(lambda self: self._p.cin)
    vals = property(lambda self: self._p.tensors[0])
    meta = property(lambda self: self._p.tensors[1])
    scale = property(lambda self: self._p.tensors[2])
    fast = property(lambda self: bool(self._p.fast))

    @classmethod
    def pack(cls, W, perm, bits, dtype=torch.bfloat16, fast=False):
        """From W [cout, cin] bfloat16, the hard permutation [cin / B, B] and the 2:4 mask in permuted positions
        ([cout, cin / 32] int32), in bfloat16 or float8_e4m3fn."""
        if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("a deployed layer is bfloat16 or float8_e4m3fn")
        (cout, cin), (nb, B) = W.shape, perm.shape
        if W.dtype != torch.bfloat16 or not W.is_contiguous() or not W.is_cuda:
            raise ValueError("W must be contiguous bfloat16 [cout, cin] on the GPU")
        if nb * B != cin or perm.dtype != torch.int32 or not perm.is_contiguous() or perm.device != W.device:
            raise ValueError("perm must be contiguous int32 [cin / B, B] on W's GPU")
        if tuple(bits.shape) != (cout, cin // 32) or bits.dtype != torch.int32 or not bits.is_contiguous() or \
                bits.device != W.device:
            raise ValueError("bits must be contiguous int32 [cout, cin / 32] on W's GPU")
        if W.get_device() != torch.cuda.current_device():
            raise ValueError("tensors must be on the current GPU")
        fp8 = dtype == torch.float8_e4m3fn
        if fast and not fp8:
            raise ValueError("fast belongs to 8-bit layers")
        vb, mb = (lcp_sparse_pack_e4m3_bytes if fp8 else lcp_sparse_pack_bytes)(cout, cin)
        vals = torch.empty(vb, dtype=torch.uint8, device=W.device)
        meta = torch.empty(mb // 4, dtype=torch.int32, device=W.device)
        scale = None
        if fp8:
            scale = torch.empty(cout, dtype=torch.float32, device=W.device)
            lcp_sparse_pack_e4m3(W, B, perm, bits, vals, meta, scale)
        else:
            lcp_sparse_pack(W, B, perm, bits, vals, meta)
        return cls(vals, meta, cout, cin, scale, fast)

    def __call__(self, x, scale=None, bias=None, act=None, gate=None, residual=None, out=None, dtype=None, ws=None,
                 stream=None):
        """act(x Ws^T + bias) * gate + residual for x [T, cin] (with scale [T] where the layer is float8_e4m3fn):
        [T, cout] bfloat16, or dtype. act: None, "relu", "silu", "gelu" or "gelu_tanh"."""
        args = (self._p, x, scale, bias, gate, residual, out, ws, _lib.act_code(act),
                _type_code(dtype, (torch.float32, torch.bfloat16)), True)
        if stream is not None and (out is None or
                                   (ws is None and lcp_sparse_linear_workspace_bytes(self._p, x.shape[0]) > 0)):
            code, out = _made_on(stream, (out,), _lib._serve.linear, *args)
        else:
            code, out = _lib._serve.linear(*args, stream)
        _lib._check("lcp_sparse_linear", code)
        return out


def _type_code(dtype, among):
    """The lcp_dtype of a torch dtype, -1 for None."""
    if dtype is None:
        return -1
    if dtype not in among:
        raise TypeError("unsupported dtype %s" % dtype)
    return {torch.float32: LCP_F32, torch.bfloat16: LCP_BF16, torch.float8_e4m3fn: _lib.LCP_E4M3}[dtype]
