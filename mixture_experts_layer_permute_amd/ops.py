"""Thin torch-tensor wrappers over the C entry points (marshalling only).

Shapes and meanings are those of include/moe.h.  Outputs not passed in are
allocated with torch on the inputs' device; workspaces likewise.  All calls
are asynchronous on torch's current HIP stream.
"""
import ctypes

import torch

from ._lib import (MOE_ACT_GELU, MOE_ACT_SWIGLU, MOE_BF16, MOE_F32, MoEError,
                   check, load)

_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _dt(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise MoEError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _need_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise MoEError("libmoe takes device tensors only")
        if t is not None and not t.is_contiguous():
            raise MoEError("libmoe takes contiguous tensors only")


def _act(act):
    if act in (MOE_ACT_GELU, "gelu"):
        return MOE_ACT_GELU
    if act in (MOE_ACT_SWIGLU, "swiglu"):
        return MOE_ACT_SWIGLU
    raise MoEError("unknown activation %r" % (act,))


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def moe_init(device=0):
    check(load().moe_init(int(device)), "moe_init")


def moe_set_overlap(enable=True):
    """Let the FFN backward run independent launches on a side stream (default)."""
    check(load().moe_set_overlap(1 if enable else 0), "moe_set_overlap")


def moe_gate_topk(x, Wg, k, logit_bias=None, renorm=1, logits=None,
                  topk_idx=None, topk_w=None):
    """-> (logits [T,E] f32, topk_idx [T,k] i32, topk_w [T,k] f32)."""
    _need_gpu(x, Wg, logit_bias)
    T, d = x.shape
    E = Wg.shape[1]
    dev = x.device
    if logits is None:
        logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    if topk_idx is None:
        topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=torch.float32, device=dev)
    check(load().moe_gate_topk(_p(x), _p(Wg), _p(logit_bias), T, d, E, k, renorm,
                               _dt(x), _p(logits), _p(topk_idx), _p(topk_w),
                               _stream(dev)), "moe_gate_topk")
    return logits, topk_idx, topk_w


def moe_permute(topk_idx, x, E, out=None, ws=None, copy=True):
    """-> (counts [E], offsets [E+1], dest [T,k], src [T*k], x_perm [T*k,d]);
    copy=False: routing only, x_perm is None (for the *_gather FFN calls)."""
    _need_gpu(topk_idx, x)
    T, k = topk_idx.shape
    d = x.shape[1]
    dev = x.device
    L = load()
    if out is None:
        out = (torch.empty(E, dtype=torch.int32, device=dev),
               torch.empty(E + 1, dtype=torch.int32, device=dev),
               torch.empty(T, k, dtype=torch.int32, device=dev),
               torch.empty(T * k, dtype=torch.int32, device=dev),
               torch.empty(T * k, d, dtype=x.dtype, device=dev) if copy else None)
    counts, offsets, dest, src, x_perm = out
    nb = L.moe_permute_workspace_bytes(T, E, k)
    if ws is None:
        ws = _ws(nb, dev)
    check(L.moe_permute(_p(topk_idx), _p(x), T, d, E, k, _dt(x), _p(counts),
                        _p(offsets), _p(dest), _p(src), _p(x_perm), _p(ws),
                        ws.numel(), _stream(dev)), "moe_permute")
    return counts, offsets, dest, src, x_perm


def moe_expert_ffn_fwd(x_perm, offsets, W1, W2, W3=None, act="gelu", out=None,
                       ws=None):
    """-> (h_save, a_save [R,f], out_perm [R,d]); h_save is the state the
    backward needs: GeLU'(H) [R,f], or [H3 SiLU'(H1) | SiLU(H1)] [R,2f]."""
    _need_gpu(x_perm, offsets, W1, W2, W3)
    a = _act(act)
    R, d = x_perm.shape
    E, _, f = W1.shape
    dev = x_perm.device
    L = load()
    if out is None:
        hw = 2 * f if a == MOE_ACT_SWIGLU else f
        out = (torch.empty(R, hw, dtype=x_perm.dtype, device=dev),
               torch.empty(R, f, dtype=x_perm.dtype, device=dev),
               torch.empty(R, d, dtype=x_perm.dtype, device=dev))
    h_save, a_save, out_perm = out
    if ws is None:
        ws = _ws(L.moe_ffn_workspace_bytes(R, E, d, f, a, _dt(x_perm), 0), dev)
    check(L.moe_expert_ffn_fwd(_p(x_perm), _p(offsets), R, E, d, f, a,
                               _dt(x_perm), _p(W1), _p(W3), _p(W2), _p(h_save),
                               _p(a_save), _p(out_perm), _p(ws), ws.numel(),
                               _stream(dev)), "moe_expert_ffn_fwd")
    return h_save, a_save, out_perm


def moe_expert_ffn_fwd_noalloc(x_perm, offsets, W1, W2, W3=None, act="gelu", out=None):
    """moe_expert_ffn_fwd with the library's static scratch instead of a
    workspace.  -> (h_save, a_save [R,f], out_perm [R,d]); pass ``out`` to
    allocate nothing at all."""
    _need_gpu(x_perm, offsets, W1, W2, W3)
    a = _act(act)
    R, d = x_perm.shape
    E, _, f = W1.shape
    dev = x_perm.device
    if out is None:
        hw = 2 * f if a == MOE_ACT_SWIGLU else f
        out = (torch.empty(R, hw, dtype=x_perm.dtype, device=dev),
               torch.empty(R, f, dtype=x_perm.dtype, device=dev),
               torch.empty(R, d, dtype=x_perm.dtype, device=dev))
    h_save, a_save, out_perm = out
    check(load().moe_expert_ffn_fwd_noalloc(_p(x_perm), _p(offsets), R, E, d, f, a,
                                            _dt(x_perm), _p(W1), _p(W3), _p(W2),
                                            _p(h_save), _p(a_save), _p(out_perm),
                                            _stream(dev)), "moe_expert_ffn_fwd_noalloc")
    return h_save, a_save, out_perm


def moe_expert_ffn_bwd(d_out_perm, x_perm, h_save, a_save, offsets, W1, W2,
                       W3=None, act="gelu", out=None, ws=None):
    """-> (dx_perm [R,d], dW1 [E,d,f], dW3 or None, dW2 [E,f,d])."""
    _need_gpu(d_out_perm, x_perm, h_save, a_save, offsets, W1, W2, W3)
    a = _act(act)
    R, d = x_perm.shape
    E, _, f = W1.shape
    dev = x_perm.device
    L = load()
    if out is None:
        out = (torch.empty(R, d, dtype=x_perm.dtype, device=dev),
               torch.empty_like(W1),
               torch.empty_like(W3) if a == MOE_ACT_SWIGLU else None,
               torch.empty_like(W2))
    dx_perm, dW1, dW3, dW2 = out
    if ws is None:
        ws = _ws(L.moe_ffn_workspace_bytes(R, E, d, f, a, _dt(x_perm), 1), dev)
    check(L.moe_expert_ffn_bwd(_p(d_out_perm), _p(x_perm), _p(h_save),
                               _p(a_save), _p(offsets), R, E, d, f, a,
                               _dt(x_perm), _p(W1), _p(W3), _p(W2), _p(dx_perm),
                               _p(dW1), _p(dW3), _p(dW2), _p(ws), ws.numel(),
                               _stream(dev)), "moe_expert_ffn_bwd")
    return dx_perm, dW1, dW3, dW2


def moe_expert_ffn_fwd_gather(x, src, offsets, W1, W2, W3=None, act="gelu",
                              out=None, ws=None):
    """moe_expert_ffn_fwd reading permuted row r as x[src[r]] (no x_perm).
    -> (h_save, a_save [R,f], out_perm [R,d]), R = src.numel()."""
    _need_gpu(x, src, offsets, W1, W2, W3)
    a = _act(act)
    T, d = x.shape
    R = src.numel()
    E, _, f = W1.shape
    dev = x.device
    L = load()
    if out is None:
        hw = 2 * f if a == MOE_ACT_SWIGLU else f
        out = (torch.empty(R, hw, dtype=x.dtype, device=dev),
               torch.empty(R, f, dtype=x.dtype, device=dev),
               torch.empty(R, d, dtype=x.dtype, device=dev))
    h_save, a_save, out_perm = out
    if ws is None:
        ws = _ws(L.moe_ffn_workspace_bytes(R, E, d, f, a, _dt(x), 0), dev)
    check(L.moe_expert_ffn_fwd_gather(_p(x), _p(src), _p(offsets), T, R, E, d, f, a,
                                      _dt(x), _p(W1), _p(W3), _p(W2), _p(h_save),
                                      _p(a_save), _p(out_perm), _p(ws), ws.numel(),
                                      _stream(dev)), "moe_expert_ffn_fwd_gather")
    return h_save, a_save, out_perm


def moe_expert_ffn_bwd_gather(d_out_perm, x, src, h_save, a_save, offsets, W1, W2,
                              W3=None, act="gelu", out=None, ws=None):
    """moe_expert_ffn_bwd reading permuted row r as x[src[r]] (no x_perm).
    -> (dx_perm [R,d], dW1 [E,d,f], dW3 or None, dW2 [E,f,d])."""
    _need_gpu(d_out_perm, x, src, h_save, a_save, offsets, W1, W2, W3)
    a = _act(act)
    T, d = x.shape
    R = src.numel()
    E, _, f = W1.shape
    dev = x.device
    L = load()
    if out is None:
        out = (torch.empty(R, d, dtype=x.dtype, device=dev),
               torch.empty_like(W1),
               torch.empty_like(W3) if a == MOE_ACT_SWIGLU else None,
               torch.empty_like(W2))
    dx_perm, dW1, dW3, dW2 = out
    if ws is None:
        ws = _ws(L.moe_ffn_workspace_bytes(R, E, d, f, a, _dt(x), 1), dev)
    check(L.moe_expert_ffn_bwd_gather(_p(d_out_perm), _p(x), _p(src), _p(h_save),
                                      _p(a_save), _p(offsets), T, R, E, d, f, a, _dt(x),
                                      _p(W1), _p(W3), _p(W2), _p(dx_perm), _p(dW1),
                                      _p(dW3), _p(dW2), _p(ws), ws.numel(),
                                      _stream(dev)), "moe_expert_ffn_bwd_gather")
    return dx_perm, dW1, dW3, dW2


def moe_combine(out_perm, dest, topk_w, y=None):
    """-> y [T,d]."""
    _need_gpu(out_perm, dest, topk_w)
    T, k = dest.shape
    d = out_perm.shape[1]
    if y is None:
        y = torch.empty(T, d, dtype=out_perm.dtype, device=out_perm.device)
    check(load().moe_combine(_p(out_perm), _p(dest), _p(topk_w), T, k, d,
                             _dt(out_perm), _p(y), _stream(out_perm.device)),
          "moe_combine")
    return y


def moe_combine_bwd(dy, out_perm, dest, topk_w, out=None):
    """-> (d_out_perm [T*k,d], d_topk_w [T,k] f32)."""
    _need_gpu(dy, out_perm, dest, topk_w)
    T, k = dest.shape
    d = dy.shape[1]
    dev = dy.device
    if out is None:
        out = (torch.empty(T * k, d, dtype=dy.dtype, device=dev),
               torch.empty(T, k, dtype=torch.float32, device=dev))
    d_out, dw = out
    check(load().moe_combine_bwd(_p(dy), _p(out_perm), _p(dest), _p(topk_w), T, k,
                                 d, _dt(dy), _p(d_out), _p(dw), _stream(dev)),
          "moe_combine_bwd")
    return d_out, dw


def moe_unpermute_grad(dx_perm, dest, dx=None, accumulate=0):
    """-> dx [T,d] (overwritten, or accumulated into when accumulate=1)."""
    _need_gpu(dx_perm, dest)
    T, k = dest.shape
    d = dx_perm.shape[1]
    if dx is None:
        dx = torch.empty(T, d, dtype=dx_perm.dtype, device=dx_perm.device)
    check(load().moe_unpermute_grad(_p(dx_perm), _p(dest), T, k, d, _dt(dx_perm),
                                    _p(dx), int(accumulate),
                                    _stream(dx_perm.device)), "moe_unpermute_grad")
    return dx


def moe_gate_topk_bwd(x, Wg, logits, topk_idx, topk_w, d_topk_w, dx, renorm=1,
                      dWg=None, ws=None, accumulate=True):
    """dx += dl Wg^T in place (dx = dl Wg^T with accumulate=False); -> dWg [d,E]."""
    _need_gpu(x, Wg, logits, topk_idx, topk_w, d_topk_w, dx)
    T, d = x.shape
    E = Wg.shape[1]
    k = topk_idx.shape[1]
    dev = x.device
    L = load()
    if dWg is None:
        dWg = torch.empty_like(Wg)
    if ws is None:
        ws = _ws(L.moe_gate_bwd_workspace_bytes(T, d, E), dev)
    check(L.moe_gate_topk_bwd(_p(x), _p(Wg), _p(logits), _p(topk_idx), _p(topk_w),
                              _p(d_topk_w), T, d, E, k, renorm, _dt(x), _p(dx),
                              int(bool(accumulate)), _p(dWg), _p(ws), ws.numel(),
                              _stream(dev)),
          "moe_gate_topk_bwd")
    return dWg


def _few_check(x, Wg, W1, W2, W3, logit_bias, a):
    """Shapes, types and devices of a few-token call -> (T, d, f, E)."""
    ts = [x, Wg, W1, W2] + ([] if W3 is None else [W3])
    _need_gpu(*ts, logit_bias)
    if x.dim() != 2 or Wg.dim() != 2 or W1.dim() != 3 or W2.dim() != 3:
        raise MoEError("x [T,d], Wg [d,E], W1 [E,d,f], W2 [E,f,d] expected")
    T, d = x.shape
    E, f = Wg.shape[1], W1.shape[2]
    if (Wg.shape[0] != d or tuple(W1.shape) != (E, d, f) or tuple(W2.shape) != (E, f, d)
            or (W3 is not None and tuple(W3.shape) != (E, d, f))):
        raise MoEError("x [T,d], Wg [d,E], W1 and W3 [E,d,f], W2 [E,f,d] do not agree")
    if (W3 is not None) != (a == MOE_ACT_SWIGLU):
        raise MoEError("W3 goes with the swiglu activation, and only with it")
    if any(t.dtype != x.dtype or t.device != x.device for t in ts):
        raise MoEError("x, Wg and the weights need one dtype and one device")
    if logit_bias is not None and (tuple(logit_bias.shape) != (E,)
                                   or logit_bias.dtype != torch.float32
                                   or logit_bias.device != x.device):
        raise MoEError("logit_bias: float32 [E] on the inputs' device")
    return T, d, f, E


def moe_layer_fwd_few(x, Wg, W1, W2, W3=None, k=1, act="gelu", logit_bias=None, renorm=1,
                      out=None, ws=None):
    """The whole layer for 1 to 64 tokens, forward only.
    -> (y [T,d], logits [T,E] f32, topk_idx [T,k] i32, topk_w [T,k] f32)."""
    a = _act(act)
    T, d, f, E = _few_check(x, Wg, W1, W2, W3, logit_bias, a)
    dev = x.device
    L = load()
    if out is None:
        out = (torch.empty(T, d, dtype=x.dtype, device=dev),
               torch.empty(T, E, dtype=torch.float32, device=dev),
               torch.empty(T, k, dtype=torch.int32, device=dev),
               torch.empty(T, k, dtype=torch.float32, device=dev))
    y, logits, topk_idx, topk_w = out
    for t, shape, dt in ((y, (T, d), x.dtype), (logits, (T, E), torch.float32),
                         (topk_idx, (T, k), torch.int32), (topk_w, (T, k), torch.float32)):
        if (tuple(t.shape) != shape or t.dtype != dt or t.device != dev
                or not t.is_contiguous()):
            raise MoEError("out: y [T,d], logits [T,E], topk_idx [T,k], topk_w [T,k]")
    if ws is None:
        ws = _ws(L.moe_layer_few_workspace_bytes(T, d, f, E, k, a, _dt(x)), dev)
    elif ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise MoEError("ws: contiguous uint8 on the inputs' device")
    with torch.cuda.device(dev):
        check(L.moe_layer_fwd_few(_p(x), _p(Wg), _p(logit_bias), _p(W1), _p(W3), _p(W2), T, d,
                                  f, E, k, renorm, a, _dt(x), _p(logits), _p(topk_idx),
                                  _p(topk_w), _p(y), _p(ws), ws.numel(), _stream(dev)),
              "moe_layer_fwd_few")
    return y, logits, topk_idx, topk_w


class GradClip:
    """The global norm of a list of gradients and clipping to a largest norm
    (moe_grad_norm, moe_clip_grads), the list's addresses and the workspace
    kept from step to step.

    grads: float32 or bfloat16 device tensors, contiguous, of one device (a
    list may mix the types; views of a flat buffer are fine).  out: where
    clip() writes, tensors like grads; None: in place.  norm() and clip()
    return the norm as a float32 tensor of one element, overwritten by the
    next call: two calls in flight at once need a GradClip each.
    The result and the workspace come from torch's current stream when the
    GradClip is made: make it outside the step (as the layers do), or on the
    stream it is then called on, and keep it until its work is done.  A tensor
    given other memory since (t.data = ...) needs a new one.
    """

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise MoEError("GradClip: as many outputs as gradients")
        _need_gpu(*self.grads, *self.out)
        dev = self.device = (self.grads[0].device if self.grads else
                             torch.device("cuda", torch.cuda.current_device()))
        for g, o in zip(self.grads, self.out):
            if g.device != dev or o.device != dev:
                raise MoEError("GradClip: all tensors on one device")
            if o.dtype != g.dtype or o.shape != g.shape:
                raise MoEError("GradClip: an output needs its gradient's shape and dtype")
        self._disjoint = False         # looked at by the first clip()
        n = self.n = len(self.grads)
        ptrs = ctypes.c_void_p * n
        self._in = ptrs(*[g.data_ptr() for g in self.grads])
        self._out = ptrs(*[o.data_ptr() for o in self.out])
        self._numel = (ctypes.c_size_t * n)(*[g.numel() for g in self.grads])
        self._dts = (ctypes.c_int32 * n)(*[_dt(g) for g in self.grads])
        L = self.lib = load()
        self.ws = _ws(L.moe_grad_norm_workspace_bytes(self._numel, self._dts, n), dev)
        self.result = torch.empty(1, dtype=torch.float32, device=dev)
        self._res, self._ws, self._ws_bytes = _p(self.result), _p(self.ws), self.ws.numel()

    def _no_overlap(self):
        """Refuse lists whose result would depend on which block comes first:
        two outputs, or an output and another gradient, that share memory."""
        span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
        used = []
        for g, o in zip(self.grads, self.out):
            if g.numel() == 0:
                continue
            used.append(span(o) + (1,))
            if o.data_ptr() != g.data_ptr():
                used.append(span(g) + (0,))
        used.sort()
        end = written = 0              # ends of all spans and of the outputs so far
        for a, b, w in used:
            if a < (end if w else written):
                raise MoEError("GradClip: tensors overlap")
            end = max(end, b)
            written = max(written, b) if w else written

    def _call(self, fn, name, args, stream):
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._call(fn, name, args, stream)
        s = _stream(self.device) if stream is None else stream
        check(fn(*args, self._res, self._ws, self._ws_bytes, s), name)
        return self.result

    def norm(self, stream=None):
        """-> the norm, [1] float32; changes no gradient."""
        return self._call(self.lib.moe_grad_norm, "moe_grad_norm",
                          (self._in, self._numel, self._dts, self.n), stream)

    def clip(self, max_norm, stream=None):
        """out = grads * min(1, max_norm / norm) -> the norm, [1] float32."""
        if not self._disjoint:
            self._no_overlap()
            self._disjoint = True
        return self._call(self.lib.moe_clip_grads, "moe_clip_grads",
                          (self._in, self._out, self._numel, self._dts, self.n,
                           ctypes.byref(ctypes.c_float(max_norm))), stream)


def moe_grad_norm(grads):
    """The L2 norm over all elements of a list of gradients -> [1] float32."""
    return GradClip(grads).norm()


def moe_clip_grads(grads, max_norm, out=None):
    """Scales a list of gradients to the norm max_norm if theirs is larger (in
    place, or into out) -> the norm before, [1] float32."""
    return GradClip(grads, out).clip(max_norm)


def _head_check(x, Wv, labels, weight, teacher, grad):
    """Shapes, types and devices of a head call -> (T, d, V, K, labels, idx, score,
    teacher's weight)."""
    idx, score, tweight = (tuple(teacher) + (None,))[:3] if teacher is not None else (None,) * 3
    _need_gpu(x, Wv, labels, weight, idx, score, tweight)
    if x.dim() != 2 or Wv.dim() != 2 or x.shape[1] != Wv.shape[1]:
        raise MoEError("x [T,d] and Wv [V,d] expected")
    _dt(x)
    T, d = x.shape
    if Wv.dtype != x.dtype:
        raise MoEError("x and Wv need one dtype")
    K = 0
    if teacher is not None:
        if idx is None or score is None or idx.dim() != 2 or idx.shape[1] < 1:
            raise MoEError("teacher: (indices [T,K], scores [T,K][, weight [T]])")
        K = idx.shape[1]
    elif labels is None:
        raise MoEError("labels or a teacher needed")
    if not grad and (weight is not None or tweight is not None):
        raise MoEError("weights go with the gradient")
    if weight is not None and labels is None:
        raise MoEError("weight goes with labels")
    for t, shape, dt, name in ((labels, (T,), torch.int32, "labels: int32 [T]"),
                               (weight, (T,), torch.float32, "weight: float32 [T]"),
                               (idx, (T, K), torch.int32, "teacher indices: int32 [T,K]"),
                               (score, (T, K), torch.float32, "teacher scores: float32 [T,K]"),
                               (tweight, (T,), torch.float32, "teacher weight: float32 [T]")):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dt):
            raise MoEError(name + " expected")
    if any(t is not None and t.device != x.device
           for t in (Wv, labels, weight, idx, score, tweight)):
        raise MoEError("all tensors of a head on one device")
    return T, d, Wv.shape[0], K, idx, score, tweight


def _head_out(t, shape, dt, dev, name):
    if t is None:
        return torch.empty(shape, dtype=dt, device=dev)
    if (tuple(t.shape) != tuple(shape) or t.dtype != dt or t.device != dev
            or not t.is_contiguous()):
        raise MoEError("out: %s %s, contiguous, %s, on the inputs' device"
                       % (name, list(shape), dt))
    return t


def _head(x, Wv, labels, weight, teacher, tau, grad, out, ws, limit):
    T, d, V, K, idx, score, tweight = _head_check(x, Wv, labels, weight, teacher, grad)
    dev, f32 = x.device, torch.float32
    out = dict(out or {})
    known = (["loss", "lse"] if labels is not None else []) + (["kd"] if K else []) + \
        (["dx", "dWv"] if grad else [])
    if set(out) - set(known):
        raise MoEError("out: %s expected" % ", ".join(known))
    res = {}
    for name in known:
        if name in ("dx", "dWv"):
            if name in out and out[name] is None:          # not wanted
                res[name] = None
                continue
            res[name] = _head_out(out.get(name), (x if name == "dx" else Wv).shape, x.dtype, dev,
                                  name)
        else:
            res[name] = _head_out(out.get(name), (T,), f32, dev, name)
    L = load()
    if ws is None:
        ws = _ws(L.moe_head_workspace_bytes(T, d, V, K, _dt(x), int(grad), limit), dev)
    elif ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise MoEError("ws: contiguous uint8 on the inputs' device")
    loss, lse = _p(res.get("loss")), _p(res.get("lse"))
    tail = (T, d, V, _dt(x))
    end = (_p(ws), ws.numel())
    t = ctypes.byref(ctypes.c_float(tau))
    with torch.cuda.device(dev):
        s = _stream(dev)
        if K and grad:
            check(L.moe_head_distill_grad(_p(x), _p(Wv), _p(idx), _p(score), _p(tweight), K, t,
                                          _p(labels), _p(weight), *tail, _p(res["kd"]), loss, lse,
                                          _p(res["dx"]), _p(res["dWv"]), *end, s),
                  "moe_head_distill_grad")
        elif K:
            check(L.moe_head_distill(_p(x), _p(Wv), _p(idx), _p(score), K, t, _p(labels), *tail,
                                     _p(res["kd"]), loss, lse, *end, s), "moe_head_distill")
        elif grad:
            check(L.moe_head_xent_grad(_p(x), _p(Wv), _p(labels), _p(weight), *tail, loss, lse,
                                       _p(res["dx"]), _p(res["dWv"]), *end, s),
                  "moe_head_xent_grad")
        else:
            check(L.moe_head_xent(_p(x), _p(Wv), _p(labels), *tail, loss, lse, *end, s),
                  "moe_head_xent")
    return res


def moe_head_xent(x, Wv, labels, out=None, ws=None, limit=0):
    """Cross entropy of the scores x Wv^T with a label a token (outside [0,V):
    none, loss and lse 0) -> {"loss" [T] f32, "lse" [T] f32}."""
    return _head(x, Wv, labels, None, None, 1.0, False, out, ws, limit)


def moe_head_xent_grad(x, Wv, labels, weight=None, out=None, ws=None, limit=0):
    """moe_head_xent and the gradients of sum_t weight[t] loss[t] (weight [T]
    f32, None: ones) -> {"loss", "lse", "dx" [T,d], "dWv" [V,d]}.  out: buffers by
    those names; None for dx or dWv leaves that gradient out."""
    return _head(x, Wv, labels, weight, None, 1.0, True, out, ws, limit)


def moe_head_distill(x, Wv, teacher, tau=1.0, labels=None, out=None, ws=None, limit=0):
    """The divergence from a teacher's top scores: teacher = (indices [T,K] i32,
    outside [0,V): no slot; scores [T,K] f32) -> {"kd" [T] f32}, with labels
    {"loss", "lse"} of the same scores too."""
    return _head(x, Wv, labels, None, teacher, tau, False, out, ws, limit)


def moe_head_distill_grad(x, Wv, teacher, tau=1.0, labels=None, weight=None, out=None, ws=None,
                          limit=0):
    """moe_head_distill and the gradients of sum_t u[t] kd[t] + weight[t] loss[t],
    u the teacher's third tensor ([T] f32, left out: ones)
    -> {"kd", "dx" [T,d], "dWv" [V,d]} and with labels {"loss", "lse"}."""
    return _head(x, Wv, labels, weight, teacher, tau, True, out, ws, limit)
