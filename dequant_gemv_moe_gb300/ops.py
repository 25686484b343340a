"""torch-facing wrappers of the C ABI (marshalling only; see include/dqmoe.h)."""
import ctypes

import torch

from ._lib import F16, F32, BF16, DqError, MoeDesc, MoeRoutingDesc, lib

_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(t):
    """The handle of the current stream; t has to lie on the current device, where kernels are launched."""
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError("tensors lie on device %d, the current device is %d" % (dev, _current_device()))
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _call(name, *args):
    rc = getattr(lib, name)(*args)
    if rc != 0:
        raise DqError(name, rc)


def _dtype_code(x):
    if x.dtype not in _DT:
        raise TypeError("activation dtype must be float32, float16 or bfloat16, got %s" % x.dtype)
    return _DT[x.dtype]


def block_geometry(fmt):
    qk, nb = ctypes.c_int(), ctypes.c_int()
    _call("dq_block_geometry", fmt, ctypes.byref(qk), ctypes.byref(nb))
    return qk.value, nb.value


def dequant(fmt, blocks, n_weights, out=None):
    """Decode n_weights weights of packed blocks (uint8 CUDA tensor) to fp32."""
    if out is None:
        out = torch.empty(n_weights, dtype=torch.float32, device=blocks.device)
    _call("dq_dequant", fmt, _ptr(blocks), n_weights, _ptr(out), _stream())
    return out


QGEMV_WEIGHTS_EARLY = 1


def qgemv(fmt, W, N, K, x, y=None, ksplit=None, weights_early=False):
    """y[b][n] = sum_k W[n][k] x[b][k]; x is [batch][K] (float32/float16/bfloat16).

    weights_early: W is not written by the kernel issued just before on the
    stream, so its first stages may stream in while that kernel drains
    (dq_qgemv_ex with DQ_QGEMV_WEIGHTS_EARLY).
    """
    x = x.reshape(-1, K)
    batch = x.shape[0]
    if y is None:
        y = torch.empty(batch, N, dtype=torch.float32, device=x.device)
    if weights_early:
        _call("dq_qgemv_ex", fmt, _ptr(W), N, K, _ptr(x), _dtype_code(x), batch, _ptr(y),
              int(ksplit or 0), QGEMV_WEIGHTS_EARLY, _stream())
    elif ksplit is None:
        _call("dq_qgemv", fmt, _ptr(W), N, K, _ptr(x), _dtype_code(x), batch, _ptr(y), _stream())
    else:
        _call("dq_qgemv_ksplit", fmt, _ptr(W), N, K, _ptr(x), _dtype_code(x), batch, _ptr(y),
              int(ksplit), _stream())
    return y


def stage(dst, src):
    """Copy src into dst (same number of bytes; CUDA or page-locked CPU tensors)
    with the library's copy kernel on the current stream (dq_stage)."""
    nb = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nb:
        raise ValueError("stage: dst and src sizes differ")
    _call("dq_stage", _ptr(dst), _ptr(src), nb, _stream())
    return dst


def device_status():
    v = ctypes.c_int()
    _call("dq_device_status", ctypes.byref(v))
    return v.value


# ---------------------------------------------------------------- MoE layer
def make_desc(E, top_k, hidden, ffn, n_shared, fmt, router_W, w_gate, w_up, w_down,
              sh_gate=None, sh_up=None, sh_down=None):
    d = MoeDesc()
    d.E, d.top_k, d.hidden, d.ffn, d.n_shared, d.fmt = E, top_k, hidden, ffn, n_shared, fmt
    d.router_W, d.w_gate, d.w_up, d.w_down = (router_W.data_ptr(), w_gate.data_ptr(),
                                              w_up.data_ptr(), w_down.data_ptr())
    d.sh_gate = sh_gate.data_ptr() if sh_gate is not None else None
    d.sh_up = sh_up.data_ptr() if sh_up is not None else None
    d.sh_down = sh_down.data_ptr() if sh_down is not None else None
    return d


def moe_workspace_size(desc, T):
    n = ctypes.c_size_t()
    _call("dq_moe_workspace_size", ctypes.byref(desc), T, ctypes.byref(n))
    return n.value


class MoeRouting:
    """How a layer's tokens choose their experts (dq_moe_routing of include/dqmoe.h).

    scores: "softmax" or "sigmoid"; bias: fp32 CUDA tensor [E] added to the scores for the choice alone, or
    None; n_groups groups of experts, of which a token keeps the top_groups best by group_score, "max" or "top2"
    (the sum of the two largest); renormalize: gates are shares of the chosen scores' sum; scale: of the gates.
    """

    def __init__(self, scores="softmax", bias=None, n_groups=1, top_groups=1, group_score="max", renormalize=True,
                 scale=1.0):
        if scores not in ("softmax", "sigmoid") or group_score not in ("max", "top2"):
            raise ValueError('scores are "softmax" or "sigmoid", group_score is "max" or "top2"')
        if bias is not None and (bias.dtype is not torch.float32 or not bias.is_cuda or not bias.is_contiguous() or
                                 bias.dim() != 1):
            raise ValueError("bias must be a contiguous CUDA tensor [E] of float32")
        self.bias = bias
        self.desc = MoeRoutingDesc(int(scores == "sigmoid"), n_groups, top_groups, int(group_score == "top2"),
                                   int(bool(renormalize)), scale, bias.data_ptr() if bias is not None else None)
        self._ref = ctypes.byref(self.desc)
        self._bias_of = None if bias is None else (bias.numel(), bias.get_device())

    def check(self, E, dev):
        if self._bias_of is not None and self._bias_of != (E, dev):
            raise ValueError("the routing's bias must hold %d experts' on device %d" % (E, dev))
        return self._ref


_DEFAULT_ROUTING = MoeRouting()
_route = lib.dq_moe_route


def moe_route(logits, top_k, routing=None, out=None):
    """The experts and gates of logits [T][E] (fp32/fp16/bf16; the row stride is free): (int32 [T][top_k],
    fp32 [T][top_k]).  routing: a MoeRouting (softmax over all experts, renormalised, unless given)."""
    shape, dev = logits.shape, logits.get_device()
    if len(shape) != 2 or dev < 0:
        raise ValueError("logits must be a CUDA tensor [T][E] with consecutive experts")
    T, E = shape
    stride, one = logits.stride()
    if one != 1 and E > 1:
        raise ValueError("logits must be a CUDA tensor [T][E] with consecutive experts")
    ref = (routing or _DEFAULT_ROUTING).check(E, dev)
    if out is None:
        out = (torch.empty(T, top_k, dtype=torch.int32, device=logits.device),
               torch.empty(T, top_k, dtype=torch.float32, device=logits.device))
    idx, gate = out
    if (idx.dtype is not torch.int32 or gate.dtype is not torch.float32 or idx.shape != (T, top_k) or
            gate.shape != (T, top_k) or idx.get_device() != dev or gate.get_device() != dev or
            not idx.is_contiguous() or not gate.is_contiguous()):
        raise ValueError("out must be contiguous CUDA tensors [%d][%d] of int32 and float32 on device %d" %
                         (T, top_k, dev))
    if T:
        rc = _route(logits.data_ptr(), _dtype_code(logits), stride if T > 1 else E, T, E, top_k, ref,
                    idx.data_ptr(), gate.data_ptr(), _stream_of(logits))
        if rc != 0:
            raise DqError("dq_moe_route", rc)
    return out


def moe_router(router_W, E, H, x, top_k, logits=None, routing=None):
    T = x.shape[0]
    dev = x.device
    if logits is None:
        logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    idx = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    gate = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    ref = routing.check(E, x.get_device()) if routing is not None else None
    _call("dq_moe_router_ex", _ptr(router_W), E, H, _ptr(x), _dtype_code(x), T, top_k, ref, _ptr(logits),
          _ptr(idx), _ptr(gate), _stream())
    return logits, idx, gate


def moe_permute(topk_idx, E):
    T, k = topk_idx.shape
    dev = topk_idx.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_ = torch.empty(T * k, dtype=torch.int32, device=dev)
    _call("dq_moe_permute", _ptr(topk_idx), T, k, E, _ptr(offsets), _ptr(sorted_), _stream())
    return offsets, sorted_


def moe_forward(desc, x, y=None, ws=None, want_routing=False, routing=None):
    """The whole MoE layer.  Returns y (and idx, gate, logits if want_routing).
    routing: a MoeRouting in place of the layer's softmax top-k."""
    T = x.shape[0]
    dev = x.device
    if y is None:
        y = torch.empty(T, desc.hidden, dtype=torch.float32, device=dev)
    need = moe_workspace_size(desc, T)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    idx = gate = logits = None
    if want_routing:
        idx = torch.empty(T, desc.top_k, dtype=torch.int32, device=dev)
        gate = torch.empty(T, desc.top_k, dtype=torch.float32, device=dev)
        logits = torch.empty(T, desc.E, dtype=torch.float32, device=dev)
    ref = routing.check(desc.E, x.get_device()) if routing is not None else None
    _call("dq_moe_forward_ex", ctypes.byref(desc), ref, _ptr(x), _dtype_code(x), T, _ptr(y), _ptr(ws),
          ws.numel(), _ptr(idx), _ptr(gate), _ptr(logits), _stream())
    if want_routing:
        return y, idx, gate, logits
    return y


# ------------------------------------------------------- expert streaming
class ExpertCache:
    """A device cache of `slots` experts for a layer whose routed experts live
    in page-locked host memory (dq_expert_cache_*; marshalling only).

    host_w_gate / host_w_up / host_w_down: pinned CPU uint8 tensors of all E
    experts; router_W and the shared experts (optional) are CUDA tensors.  The
    slot buffers are allocated here as CUDA tensors and kept by this object.
    """

    def __init__(self, E, top_k, hidden, ffn, n_shared, fmt, router_W, host_w_gate, host_w_up,
                 host_w_down, sh_gate=None, sh_up=None, sh_down=None, slots=None,
                 max_tokens=1, phases=2, routing=None):
        self.desc = make_desc(E, top_k, hidden, ffn, n_shared, fmt, router_W, host_w_gate,
                              host_w_up, host_w_down, sh_gate, sh_up, sh_down)
        self._keep = (router_W, host_w_gate, host_w_up, host_w_down, sh_gate, sh_up, sh_down)
        if slots is None:
            slots = min(E, max_tokens * top_k)
        dev = router_W.device
        gu = host_w_gate.numel() // E
        dn = host_w_down.numel() // E
        self.slot_gate = torch.empty(slots * gu, dtype=torch.uint8, device=dev)
        self.slot_up = torch.empty(slots * gu, dtype=torch.uint8, device=dev)
        self.slot_down = torch.empty(slots * dn, dtype=torch.uint8, device=dev)
        self.max_tokens = max_tokens
        h = ctypes.c_void_p()
        _call("dq_expert_cache_create", ctypes.byref(self.desc), slots, _ptr(self.slot_gate),
              _ptr(self.slot_up), _ptr(self.slot_down), max_tokens, phases, ctypes.byref(h))
        self.handle = h
        self.set_routing(routing)
        self.copy_stream = torch.cuda.Stream(device=dev)

    def set_routing(self, routing):
        """The routing of the calls that follow: a MoeRouting, or None for the layer's softmax top-k."""
        ref = routing.check(self.desc.E, self.slot_gate.get_device()) if routing is not None else None
        _call("dq_expert_cache_set_routing", self.handle, ref)
        self.routing = routing

    def workspace_size(self, T):
        n = ctypes.c_size_t()
        _call("dq_expert_cache_workspace_size", self.handle, T, ctypes.byref(n))
        return n.value

    def forward(self, x, y=None, ws=None):
        """The layer for x [T][hidden] on the current stream (copies on this
        cache's copy stream)."""
        T = x.shape[0]
        if y is None:
            y = torch.empty(T, self.desc.hidden, dtype=torch.float32, device=x.device)
        if ws is None:
            ws = torch.empty(self.workspace_size(T), dtype=torch.uint8, device=x.device)
        _call("dq_moe_forward_streamed", self.handle, _ptr(x), _dtype_code(x), T, _ptr(y),
              _ptr(ws), ws.numel(), _stream(), ctypes.c_void_p(self.copy_stream.cuda_stream))
        return y

    def stats(self):
        h, m, b = ctypes.c_longlong(), ctypes.c_longlong(), ctypes.c_longlong()
        _call("dq_expert_cache_stats", self.handle, ctypes.byref(h), ctypes.byref(m),
              ctypes.byref(b))
        return {"hits": h.value, "misses": m.value, "bytes_copied": b.value}

    def close(self):
        if self.handle:
            _call("dq_expert_cache_destroy", self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
