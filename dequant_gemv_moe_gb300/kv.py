"""torch-facing wrappers of the 4-bit paged K/V cache (marshalling only; see
the dq_kv_* section of include/dqmoe.h for what each call computes)."""
import ctypes
import struct

import torch

from ._lib import F16, F32, BF16, Q4_0, DqError, KvAttn, KvCacheDesc, KvRope, KvScores, lib

_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_plan, _append, _read, _attention, _rope = (lib.dq_kv_plan, lib.dq_kv_append, lib.dq_kv_read,
                                            lib.dq_kv_attention_ex, lib.dq_kv_append_rope)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# dq_kv_rope's fields as the compiler lays them out (a packed string is made in a third of a structure's time)
_ROPE = struct.Struct("@QqQqQqiiiQQQiifQqi0q")
assert _ROPE.size == ctypes.sizeof(KvRope)

# A decode step's calls take a few microseconds on the GPU, so the wrappers keep to few Python
# operations: bound functions, plain integers, the stream's handle without a Stream object.


def _stream(t):
    """The handle of the current stream; t has to lie on the current device, where kernels are launched."""
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError("tensors lie on device %d, the current device is %d" % (dev, _current_device()))
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(t.device).cuda_stream


def _raise(name, rc):
    raise DqError(name, rc)


def _device(t, name):
    """The index of t's CUDA device, on which all of a call's tensors have to lie."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _check(t, name, dtype, dev, shape=None):
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor of %s on device %d" % (name, dtype, dev))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))


class KvPlan:
    """A step's outputs of kv_plan: kv_len, q_start, positions, free_count, unserved (int32) and
    slots (int64), for B requests and n_tokens rows; a step may write to an earlier one's."""

    __slots__ = ("kv_len", "q_start", "slots", "positions", "free_count", "unserved", "size", "dev", "_ptrs")

    def __init__(self, B, n_tokens, device="cuda"):
        i32 = torch.empty(2 * B + 3 + n_tokens, dtype=torch.int32, device=device)
        self.kv_len, self.q_start = i32[:B], i32[B:2 * B + 1]
        self.free_count, self.unserved = i32[2 * B + 1:2 * B + 2], i32[2 * B + 2:2 * B + 3]
        self.positions = i32[2 * B + 3:]
        self.slots = torch.empty(n_tokens, dtype=torch.int64, device=device)
        self.size = (B, n_tokens)
        self.dev = _device(i32, "a plan")
        self._ptrs = tuple(t.data_ptr() for t in (self.kv_len, self.q_start, self.slots, self.positions,
                                                  self.free_count, self.unserved))


class KvCache:
    """A paged K/V cache in Q4_0 blocks over a caller's uint8 CUDA tensor.

    pages: the buffer, KvCache.size(...) bytes (its first dimension may be the
    pages); kept by this object, never written except by kv_append.
    """

    def __init__(self, pages, page_size, n_kv_heads, head_dim, fmt=Q4_0):
        d = KvCacheDesc(fmt, n_kv_heads, head_dim, page_size, 1, None)
        per_page = _size(d)
        self.dev = _device(pages, "pages")
        _check(pages, "pages", torch.uint8, self.dev)
        if pages.numel() < per_page or pages.numel() % per_page:
            raise ValueError("pages must hold a whole number of pages of %d bytes" % per_page)
        d.n_pages = pages.numel() // per_page
        d.pages = pages.data_ptr()
        self.pages, self.desc = pages, d
        self.page_size, self.n_kv_heads, self.head_dim = page_size, n_kv_heads, head_dim
        self.n_pages = d.n_pages
        self._ref = ctypes.byref(d)

    @staticmethod
    def size(n_pages, page_size, n_kv_heads, head_dim, fmt=Q4_0):
        """Bytes of a cache of n_pages pages."""
        return _size(KvCacheDesc(fmt, n_kv_heads, head_dim, page_size, n_pages, None))

    @classmethod
    def empty(cls, n_pages, page_size, n_kv_heads, head_dim, fmt=Q4_0, device="cuda"):
        """A cache over a new buffer (its contents are whatever the memory held)."""
        nb = cls.size(n_pages, page_size, n_kv_heads, head_dim, fmt)
        return cls(torch.empty(nb, dtype=torch.uint8, device=device), page_size, n_kv_heads,
                   head_dim, fmt)


def _size(desc):
    n = ctypes.c_size_t()
    rc = lib.dq_kv_cache_size(ctypes.byref(desc), ctypes.byref(n))
    return n.value if rc == 0 else _raise("dq_kv_cache_size", rc)


def kv_plan(ctx_len, new_len, block_table, free_pages, free_count, page_size, n_tokens, out=None):
    """One step's block tables (updated in place), slots and query starts.

    ctx_len, new_len: int32 [B]; block_table: int32 [B][max_pages]; free_pages:
    int32 stack, free_count: int32 [1]; n_tokens: rows of slots and positions.
    out: a KvPlan of an earlier step to write to (its free_count and kv_len may
    not be this call's inputs).
    """
    B, dev = ctx_len.numel(), _device(ctx_len, "ctx_len")
    _check(ctx_len, "ctx_len", torch.int32, dev)
    _check(new_len, "new_len", torch.int32, dev, (B,))
    _check(block_table, "block_table", torch.int32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B][max_pages]")
    _check(free_pages, "free_pages", torch.int32, dev)
    _check(free_count, "free_count", torch.int32, dev, (1,))
    if out is None:
        out = KvPlan(B, n_tokens, ctx_len.device)
    elif out.size != (B, n_tokens):
        raise ValueError("out holds %d requests and %d rows, not %d and %d" % (*out.size, B, n_tokens))
    elif out.dev != dev:
        raise ValueError("out must lie on device %d" % dev)
    rc = _plan(ctx_len.data_ptr(), new_len.data_ptr(), B, page_size, block_table.data_ptr(),
               block_table.shape[1], free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(),
               n_tokens, *out._ptrs, _stream(ctx_len))
    return out if rc == 0 else _raise("dq_kv_plan", rc)


def _rows(cache, t, name):
    """The token stride of rows [T][n_kv_heads][head_dim] (only the first may be strided)."""
    T, H, D = t.shape
    a, b, c = t.stride()
    if (H != cache.n_kv_heads or D != cache.head_dim or t.get_device() != cache.dev or c != 1 or
            (b != D and H > 1)):
        raise ValueError("%s must be a CUDA tensor [T][%d][%d] on device %d with consecutive heads" %
                         (name, cache.n_kv_heads, cache.head_dim, cache.dev))
    return a if T > 1 else H * D


def kv_append(cache, k, v, slots):
    """Write K and V rows ([T][n_kv_heads][head_dim], fp32/fp16/bf16; the token
    stride is free) into their slots (int64 [T], -1: left out)."""
    T = k.shape[0]
    if k.dtype != v.dtype or k.dtype not in _DT or v.shape[0] != T:
        raise ValueError("k and v must be rows of one dtype: float32, float16 or bfloat16")
    ks, vs = _rows(cache, k, "k"), _rows(cache, v, "v")
    _check(slots, "slots", torch.int64, cache.dev, (T,))
    if T:
        rc = _append(cache._ref, k.data_ptr(), ks, v.data_ptr(), vs, _DT[k.dtype], slots.data_ptr(), T,
                     _stream(k))
        if rc != 0:
            _raise("dq_kv_append", rc)


def _heads(t, D, dev, name):
    """The row stride of t [T][heads][D], whose heads are consecutive."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must be [T][heads][%d]" % (name, D))
    T, H, d = shape
    a, b, c = t.stride()
    if d != D or t.get_device() != dev or c != 1 or (b != D and H > 1) or t.dtype not in _DT:
        raise ValueError("%s must be a CUDA tensor [T][heads][%d] of float32, float16 or bfloat16 on device %d "
                         "with consecutive heads" % (name, D, dev))
    return a if T > 1 else H * D


def kv_append_rope(cache, q, k, v, slots, positions, inv_freq, interleaved=False, factor=1.0, out=None,
                   out_dtype=None):
    """kv_append of k rotated by its positions, and q rotated: the rows [T][n_q_heads][head_dim] of out.

    q, k, v: rows of one type (fp32/fp16/bf16; the token strides are free); q may be None.  positions int32 [T]:
    rows below 0 are left out; slots int64 [T] as kv_append's.  inv_freq fp32 [rotary_dim / 2]: the first
    rotary_dim values of a head turn, in pairs half of them apart or, interleaved, next to one another;
    factor: of cos and sin.  out: fp32/fp16/bf16 rows (out_dtype, q's unless given); q itself may be given.
    K's codes are those of the rotated values in 64 bits, its scales those of a group's largest value as fp32.
    """
    shape, D, dev = k.shape, cache.head_dim, cache.dev
    T, dt = shape[0], k.dtype
    (ks, kh, kd), (vs, vh, vd) = k.stride(), v.stride()
    H = cache.n_kv_heads
    # one test of all that has to hold; what is wrong is found out after it fails
    if not (shape == (T, H, D) and v.shape == shape and v.dtype is dt and dt in _DT and kd == 1 and vd == 1 and
            (H == 1 or (kh == D and vh == D)) and k.get_device() == dev and v.get_device() == dev and
            slots.shape == (T,) and slots.dtype is torch.int64 and slots.get_device() == dev and
            positions.shape == (T,) and positions.dtype is torch.int32 and positions.get_device() == dev and
            (T < 2 or (slots.stride(0) == 1 and positions.stride(0) == 1))):
        if k.dtype != v.dtype or k.dtype not in _DT or v.shape[0] != T:
            raise ValueError("k and v must be rows of one dtype: float32, float16 or bfloat16")
        _rows(cache, k, "k")
        _rows(cache, v, "v")
        _check(slots, "slots", torch.int64, dev, (T,))
        _check(positions, "positions", torch.int32, dev, (T,))
        raise ValueError("k, v, slots and positions do not fit together")
    _check(inv_freq, "inv_freq", torch.float32, dev)
    row = H * D
    n_q = qs = q_ptr = os = out_ptr = out_dt = 0
    if q is not None:
        qs = _heads(q, D, dev, "q")
        qshape = q.shape
        if q.dtype is not dt or qshape[0] != T:
            raise ValueError("q must be rows of k's dtype")
        if out is None:
            out = torch.empty(qshape, dtype=out_dtype or dt, device=q.device)
        elif out.shape != qshape:
            raise ValueError("out must have q's shape")
        n_q, q_ptr, out_ptr = qshape[1], q.data_ptr(), out.data_ptr()
        os, out_dt = _heads(out, D, dev, "out"), _DT[out.dtype]
    elif out is not None:
        raise ValueError("out is for q's rows")
    if T:
        a = _ROPE.pack(q_ptr, qs, k.data_ptr(), ks if T > 1 else row, v.data_ptr(), vs if T > 1 else row, _DT[dt], n_q, T,
                       slots.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.numel(), interleaved,
                       factor, out_ptr, os, out_dt)
        rc = _rope(cache._ref, a, _stream(k))
        if rc != 0:
            _raise("dq_kv_append_rope", rc)
    return out


def kv_read(cache, slots, dtype=torch.float32, out=None):
    """The values that slots stand for: (k, v), each [T][n_kv_heads][head_dim]."""
    T = slots.numel()
    _check(slots, "slots", torch.int64, cache.dev)
    shape = (T, cache.n_kv_heads, cache.head_dim)
    if out is None:
        out = (torch.empty(shape, dtype=dtype, device=slots.device),
               torch.empty(shape, dtype=dtype, device=slots.device))
    k, v = out
    dt = k.dtype
    if dt not in _DT:
        raise ValueError("values are float32, float16 or bfloat16")
    _check(k, "k", dt, cache.dev, shape)
    _check(v, "v", dt, cache.dev, shape)
    if T:
        rc = _read(cache._ref, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), _DT[dt], _stream(k))
        if rc != 0:
            _raise("dq_kv_read", rc)
    return k, v


def kv_attention_workspace_size(cache, n_q_heads, B, T, max_q_len=None):
    n = ctypes.c_size_t()
    rc = lib.dq_kv_attention_workspace_size(cache._ref, n_q_heads, T, B,
                                            T if max_q_len is None else max_q_len, ctypes.byref(n))
    return n.value if rc == 0 else _raise("dq_kv_attention_workspace_size", rc)


def kv_attention(cache, q, q_start, kv_len, block_table, scale=None, causal=True, window=0,
                 max_q_len=None, out=None, out_dtype=None, lse=None, ws=None, softcap=0.0, slopes=None,
                 prefix_len=None, first_pos=None):
    """Attention of q [T][n_q_heads][head_dim] (fp16/bf16; the row stride is
    free) over the cache: (out, lse), lse fp32 [T][n_q_heads].

    q_start int32 [B+1], kv_len int32 [B], block_table int32 [B][max_pages] as
    kv_plan leaves them; scale: head_dim ** -0.5 unless given; max_q_len: the
    most rows a request has (T unless given; a step that says 1 is one launch or two
    instead of four).  ws: kv_attention_workspace_size bytes for these T and max_q_len, or more.

    softcap: scores become softcap * tanh(scores / softcap); slopes fp32 [n_q_heads]: a head's scores lose its
    slope times the distance; prefix_len int32 [B]: the rows of a request see the positions below it whatever
    their own; first_pos int32 [T], not descending within a request: a row sees no position below it.

    Sums are fp32, operands fp16: weights are rounded to it, and where a request has
    many rows V and K as decoded too.  Whatever out_dtype is, out carries 1.5e-4 to
    4e-4 of its size from that; lse 1e-7, or up to 6e-6 for many rows that see more
    than 1024 tokens, or up to 1e-6 where scores are biased or masked.  A cap adds its own error: 2.5e-7 of a
    score, or, for many rows with caps up to 100 and no slopes, at most 7e-7 of the cap.
    """
    T, H, D = q.shape
    qs, qh, qd = q.stride()
    B, dev = kv_len.numel(), cache.dev
    if q.dtype not in _DT:
        raise TypeError("q must be float16 or bfloat16, got %s" % q.dtype)
    if D != cache.head_dim or q.get_device() != dev or qd != 1 or (qh != D and H > 1):
        raise ValueError("q must be a CUDA tensor [T][n_q_heads][%d] on device %d with consecutive heads" %
                         (cache.head_dim, dev))
    _check(q_start, "q_start", torch.int32, dev, (B + 1,))
    _check(kv_len, "kv_len", torch.int32, dev)
    _check(block_table, "block_table", torch.int32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B][max_pages]")
    if out is None:
        out = torch.empty((T, H, D), dtype=out_dtype or q.dtype, device=q.device)
    os, oh, od = out.stride()
    if (out.dtype not in _DT or out.shape != (T, H, D) or out.get_device() != dev or od != 1 or
            (oh != D and H > 1)):
        raise ValueError("out must be a CUDA tensor [T][n_q_heads][head_dim] on device %d with consecutive heads" % dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    else:
        _check(lse, "lse", torch.float32, dev, (T, H))
    if T == 0:
        return out, lse
    if max_q_len is None:
        max_q_len = T
    if ws is None:
        ws = torch.empty(kv_attention_workspace_size(cache, H, B, T, max_q_len), dtype=torch.uint8,
                         device=q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor on device %d" % dev)
    a = KvAttn(q.data_ptr(), qs if T > 1 else H * D, _DT[q.dtype], H, T, B, q_start.data_ptr(),
               kv_len.data_ptr(), block_table.data_ptr(), block_table.shape[1], max_q_len,
               D ** -0.5 if scale is None else scale, causal, window, out.data_ptr(),
               os if T > 1 else H * D, _DT[out.dtype], lse.data_ptr())
    x = None
    if softcap or slopes is not None or prefix_len is not None or first_pos is not None:
        x = KvScores(softcap)
        if slopes is not None:
            _check(slopes, "slopes", torch.float32, dev, (H,))
            x.slopes = slopes.data_ptr()
        if prefix_len is not None:
            _check(prefix_len, "prefix_len", torch.int32, dev, (B,))
            x.prefix_len = prefix_len.data_ptr()
        if first_pos is not None:
            _check(first_pos, "first_pos", torch.int32, dev, (T,))
            x.first_pos = first_pos.data_ptr()
        x = ctypes.byref(x)
    rc = _attention(cache._ref, ctypes.byref(a), x, ws.data_ptr(), ws.nbytes, _stream(q))
    return (out, lse) if rc == 0 else _raise("dq_kv_attention", rc)
