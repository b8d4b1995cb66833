"""ctypes binding of the decode-state operators (include/qgkv.h): the 8-bit
paged key/value cache, its attention, page operations, the adjustment of logits and
beam selection.

Argument marshalling only: each function checks torch CUDA tensors and calls
the C entry point on the current torch stream (or on `stream=`).  There is
no CPU fallback; a refused call raises ``qgemv.QGError``, a wrong type or shape
``TypeError`` / ``ValueError``, and so do tensors that are not on the current
device.  Tensors given to a call with `stream=` are recorded on that stream; the
caller orders the streams.

    cache = KVCache.allocate(layers=22, pages=4096, heads=4, page_tokens=64, head_dim=64)
    ws = KVWorkspace("cuda")
    kv_reserve(cache, table, lens, refs, workspace=ws)       # pages for one token each
    q = kv_append_rotary(cache, layer, q, k, v, rope, table, lens)  # or kv_append; then lens += 1
    out = kv_attention(cache, layer, q, table, lens, workspace=ws)
    plan = kv_share(cache, table, lens, groups)              # once a step: what its sequences have in common
    out = kv_attention_shared(cache, layer, q, table, lens, plan, workspace=ws)
    logits = adjust_logits(logits, history, history_lens, repetition=penalty, mask=allowed)
    scores, tokens, parents = beam_select(logits, cum, keep, workspace=ws)
    table, lens, refs = kv_fork(cache, table, lens, parents.view(-1), refs, workspace=ws)
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import qgemv as _q

QGKV_E4M3 = 1
QGKV_INT8 = 2
QGKV_HND = 0
QGKV_NHD = 1
QGKV_MAX_BATCH = 4096
QGKV_MAX_PAGES = 1 << 20
QGKV_MAX_BEAMS = 64
QGKV_MAX_KEEP = 128
QGKV_MAX_HISTORY = (1 << 20) - 1
QGKV_MAX_BIASES = 2047
FORMATS = {"e4m3": QGKV_E4M3, "int8": QGKV_INT8}
ORDERS = {"hnd": QGKV_HND, "nhd": QGKV_NHD}
PAIRS = {"interleaved": 0, "halves": 1}
TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

EXPORTS = ("qgkv_workspace_bytes", "qgkv_append", "qgkv_attention", "qgkv_copy_pages", "qgkv_fork", "qgkv_compact",
           "qgkv_reserve", "qgkv_free", "qgbeam_select", "qgkv_append_rotary", "qglogits_adjust", "qgkv_share",
           "qgkv_attention_shared")


class QgkvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("layers", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int),
                ("order", ctypes.c_int)]


_fns = {}


def load():
    """The entry points of libqgemv.so declared in include/qgkv.h, by name."""
    if _fns:
        return _fns
    lib = _q.load()
    vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sigs = {
        "qgkv_workspace_bytes": [],
        "qgkv_append": [vp, i64, vp, vp, ci, i64, i64, i64, vp, i64, vp, vp, ci, vp],
        "qgkv_attention": [vp, i64, vp, vp, vp, ci, i64, ci, i64, i64, vp, i64, vp, vp, ci, cf, vp, i64, vp],
        "qgkv_attention_shared": [vp, i64, vp, vp, vp, ci, i64, ci, i64, i64, vp, i64, vp, vp, ci, vp, ci, cf, vp, i64, vp],
        "qgkv_share": [i64, ci, vp, i64, vp, vp, i64, ci, vp, ci, vp, vp],
        "qgkv_copy_pages": [vp, vp, vp, vp, i64, vp],
        "qgkv_fork": [vp, vp, i64, vp, ci, vp, ci, vp, vp, vp, vp, vp, i64, vp],
        "qgkv_compact": [vp, vp, i64, vp, ci, vp, vp, vp, vp, vp, vp, vp, i64, vp],
        "qgkv_reserve": [i64, ci, vp, i64, vp, vp, ci, vp, vp, i64, vp],
        "qgkv_free": [i64, ci, vp, i64, vp, vp, ci, vp, vp],
        "qgkv_append_rotary": [vp, i64, vp, vp, vp, ci, i64, ci, i64, i64, i64, i64, vp, i64, ci, ci, vp, vp, i64, vp, vp,
                               ci, vp],
        "qglogits_adjust": [vp, ci, i64, i64, i64, vp, ci, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, ci, vp, vp, i64, ci,
                            vp, vp],
        "qgbeam_select": [vp, ci, vp, ci, ci, i64, i64, ci, vp, vp, vp, vp, i64, vp],
    }
    got = {}
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = i64 if name == "qgkv_workspace_bytes" else ci
        got[name] = f
    _fns.update(got)
    return _fns


def _call(name, *args):
    rc = (_fns or load())[name](*args)
    if rc:
        _q._check(name, rc)


def _other(stream, *tensors):
    """Whether a call has to be made again with `stream` current, so that what it allocates belongs to it.
    What it is given (None, caches and workspaces too) is lent to that stream: memory of a tensor that the
    caller drops after the call is not used again before the stream is done with it."""
    if stream is None or stream == torch.cuda.current_stream():
        return False
    for t in tensors:
        if isinstance(t, KVCache):
            _other(stream, t.k, t.k_scale, t.v, t.v_scale)
        elif isinstance(t, KVWorkspace):
            t.buffer.record_stream(stream)
        elif isinstance(t, (tuple, list)):
            _other(stream, *t)
        elif isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return True


def _stream(*tensors):
    """The current stream of the tensors' device (None is passed over).  They lie on one device and it is
    the current one: the library launches there, on the pointers it is given."""
    device = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor lies on cuda:{t.get_device()}, the current device is cuda:{device}: all "
                             "have to be on the current device (torch.cuda.device)")
    return torch._C._cuda_getCurrentRawStream(device)


def _need(t, dtype, name, shape=None):
    """The address of a contiguous CUDA tensor of this type (and shape, None where free)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        if t.dim() != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape)):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    return t.data_ptr()


def _rows(t, heads, dim, name):
    """(pointer, type, rows, row stride, head stride) of a [rows, heads, dim] tensor with dense heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    kind = TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, not (rows, {heads}, {dim})")
    row, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: a head's values must be dense")
    # strides of a dimension of one element carry no meaning
    rows = shape[0]
    if heads == 1:
        head = dim
    if rows == 1:
        row = heads * head
    return t.data_ptr(), kind, rows, row, head


class KVWorkspace:
    """Device workspace of the operators; one serves one stream (calls that may overlap need one each).

    A call without one (``workspace=None``) allocates and clears its own, 47 MB of memory traffic and a launch
    more: give every call of a decode loop the same one.
    """

    def __init__(self, device="cuda"):
        self.bytes = int(load()["qgkv_workspace_bytes"]())
        self.buffer = torch.zeros(self.bytes, dtype=torch.uint8, device=device)
        self.ptr = self.buffer.data_ptr()


class KVCache:
    """An 8-bit paged cache over the caller's tensors.

    k, v: uint8 [layers, pages, heads, page_tokens, head_dim] (order "hnd") or
    [layers, pages, page_tokens, heads, head_dim] ("nhd"), dense inside a page;
    k_scale, v_scale: float32 [layers, pages, heads].  fmt: "e4m3" or "int8".
    """

    def __init__(self, k, k_scale, v, v_scale, fmt="e4m3", order="hnd"):
        if fmt not in FORMATS:
            raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
        if order not in ORDERS:
            raise ValueError(f"order must be one of {sorted(ORDERS)}, got {order!r}")
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8:
                raise TypeError(f"{name} must be a uint8 CUDA tensor")
            if t.dim() != 5 or not t[0, 0].is_contiguous():
                raise ValueError(f"{name} must be [layers, pages, ...] of pages that are dense inside")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must have the same shape and strides")
        self.k, self.v, self.k_scale, self.v_scale, self.fmt, self.order = k, v, k_scale, v_scale, fmt, order
        self.layers, self.pages = int(k.shape[0]), int(k.shape[1])
        a, b, self.head_dim = int(k.shape[2]), int(k.shape[3]), int(k.shape[4])
        self.heads, self.page_tokens = (a, b) if order == "hnd" else (b, a)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t, torch.float32, name, (self.layers, self.pages, self.heads))
        if not k.get_device() == v.get_device() == k_scale.get_device() == v_scale.get_device():
            raise ValueError("k, v and their scales must lie on one device")
        dense = a * b * self.head_dim
        self.c = QgkvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.layers, self.pages,
                           k.stride(0) if self.layers > 1 else dense, k.stride(1) if self.pages > 1 else dense,
                           self.heads, self.page_tokens, self.head_dim, FORMATS[fmt], ORDERS[order])
        self.ref = ctypes.addressof(self.c)
        self.scale = 1.0 / math.sqrt(self.head_dim)

    @classmethod
    def allocate(cls, layers, pages, heads, page_tokens, head_dim, fmt="e4m3", order="hnd", device="cuda"):
        """A cache of its own tensors, codes and scales zero."""
        inner = (heads, page_tokens) if order == "hnd" else (page_tokens, heads)
        k = torch.zeros((layers, pages, *inner, head_dim), dtype=torch.uint8, device=device)
        s = torch.zeros((layers, pages, heads), device=device)
        return cls(k, s, torch.zeros_like(k), torch.zeros_like(s), fmt, order)


def _batch(table, lens, starts):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [batch, width]")
    batch, width = table.shape
    t, n = _need(table, torch.int32, "table"), _need(lens, torch.int32, "lens", (batch,))
    s = None if starts is None else _need(starts, torch.int32, "starts", (batch + 1,))
    return batch, width, t, n, s


def _ws(workspace, t):
    """The workspace of a call; where None is given, a cleared one for this call alone."""
    w = KVWorkspace(t.device) if workspace is None else workspace
    return w, w.ptr, w.bytes


def kv_append(cache, layer, k, v, table, lens, starts=None, stream=None):
    """Quantise new tokens k, v [rows, heads, head_dim] into the cache behind each
    sequence's lens[b] tokens (qgkv_append); rows by `starts`, or one a sequence."""
    if _other(stream, cache, k, v, table, lens, starts):
        with torch.cuda.stream(stream):
            return kv_append(cache, layer, k, v, table, lens, starts)
    batch, width, tp, lp, sp = _batch(table, lens, starts)
    kp, kind, rows, row, head = _rows(k, cache.heads, cache.head_dim, "k")
    vp, kind_v, rows_v, row_v, head_v = _rows(v, cache.heads, cache.head_dim, "v")
    if (kind, rows, row, head) != (kind_v, rows_v, row_v, head_v):
        raise ValueError("k and v must have the same type, shape and strides")
    _call("qgkv_append", cache.ref, layer, kp, vp, kind, rows, row, head, tp, width, lp, sp, batch,
          _stream(k, v, cache.k, table, lens, starts))


def rotary_table(positions, turned, base=10000.0, device="cuda"):
    """The table that kv_append_rotary takes, float32 [positions, turned]: for each position
    turned / 2 cosines, then as many sines, of position * base ** (-2 j / turned), angles in 64 bits."""
    half = turned // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((torch.cos(angle), torch.sin(angle)), dim=1).float()


def kv_append_rotary(cache, layer, q, k, v, rope, table, lens, starts=None, pairs="interleaved", out=None, stream=None):
    """kv_append of keys turned to their positions, lens[b] + i for row i of sequence b, and the queries
    of the same rows turned alike (qgkv_append_rotary).  q [rows, q_heads, head_dim] or None, k, v [rows,
    heads, head_dim]; rope float32 [positions, turned], as rotary_table makes it; pairs "interleaved" or
    "halves".  Returns the turned queries (`out`, which may be q where q is contiguous), None without q."""
    if stream is not None and _other(stream, cache, q, k, v, rope, table, lens, starts, out):
        with torch.cuda.stream(stream):
            return kv_append_rotary(cache, layer, q, k, v, rope, table, lens, starts, pairs, out)
    if pairs not in PAIRS:
        raise ValueError(f"pairs must be one of {sorted(PAIRS)}, got {pairs!r}")
    batch, width, tp, lp, sp = _batch(table, lens, starts)
    kp, kind, rows, row, head = _rows(k, cache.heads, cache.head_dim, "k")
    vp, kind_v, rows_v, row_v, head_v = _rows(v, cache.heads, cache.head_dim, "v")
    if (kind, rows, row, head) != (kind_v, rows_v, row_v, head_v):
        raise ValueError("k and v must have the same type, shape and strides")
    rp = _need(rope, torch.float32, "rope", (None, None))
    qp = op = None
    q_heads = q_row = q_head = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [rows, q_heads, head_dim]")
        q_heads = q.shape[1]
        qp, kind_q, rows_q, q_row, q_head = _rows(q, q_heads, cache.head_dim, "q")
        if (kind_q, rows_q) != (kind, rows):
            raise ValueError("q must have the type and the rows of k and v")
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            op = out.data_ptr()
        else:
            op = _need(out, q.dtype, "out", (rows, q_heads, cache.head_dim))
    elif out is not None:
        raise ValueError("out is for the turned queries, there is no q")
    _call("qgkv_append_rotary", cache.ref, layer, qp, kp, vp, kind, rows, q_heads, q_row, q_head, row, head, rp,
          rope.shape[0], rope.shape[1], PAIRS[pairs], op, tp, width, lp, sp, batch,
          _stream(q, k, v, cache.k, rope, out, table, lens, starts))
    return out


def _queries(cache, q, out, lse, return_lse):
    """(rows, q_heads, the C call's arguments for q, out, lse) of an attention, with the outputs made where None."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    heads = q.shape[1]
    qp, kind, rows, row, head = _rows(q, heads, cache.head_dim, "q")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        op = _need(out, q.dtype, "out", (rows, heads, cache.head_dim))
    if lse is not None:
        ep = _need(lse, torch.float32, "lse", (rows, heads))
    elif return_lse:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=q.device)
        ep = lse.data_ptr()
    else:
        ep = None
    return out, lse, (qp, op, ep, kind, rows, heads, row, head)


def kv_attention(cache, layer, q, table, lens, starts=None, scale=None, out=None, lse=None, return_lse=False,
                 workspace=None, stream=None):
    """softmax(scale * q k^T) v over each sequence's lens[b] tokens, causal at their end
    (qgkv_attention).  q [rows, q_heads, head_dim]; returns out, or (out, lse) with
    return_lse.  scale: 1 / sqrt(head_dim) where None."""
    if stream is not None and _other(stream, cache, q, table, lens, starts, out, lse, workspace):
        with torch.cuda.stream(stream):
            return kv_attention(cache, layer, q, table, lens, starts, scale, out, lse, return_lse, workspace)
    batch, width, tp, lp, sp = _batch(table, lens, starts)
    out, lse, args = _queries(cache, q, out, lse, return_lse)
    w, wp, wb = _ws(workspace, q)
    _call("qgkv_attention", cache.ref, layer, *args, tp, width, lp, sp, batch,
          cache.scale if scale is None else scale, wp, wb,
          _stream(q, cache.k, out, lse, table, lens, starts, w.buffer))
    return (out, lse) if return_lse else out


def kv_share(cache, table, lens, groups, starts=None, rows=None, out=None, stream=None):
    """What the sequences of each group have in common, for kv_attention_shared (qgkv_share): sequences
    groups[g] .. groups[g + 1] - 1 (int32 [n + 1]) are group g, lens counts the step's tokens already.  Returns
    the plan, int32 [4 n + batch]: (first row, rows, tokens shared, first sequence) of each group, then the
    tokens that each sequence shares.  It is read and made on the device, once for all layers of a step.
    rows: the number of query rows; where None, and with starts, rows outside the queries are first found by
    the attention.

    A group shares what all its sequences have in common, so a short one, or one that left the prompt, sets it for
    the others.  A batch of fewer than four sequences to a group shares nothing: leave sequences of their own before
    the first border or behind the last, not as groups of one."""
    if stream is not None and _other(stream, cache, table, lens, groups, starts, out):
        with torch.cuda.stream(stream):
            return kv_share(cache, table, lens, groups, starts, rows, out)
    batch, width, tp, lp, sp = _batch(table, lens, starts)
    gp = _need(groups, torch.int32, "groups", (None,))
    n = groups.shape[0] - 1
    if n < 1:
        raise ValueError("groups must be [number of groups + 1]")
    if out is None:
        out = torch.empty((4 * n + batch,), dtype=torch.int32, device=table.device)
    op = _need(out, torch.int32, "out", (4 * n + batch,))
    if rows is None:
        rows = batch if starts is None else (1 << 31) - 1
    _call("qgkv_share", cache.pages, cache.page_tokens, tp, width, lp, sp, rows, batch, gp, n, op,
          _stream(table, lens, groups, starts, out, cache.k))
    return out


def kv_attention_shared(cache, layer, q, table, lens, plan, starts=None, scale=None, out=None, lse=None,
                        return_lse=False, workspace=None, stream=None):
    """kv_attention of a batch whose groups share pages, which are read once for all rows of a group
    (qgkv_attention_shared).  plan: what kv_share gave for the same table, lens and starts."""
    if stream is not None and _other(stream, cache, q, table, lens, plan, starts, out, lse, workspace):
        with torch.cuda.stream(stream):
            return kv_attention_shared(cache, layer, q, table, lens, plan, starts, scale, out, lse, return_lse, workspace)
    batch, width, tp, lp, sp = _batch(table, lens, starts)
    pp = _need(plan, torch.int32, "plan", (None,))
    groups = (plan.shape[0] - batch) // 4
    if groups < 1 or 4 * groups + batch != plan.shape[0]:
        raise ValueError(f"plan has {plan.shape[0]} entries, not 4 * groups + batch")
    out, lse, args = _queries(cache, q, out, lse, return_lse)
    w, wp, wb = _ws(workspace, q)
    _call("qgkv_attention_shared", cache.ref, layer, *args, tp, width, lp, sp, batch, pp, groups,
          cache.scale if scale is None else scale, wp, wb,
          _stream(q, cache.k, out, lse, table, lens, starts, plan, w.buffer))
    return (out, lse) if return_lse else out


def kv_copy_pages(cache, src, dst, count=None, stream=None):
    """Copy pages src[i] to dst[i] (int32), codes and scales of every layer; `count` (int32 [1])
    limits them on the device."""
    if _other(stream, cache, src, dst, count):
        with torch.cuda.stream(stream):
            return kv_copy_pages(cache, src, dst, count)
    sp, dp = _need(src, torch.int32, "src", (None,)), _need(dst, torch.int32, "dst", tuple(src.shape))
    cp = None if count is None else _need(count, torch.int32, "count", (1,))
    _call("qgkv_copy_pages", cache.ref, sp, dp, cp, src.shape[0], _stream(src, dst, count, cache.k))


def _outs(table, refs, rows, out):
    if out is None:
        return (torch.empty((rows, table.shape[1]), dtype=torch.int32, device=table.device),
                torch.empty((rows,), dtype=torch.int32, device=table.device), torch.empty_like(refs))
    table2, lens2, refs2 = out
    _need(table2, torch.int32, "table2", (rows, table.shape[1]))
    _need(lens2, torch.int32, "lens2", (rows,))
    _need(refs2, torch.int32, "refs2", tuple(refs.shape))
    return table2, lens2, refs2


def kv_fork(cache, table, lens, parent, refs, out=None, workspace=None, stream=None):
    """New sequences that continue sequences parent[i] (qgkv_fork): whole pages shared,
    shared partly filled pages copied.  Returns (table2, lens2, refs2); `out` takes the three."""
    if _other(stream, cache, table, lens, parent, refs, out, workspace):
        with torch.cuda.stream(stream):
            return kv_fork(cache, table, lens, parent, refs, out, workspace)
    batch, width, tp, lp, _ = _batch(table, lens, None)
    pp = _need(parent, torch.int32, "parent", (None,))
    rp = _need(refs, torch.int32, "refs", (cache.pages,))
    rows = parent.shape[0]
    table2, lens2, refs2 = _outs(table, refs, rows, out)
    w, wp, wb = _ws(workspace, table)
    _call("qgkv_fork", cache.ref, tp, width, lp, batch, pp, rows, rp, table2.data_ptr(), lens2.data_ptr(),
          refs2.data_ptr(), wp, wb, _stream(table, lens, parent, refs, table2, lens2, refs2, cache.k, w.buffer))
    return table2, lens2, refs2


def kv_compact(cache, table, lens, refs, drop=None, out=None, workspace=None, stream=None):
    """Free the sequences marked by drop (bool or uint8 [batch]) and move the held pages to the
    lowest numbers (qgkv_compact).  Returns (table2, lens2, refs2, count of held pages [1])."""
    if _other(stream, cache, table, lens, refs, drop, out, workspace):
        with torch.cuda.stream(stream):
            return kv_compact(cache, table, lens, refs, drop, out, workspace)
    batch, width, tp, lp, _ = _batch(table, lens, None)
    rp = _need(refs, torch.int32, "refs", (cache.pages,))
    dp = _mask(drop, batch)
    table2, lens2, refs2 = _outs(table, refs, batch, out)
    count = torch.empty((1,), dtype=torch.int32, device=table.device)
    w, wp, wb = _ws(workspace, table)
    _call("qgkv_compact", cache.ref, tp, width, lp, batch, dp, rp, table2.data_ptr(), lens2.data_ptr(),
          refs2.data_ptr(), count.data_ptr(), wp, wb,
          _stream(table, lens, drop, refs, table2, lens2, refs2, cache.k, w.buffer))
    return table2, lens2, refs2, count


def _mask(drop, batch):
    if drop is None:
        return None
    return _need(drop, torch.bool if drop.dtype == torch.bool else torch.uint8, "drop", (batch,))


def kv_reserve(cache, table, lens, refs, add=None, workspace=None, stream=None):
    """Give each sequence the pages that lens[b] + add[b] tokens need (add None: one token each);
    table and refs are updated (qgkv_reserve).  Raise lens once the tokens are stored, before any
    fork, compaction or free: pages beyond lens do not count for these."""
    if _other(stream, cache, table, lens, refs, add, workspace):
        with torch.cuda.stream(stream):
            return kv_reserve(cache, table, lens, refs, add, workspace)
    batch, width, tp, lp, _ = _batch(table, lens, None)
    ap = None if add is None else _need(add, torch.int32, "add", (batch,))
    rp = _need(refs, torch.int32, "refs", (cache.pages,))
    w, wp, wb = _ws(workspace, table)
    _call("qgkv_reserve", cache.pages, cache.page_tokens, tp, width, lp, ap, batch, rp, wp, wb,
          _stream(table, lens, add, refs, w.buffer))


def kv_free(cache, table, lens, refs, drop=None, stream=None):
    """Free the sequences marked by drop (None: all): table, lens and refs are updated (qgkv_free)."""
    if _other(stream, cache, table, lens, refs, drop):
        with torch.cuda.stream(stream):
            return kv_free(cache, table, lens, refs, drop)
    batch, width, tp, lp, _ = _batch(table, lens, None)
    rp = _need(refs, torch.int32, "refs", (cache.pages,))
    _call("qgkv_free", cache.pages, cache.page_tokens, tp, width, lp, _mask(drop, batch), batch, rp,
          _stream(table, lens, drop, refs))


def beam_select(logits, cum, keep, workspace=None, stream=None):
    """The `keep` best continuations of each request (qgbeam_select): logits
    [requests * beams, vocab], cum float32 [requests, beams].  Returns scores float32, tokens
    int32 and parents int32 (row numbers), each [requests, keep]."""
    if _other(stream, logits, cum, workspace):
        with torch.cuda.stream(stream):
            return beam_select(logits, cum, keep, workspace)
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 2:
        raise TypeError("logits must be a CUDA tensor [rows, vocab]")
    kind = TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    cp = _need(cum, torch.float32, "cum", (None, None))
    requests, beams = cum.shape
    rows, vocab = logits.shape
    if rows != requests * beams:
        raise ValueError(f"logits has {rows} rows, not requests * beams = {requests * beams}")
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("a row of logits must be dense")
    scores = torch.empty((requests, keep), dtype=torch.float32, device=logits.device)
    ints = torch.empty((2, requests, keep), dtype=torch.int32, device=logits.device)
    tokens, parents = ints.unbind(0)
    w, wp, wb = _ws(workspace, logits)
    _call("qgbeam_select", logits.data_ptr(), kind, cp, requests, beams, vocab,
          logits.stride(0) if rows > 1 else vocab, keep, scores.data_ptr(), tokens.data_ptr(), parents.data_ptr(), wp,
          wb, _stream(logits, cum, w.buffer))
    return scores, tokens, parents


def adjust_logits(logits, history=None, lens=None, prompt_lens=None, repetition=None, presence=None, frequency=None,
                  bias_tokens=None, bias=None, temperature=None, mask=None, mask_rows=None, out=None, stream=None):
    """Penalties for tokens that have come before, listed biases, temperature and a grammar's mask, in
    this order (qglogits_adjust).  logits [rows, vocab]; history int32 [rows, width] of which lens int32
    [rows] tokens count, the first prompt_lens of them given and not produced; repetition, presence,
    frequency, temperature float32 [rows]; bias_tokens int32 and bias float32 [rows, biases], places
    without one -1; mask int32 [masks, words], bit t % 32 of word t // 32 is 1 where token t is allowed, one
    a row or named by mask_rows int32 [rows] (-1: none).  Returns `out` (of the logits' type or float32;
    logits itself works in place), a new tensor of the logits' type where None."""
    if stream is not None and _other(stream, logits, history, lens, prompt_lens, repetition, presence, frequency,
                                     bias_tokens, bias, temperature, mask, mask_rows, out):
        with torch.cuda.stream(stream):
            return adjust_logits(logits, history, lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias,
                                 temperature, mask, mask_rows, out)
    kind, rows, vocab, row = _logits(logits, "logits")
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    out_kind, out_rows, out_vocab, out_row = (kind, rows, vocab, row) if out is logits else _logits(out, "out")
    if (out_rows, out_vocab) != (rows, vocab):
        raise ValueError(f"out has shape {tuple(out.shape)}, not {(rows, vocab)}")

    i32, f32, each = torch.int32, torch.float32, (rows,)
    hp = width = tp = bp = mp = None
    past = (None if lens is None else _need(lens, i32, "lens", each),
            None if prompt_lens is None else _need(prompt_lens, i32, "prompt_lens", each),
            None if repetition is None else _need(repetition, f32, "repetition", each),
            None if presence is None else _need(presence, f32, "presence", each),
            None if frequency is None else _need(frequency, f32, "frequency", each))
    if history is not None:
        hp, width = _need(history, i32, "history", (rows, None)), history.shape[1]
        if width == 0:  # nothing has come yet
            hp, past = None, (None,) * 5
    biases = 0
    if bias_tokens is not None and bias is not None:
        tp, biases = _need(bias_tokens, i32, "bias_tokens", (rows, None)), bias_tokens.shape[1]
        bp = _need(bias, f32, "bias", (rows, biases))
        if biases == 0:
            tp = bp = None
    elif bias_tokens is not None or bias is not None:
        raise ValueError("bias_tokens and bias belong together")
    masks = words = 0
    if mask is not None:
        mp, (masks, words) = _need(mask, i32, "mask", (None, None)), mask.shape
    _call("qglogits_adjust", logits.data_ptr(), kind, rows, vocab, row, out.data_ptr(), out_kind, out_row, hp, width or 0,
          *past, tp, bp, biases, None if temperature is None else _need(temperature, f32, "temperature", each), mp, words,
          masks, None if mask_rows is None else _need(mask_rows, i32, "mask_rows", each),
          _stream(logits, out, history, lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias,
                  temperature, mask, mask_rows))
    return out


def _logits(t, name):
    """(type, rows, vocab, row stride) of a [rows, vocab] tensor with dense rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise TypeError(f"{name} must be a CUDA tensor [rows, vocab]")
    kind = TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    rows, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"a row of {name} must be dense")
    return kind, rows, vocab, t.stride(0) if rows > 1 else vocab
