"""Operators of language models: attention with a sliding window and sinks, per-head norms of queries
and keys with the position rotation, and a paged key/value cache.

The bindings of the second half of include/st_attn.h, same names; they marshal tensors (with their
strides) into the C calls.  As elsewhere in the package there is no CPU path.  Calls are
asynchronous on ``stream`` (default: the current stream of the inputs' device); what they return is
allocated for that stream.

    win = WindowLayout(heads=16, kv_heads=4, window=1024, sinks=16).upload()
    rope = RopeTable(128, scaling="yarn", factor=16, original=8192, device="cuda")
    # training: norm + rotation, attention, both with gradients
    q, k = QKNormRope.apply(q, k, wq, wk, rope)
    o = WindowAttention.apply(q, k, v, win)
    # serving: plan the step, store the new tokens, attend over the pages
    plan = st_paged_plan(lens, new, block_table, free_pages, free_count, page_size, tokens)
    q = st_paged_append(q, k, v, rope, plan.slots, plan.positions, k_pages, v_pages, wq=wq, wk=wk, q_out=buf)
    o, lse = st_paged_decode(q, k_pages, v_pages, block_table, plan.lens, win)

Decode takes one token a request.  A step with more of them (a prompt's chunk) is planned and stored the
same way, but no call attends for a chunk over the pages: its attention takes contiguous keys
(st_window_fwd with q_start).
"""
from __future__ import annotations

import ctypes as _c
import struct as _struct

import torch
from torch.autograd.function import once_differentiable

from . import _abi

_DTYPES = {torch.bfloat16: _abi.ST_BF16, torch.float16: _abi.ST_FP16, torch.float32: _abi.ST_FP32}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class _On:
    """The inputs' device made current for the call, and the stream to launch on.  What a call
    allocates (outputs, workspaces) is allocated inside, so it belongs to that stream too: memory
    that another stream has yet to finish with is not handed out, and a workspace dropped at the end
    of the call is reused behind the kernels that read it."""

    __slots__ = ("guard", "stream")

    def __init__(self, index, stream):
        if stream is None:
            self.guard = None if index == torch._C._cuda_getDevice() else torch.cuda.device(index)
            self.stream = torch._C._cuda_getCurrentRawStream(index)
            return
        device = torch.device("cuda", index)
        if not isinstance(stream, torch.cuda.Stream):
            raw = int(stream)
            stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
        elif stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        self.guard = torch.cuda.stream(stream)
        self.stream = stream.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _dtype(t):
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _strides(name, t, shape, dtype, index):
    """t's strides, for a CUDA tensor of this shape, type and device whose rows are contiguous."""
    s = t.stride()
    if t.shape != shape or t.dtype != dtype or t.get_device() != index or index < 0 or (s and s[-1] != 1 and shape[-1] > 1):
        _refuse(name, t, shape, dtype, index)
    return s


def _refuse(name, t, shape, dtype, index):
    if not t.is_cuda or index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.shape != shape or t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on cuda:{index}, not {tuple(t.shape)} {t.dtype} on {t.device}")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _check_flat(name, t, shape, dtype, index):
    _strides(name, t, shape, dtype, index)
    if len(shape) > 1 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _by_token(s):
    """Strides of [tokens, heads, d] as (batch, head, row)."""
    return 0, s[1], s[0]


class _Packer:
    """Builds a descriptor from a flat list of its fields (several times faster than assigning them)."""

    def __init__(self, cls, fmt):
        self.cls, self.s = cls, _struct.Struct("=" + fmt)
        assert self.s.size == _c.sizeof(cls)

    def __call__(self, *fields):
        return self.cls.from_buffer_copy(self.s.pack(*fields))


_window_fields = _Packer(_abi.st_window_desc_t, "5q2i24q")
_rope_fields = _Packer(_abi.st_rope_desc_t, "7q4i2f18q")
_paged_fields = _Packer(_abi.st_paged_desc_t, "4q2i8q")
_pages_fields = _Packer(_abi.st_pages_t, "8q")
_strides_fields = _Packer(_abi.st_strides_t, "3q")
_NO_STRIDES = (0, 0, 0)


def _p(t):
    return None if t is None else t.data_ptr()


def _workspace(ws, need, like):
    if ws is None:
        return like.new_empty(need, dtype=torch.uint8) if need else None
    if ws.get_device() != like.get_device() or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    return ws


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# ---- sliding-window attention -----------------------------------------------------------------
class WindowLayout:
    """Owner of an st_window_t: query position p sees the keys j <= p with j > p - window (0: no
    limit) or j < sinks; head h reads key head h // (heads // kv_heads).  A captured graph of its calls
    does not keep it alive: hold it as long as the graph."""

    def __init__(self, heads: int, kv_heads: int, window: int, sinks: int = 0):
        self._lib = _abi.load()
        self._h = _c.c_void_p()
        _abi.check(self._lib.st_window_create(heads, kv_heads, window, sinks, _c.byref(self._h)), "st_window_create")
        self.heads, self.kv_heads, self.window, self.sinks = heads, kv_heads, window, sinks

    @property
    def handle(self):
        return self._h

    def upload(self, device=None, stream=None) -> "WindowLayout":
        """Bind to ``device`` (default: the current one)."""
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with _On(device.index, stream) as s:
            _abi.check(self._lib.st_window_upload(self._h, s), "st_window_upload")
        self.device = device
        return self

    def check(self, stream=None) -> None:
        """Synchronise and raise StError for a device wait that ran out (ST_ERR_DEVICE_TIMEOUT) or a
        page outside the cache (ST_ERR_BAD_PAGE) since the last check."""
        device = getattr(self, "device", None)
        with _On(torch.cuda.current_device() if device is None else device.index, stream) as s:
            _abi.check(self._lib.st_window_check(self._h, s), "st_window_check")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.st_window_destroy(h)
            h.value = None


def _window_call(q, k, v, layout, q_start, lens):
    """What a call's tensors agree on: device index, the leading fields of the descriptor, and the
    strides of q, k and v."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected [batch, heads, n, d] tensors")
    B, H, nq, d = q.shape
    nk = k.shape[2]
    index, dtype = q.get_device(), q.dtype
    kshape = (B, layout.kv_heads, nk, d)
    strides = (_strides("q", q, (B, layout.heads, nq, d), dtype, index)[:3] + _strides("k", k, kshape, dtype, index)[:3] +
               _strides("v", v, kshape, dtype, index)[:3])
    if lens is not None:
        _check_flat("lens", lens, (B,), torch.int32, index)
    if q_start is None:
        q_start = nk - nq
        if q_start < 0:
            raise ValueError("more queries than keys: give q_start")
    return index, (B, nq, nk, d, q_start, _dtype(q), 0), strides


def st_window_fwd(q, k, v, layout: WindowLayout, q_start=None, lens=None, o=None, lse=None, stream=None, check=False):
    """O [B, H, nq, d] and lse [B, H, nq] (fp32, natural log) of sliding-window attention.

    q: [B, H, nq, d]; k, v: [B, KV, nk, d] (bf16 or fp16, d 64 or 128, any strides with contiguous
    rows).  Row i stands at position q_start + i (default: the last nq of nk).  lens: int32 [B]
    lengths of a padded batch; rows and keys at lens[b] and beyond are padding (O = 0, lse = -inf).  A
    row that sees a score of NaN or +inf gets NaN in O and lse.
    Asynchronous: ``layout.check()`` or ``check=True`` reports a device wait that ran out."""
    index, head, strides = _window_call(q, k, v, layout, q_start, lens)
    with _On(index, stream) as s:
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = q.new_empty(q.shape[:3], dtype=torch.float32)
        else:
            _check_flat("lse", lse, q.shape[:3], torch.float32, index)
        desc = _window_fields(*head, *strides, *_strides("o", o, q.shape, q.dtype, index)[:3], *_NO_STRIDES * 4)
        _abi.check(layout._lib.st_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lens), layout._h, o.data_ptr(),
                                             lse.data_ptr(), _c.byref(desc), s), "st_window_fwd")
    if check:
        layout.check(stream)
    return o, lse


def st_window_bwd_workspace_bytes(q, k, layout: WindowLayout, q_start=None) -> int:
    index, head, strides = _window_call(q, k, k, layout, q_start, None)
    desc = _window_fields(*head, *strides, *_NO_STRIDES * 5)
    with _On(index, None):
        return int(layout._lib.st_window_bwd_workspace_bytes(_c.byref(desc), layout.handle))


def st_window_bwd(q, k, v, o, lse, do, layout: WindowLayout, q_start=None, lens=None, dq=None, dk=None, dv=None,
                  workspace=None, stream=None, check=False):
    """dQ, dK, dV of st_window_fwd (recomputing P from the saved lse); deterministic."""
    index, head, strides = _window_call(q, k, v, layout, q_start, lens)
    with _On(index, stream) as s:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        for name, t, like in (("o", o, q), ("do", do, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            strides += _strides(name, t, like.shape, q.dtype, index)[:3]
        _check_flat("lse", lse, q.shape[:3], torch.float32, index)
        desc = _window_fields(*head, *strides)
        if workspace is None:
            need = layout._lib.st_window_bwd_workspace_bytes(_c.byref(desc), layout._h)
        workspace = _workspace(workspace, need if workspace is None else 0, q)
        _abi.check(layout._lib.st_window_bwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(do), _p(lens), layout._h,
                                             _p(dq), _p(dk), _p(dv), _p(workspace), _nbytes(workspace),
                                             _c.byref(desc), s), "st_window_bwd")
    if check:
        layout.check(stream)
    return dq, dk, dv


def _as_rows(t):
    """A gradient as the kernels read it: contiguous rows on 16-byte boundaries (an expanded one, as of
    a sum, has strides of 0)."""
    es = t.element_size()
    ok = t.data_ptr() % 16 == 0 and t.stride(-1) == 1 and all(
        t.shape[i] == 1 or (t.stride(i) >= t.shape[-1] and t.stride(i) * es % 16 == 0) for i in range(t.dim() - 1))
    return t if ok else t.clone(memory_format=torch.contiguous_format)  # (contiguous() keeps a slice off a boundary)


class WindowAttention(torch.autograd.Function):
    """Autograd wrapper: apply(q, k, v, layout, lens=None, q_start=None) -> o.

    To capture a training step into a CUDA graph, hold no autograd graph of the same leaves from
    outside the capture while it runs (PyTorch would wait across the capture's streams); calls of
    st_window_fwd and st_window_bwd themselves may be captured at any time."""

    @staticmethod
    def forward(ctx, q, k, v, layout, lens=None, q_start=None):
        o, lse = st_window_fwd(q, k, v, layout, q_start=q_start, lens=lens)
        ctx.save_for_backward(q, k, v, o, lse, lens)
        ctx.layout, ctx.q_start = layout, q_start
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, lens = ctx.saved_tensors
        dq, dk, dv = st_window_bwd(q, k, v, o, lse, _as_rows(do), ctx.layout, q_start=ctx.q_start, lens=lens)
        return dq, dk, dv, None, None, None


# ---- norm and rotation ------------------------------------------------------------------------
class RopeTable:
    """Rotation speeds of the first ``rot`` elements of a head (made once per model).

    scaling: "none", "linear", "ntk" or "yarn", by ``factor`` for contexts that many times the
    ``original`` one (st_rope_turns gives the formulas); interleaved: pairs (2i, 2i + 1), else
    (i, i + rot / 2)."""

    def __init__(self, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original: float = 8192, interleaved: bool = False, device="cuda"):
        if scaling not in _SCALINGS:
            raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(_SCALINGS)}")
        turns = torch.empty(max(rot // 2, 1), dtype=torch.int64, device="cpu")  # 2^-64 turns per position
        mscale = _c.c_float()
        _abi.check(_abi.load().st_rope_turns(rot, base, _SCALINGS[scaling], factor, original, turns.data_ptr(),
                                             _c.byref(mscale)), "st_rope_turns")
        self.rot, self.interleaved, self.mscale = rot, bool(interleaved), mscale.value
        self.turns = turns.to(device)


def _rope_call(q, k, rope, wq, wk, eps, positions, start, token_major):
    """q, k: [B, H, n, d] and [B, KV, n, d], or packed [n, H, d] and [n, KV, d] (token_major).  Returns
    the device index, the leading fields of the descriptor, and the strides of q and k."""
    if q.dim() != (3 if token_major else 4) or k.dim() != q.dim():
        raise ValueError("expected [tokens, heads, d] tensors" if token_major else "expected [batch, heads, n, d] tensors")
    index, dtype = q.get_device(), q.dtype
    if token_major:
        (n, H, d), B, KV = q.shape, 1, k.shape[1]
        kshape = (n, KV, d)
    else:
        (B, H, n, d), KV = q.shape, k.shape[1]
        kshape = (B, KV, n, d)
    qs, ks = _strides("q", q, q.shape, dtype, index), _strides("k", k, kshape, dtype, index)
    if (wq is None) != (wk is None):
        raise ValueError("give both norm weights or neither")
    wdt = _dtype(q)
    if wq is not None:
        for name, w in (("wq", wq), ("wk", wk)):
            _check_flat(name, w, (d,), wq.dtype, index)
        if wq.dtype not in (torch.float32, dtype):
            raise TypeError("norm weights must be fp32 or of the queries' type")
        wdt = _dtype(wq)
    if rope.turns.get_device() != index:
        raise ValueError("the rotation table is on another device")
    pos_batch = 0
    if positions is not None:
        shape = (n,) if positions.dim() == 1 else (B, n)
        _check_flat("positions", positions, shape, torch.int32, index)
        pos_batch = n if positions.dim() == 2 else 0
    head = (B, H, KV, n, d, start, pos_batch, rope.rot, int(rope.interleaved), _dtype(q), wdt, eps, rope.mscale)
    return index, head, (_by_token(qs) + _by_token(ks) if token_major else qs[:3] + ks[:3])


def st_qk_norm_rope(q, k, rope: RopeTable, wq=None, wk=None, eps: float = 1e-6, positions=None, start: int = 0,
                    q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q [B, H, n, d] and k [B, KV, n, d] (weights [d], or no norm) and their
    rotation, in one pass; returns (q_out, k_out), contiguous unless given (q_out may be q).
    Positions are positions ([n] or [B, n] int32), or start, start + 1, ..."""
    index, head, strides = _rope_call(q, k, rope, wq, wk, eps, positions, start, False)
    with _On(index, stream) as s:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format) if q_out is None else q_out
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format) if k_out is None else k_out
        desc = _rope_fields(*head, *strides, *_strides("q_out", q_out, q.shape, q.dtype, index)[:3],
                            *_strides("k_out", k_out, k.shape, q.dtype, index)[:3], *_NO_STRIDES * 2)
        _abi.check(_abi.load().st_qk_norm_rope(_p(q), _p(k), _p(wq), _p(wk), _p(rope.turns), _p(positions), _p(q_out),
                                               _p(k_out), _c.byref(desc), s), "st_qk_norm_rope")
    return q_out, k_out


def st_qk_norm_rope_bwd_workspace_bytes(q, k, rope: RopeTable) -> int:
    index, head, strides = _rope_call(q, k, rope, None, None, 0.0, None, 0, False)
    desc = _rope_fields(*head, *strides, *_NO_STRIDES * 4)
    with _On(index, None):
        return int(_abi.load().st_qk_norm_rope_bwd_workspace_bytes(_c.byref(desc)))


def st_qk_norm_rope_bwd(q, k, gq, gk, rope: RopeTable, wq=None, wk=None, eps: float = 1e-6, positions=None,
                        start: int = 0, dq=None, dk=None, workspace=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) for the output gradients gq, gk; dwq and dwk are fp32, or None
    without weights.  dq may be gq and dk may be gk."""
    index, head, strides = _rope_call(q, k, rope, wq, wk, eps, positions, start, False)
    lib = _abi.load()
    dwq = dwk = None
    with _On(index, stream) as s:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        for name, t, like in (("gq", gq, q), ("gk", gk, k), ("dq", dq, q), ("dk", dk, k)):
            strides += _strides(name, t, like.shape, q.dtype, index)[:3]
        desc = _rope_fields(*head, *strides)
        if wq is not None:
            dwq, dwk = q.new_empty((2, q.shape[-1]), dtype=torch.float32).unbind()
            if workspace is None:
                need = lib.st_qk_norm_rope_bwd_workspace_bytes(_c.byref(desc))
            workspace = _workspace(workspace, need if workspace is None else 0, q)
        _abi.check(lib.st_qk_norm_rope_bwd(_p(q), _p(k), _p(gq), _p(gk), _p(wq), _p(wk), _p(rope.turns),
                                           _p(positions), _p(dq), _p(dk), _p(dwq), _p(dwk), _p(workspace),
                                           _nbytes(workspace), _c.byref(desc), s), "st_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


class QKNormRope(torch.autograd.Function):
    """Autograd wrapper: apply(q, k, wq, wk, rope, eps=1e-6, positions=None, start=0) -> (q, k).
    Under CUDA graph capture the note of WindowAttention holds."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, rope, eps=1e-6, positions=None, start=0):
        ctx.save_for_backward(q, k, wq, wk, positions)
        ctx.rope, ctx.eps, ctx.start = rope, eps, start
        return st_qk_norm_rope(q, k, rope, wq=wq, wk=wk, eps=eps, positions=positions, start=start)

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        q, k, wq, wk, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = st_qk_norm_rope_bwd(q, k, _as_rows(gq), _as_rows(gk), ctx.rope, wq=wq, wk=wk, eps=ctx.eps,
                                               positions=positions, start=ctx.start)
        if wq is not None:
            dwq, dwk = dwq.to(wq.dtype), dwk.to(wk.dtype)
        return dq, dk, dwq, dwk, None, None, None, None


# ---- paged cache ------------------------------------------------------------------------------
class PagedPlan:
    """Outputs of st_paged_plan for up to ``tokens`` new tokens of ``requests`` requests, all int32:
    lens [requests], free_left [1], offsets [requests + 1], slots and positions [tokens], status
    [requests].  A program may keep one and plan into it every step; outputs may not be inputs, so lens
    and free_left are copied into the program's own (lens.copy_(plan.lens)) before the next one."""

    def __init__(self, requests: int, tokens: int, device="cuda"):
        self.requests, self.tokens = requests, tokens
        sizes = (requests, 1, requests + 1, tokens, tokens, requests)
        at = [0]
        for n in sizes:
            at.append(at[-1] + (n + 63) // 64 * 64)
        buf = torch.empty(at[-1], dtype=torch.int32, device=device)
        self.device = buf.device
        (self.lens, self.free_left, self.offsets, self.slots, self.positions,
         self.status) = (buf[a:a + n] for a, n in zip(at, sizes))


def st_paged_plan(lens, new, block_table, free_pages, free_count, page_size: int, tokens: int, plan: PagedPlan = None,
                  stream=None) -> PagedPlan:
    """Plan a serving step on the device: lens, new [requests], block_table [requests, max_pages]
    (newly taken pages are written in place), free_pages [*] with free_count [1] of them free, all
    int32; free_pages may be empty.  ``tokens`` is the room for new tokens; entries past the last one are
    -1."""
    if lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("expected lens [requests], block_table [requests, max_pages] and free_pages [*]")
    R, index, i32 = lens.shape[0], lens.get_device(), torch.int32
    _check_flat("lens", lens, (R,), i32, index)
    _check_flat("new", new, (R,), i32, index)
    max_pages, capacity = block_table.shape[1], free_pages.shape[0]
    table_stride = _strides("block_table", block_table, (R, max_pages), i32, index)[0]
    _check_flat("free_pages", free_pages, (capacity,), i32, index)
    _check_flat("free_count", free_count, (1,), i32, index)
    desc = _abi.st_plan_desc_t(R, tokens, max_pages, table_stride, page_size, capacity)
    with _On(index, stream) as s:
        if plan is None:
            plan = PagedPlan(R, tokens, lens.device)
        elif plan.requests != R or plan.tokens != tokens or plan.lens.get_device() != index:
            raise ValueError("plan was made for other sizes or another device")
        _abi.check(_abi.load().st_paged_plan(_p(lens), _p(new), _p(block_table), _p(free_pages), _p(free_count),
                                             _p(plan.lens), _p(plan.free_left), _p(plan.offsets), _p(plan.slots),
                                             _p(plan.positions), _p(plan.status), _c.byref(desc), s), "st_paged_plan")
    return plan


def _pages(k_pages, v_pages, kv, d, dtype, index):
    """Fields of st_pages_t."""
    if k_pages.dim() != 4:
        raise ValueError("pages must be [num_pages, kv_heads, page_size, d]")
    P, ps = k_pages.shape[0], k_pages.shape[2]
    shape = (P, kv, ps, d)
    return (P, ps) + _strides("k_pages", k_pages, shape, dtype, index)[:3] + _strides("v_pages", v_pages, shape, dtype, index)[:3]


def st_paged_append(q, k, v, rope: RopeTable, slots, positions, k_pages, v_pages, wq=None, wk=None, eps: float = 1e-6,
                    q_out=None, stream=None):
    """New tokens into the cache: q [tokens, H, d] is normed and rotated into q_out, k [tokens, KV, d]
    likewise into its slot of k_pages, v into v_pages ([num_pages, KV, page_size, d] each).  Tokens
    with slot -1 are skipped: their rows of q_out stay as they were.  A q_out made here has them 0, which
    costs a pass over it (8192 tokens of 32 heads, bf16: 61 us instead of 43); q_out may be q."""
    index, head, strides = _rope_call(q, k, rope, wq, wk, eps, positions, 0, True)
    n, KV, d = k.shape
    vs = _strides_fields(*_by_token(_strides("v", v, k.shape, q.dtype, index)))
    _check_flat("slots", slots, (n,), torch.int32, index)
    if positions is None or positions.dim() != 1:
        raise ValueError("positions must be [tokens]")
    pages = _pages_fields(*_pages(k_pages, v_pages, KV, d, q.dtype, index))
    with _On(index, stream) as s:
        q_out = torch.zeros_like(q, memory_format=torch.contiguous_format) if q_out is None else q_out
        qo = _by_token(_strides("q_out", q_out, q.shape, q.dtype, index))
        desc = _rope_fields(*head, *strides, *qo, *_NO_STRIDES * 3)
        _abi.check(_abi.load().st_paged_append(_p(q), _p(k), _p(v), _p(wq), _p(wk), _p(rope.turns), _p(positions),
                                               _p(slots), _p(q_out), _p(k_pages), _p(v_pages), _c.byref(vs),
                                               _c.byref(pages), _c.byref(desc), s), "st_paged_append")
    return q_out


def st_paged_decode_workspace_bytes(q, layout: WindowLayout) -> int:
    """Bytes for any decode call of q's shape [requests, H, d] with this layout."""
    d = q.shape[2]
    desc = _paged_fields(q.shape[0], d, 1, 1, _dtype(q), 0, 1, 16, 0, d, d, 0, d, d)
    with _On(q.get_device(), None):
        return int(layout._lib.st_paged_decode_workspace_bytes(_c.byref(desc), layout.handle))


def st_paged_decode(q, k_pages, v_pages, block_table, lens, layout: WindowLayout, o=None, lse=None, workspace=None,
                    stream=None, check=False):
    """One new token per request over its pages: q [requests, H, d] at position lens - 1 against the
    keys of block_table [requests, max_pages] (int32), behind the layout's window and sinks.  Returns
    o [requests, H, d] and lse [requests, H]; a request of length 0 gets O = 0, lse = -inf.  For the
    product with the values the probabilities are rounded to q's type; in bf16 and for up to 8 heads a
    key head they keep 16 bits.  Asynchronous: ``layout.check()`` or ``check=True`` reports a page outside the cache."""
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("expected q [requests, heads, d] and block_table [requests, max_pages]")
    R, H, d = q.shape
    index, dtype = q.get_device(), q.dtype
    _check_flat("q", q, (R, layout.heads, d), dtype, index)
    pages = _pages(k_pages, v_pages, layout.kv_heads, d, dtype, index)
    max_pages = block_table.shape[1]
    table_stride = _strides("block_table", block_table, (R, max_pages), torch.int32, index)[0]
    _check_flat("lens", lens, (R,), torch.int32, index)
    desc = _paged_fields(R, d, max_pages, table_stride, _dtype(q), 0, *pages)
    with _On(index, stream) as s:
        if o is None:
            o = torch.empty_like(q)
        else:
            _check_flat("o", o, q.shape, dtype, index)
        if lse is None:
            lse = q.new_empty((R, H), dtype=torch.float32)
        else:
            _check_flat("lse", lse, (R, H), torch.float32, index)
        if workspace is None:
            need = layout._lib.st_paged_decode_workspace_bytes(_c.byref(desc), layout._h)
        workspace = _workspace(workspace, need if workspace is None else 0, q)
        _abi.check(layout._lib.st_paged_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                               lens.data_ptr(), layout._h, o.data_ptr(), lse.data_ptr(), _p(workspace),
                                               _nbytes(workspace), _c.byref(desc), s), "st_paged_decode")
    if check:
        layout.check(stream)
    return o, lse
