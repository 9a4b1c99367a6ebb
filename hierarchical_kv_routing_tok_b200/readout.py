"""Dense readout: attention without the router, as the pages evaluate and generate with it ("dense
readout", pith.science review; gist.science Technical Summary 4: the router is disabled).

``packed_attention`` is causal attention over a packed batch of whole prompts, differentiable;
``PagedKVCache`` holds the K/V of growing sequences in pages that sequences may share, in device
memory together with its integers (page table, lengths, reference counts), so that a decode step
needs no host synchronisation and can be captured into a CUDA graph.  Every computation runs in
``libhga.so``.
"""
from __future__ import annotations

import ctypes

import torch
import torch.autograd.forward_ad as forward_ad

from . import _capi as C
from .api import _need, read_status

_DT = {torch.float32: C.HGA_F32, torch.bfloat16: C.HGA_BF16}
_STEP = {torch.float32: 4, torch.bfloat16: 8}          # elements of 16 bytes
_D = 128

# The checks below read each property of a tensor once, by the cheapest accessor: a decode step's kernel takes
# about as long as a handful of Python calls.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(fn, dev: int, *args) -> None:
    """fn(*args, stream) on the current stream of device dev, which must be the current device meanwhile."""
    if torch._C._cuda_getDevice() == dev:
        fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            fn(*args, _raw_stream(dev))


def _like(t: torch.Tensor, shape) -> torch.Tensor:
    """A new contiguous tensor of t's type and device (of t's own shape: by the cheaper call)."""
    return torch.empty_like(t) if t.is_contiguous() and t.shape == shape else t.new_empty(shape)


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t, contiguous and on a 16-byte boundary."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _flat(t: torch.Tensor, name: str, shape, dtype, dev: int) -> None:
    """t is contiguous, of this shape and type, on CUDA device dev."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        if dev < 0 or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
        _need(t, name, shape, dtype)


def _strides(t: torch.Tensor, name: str, T: int, H: int, dtype, dev: int) -> tuple[int, int]:
    """Element strides of [T, H, 128] for the library: rows of contiguous elements, 16-byte steps."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor" if not t.is_cuda else f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (T, H, _D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H, _D)}")
    st, sh, sd = t.stride()
    if T <= 1:                            # (the stride of a single element means nothing)
        st = H * _D
    if H == 1:
        sh = _D
    step = _STEP[dtype]
    if T and (sd != 1 or st < _D or sh < _D or st % step or sh % step or t.data_ptr() & 15):
        raise ValueError(f"{name}: rows of {_D} contiguous elements at 16-byte steps are needed, got strides "
                         f"{tuple(t.stride())}")
    return st, sh


def _scale(softmax_scale: float | None) -> float:
    """For the library, to which 0 means 1 / sqrt(128)."""
    if softmax_scale is None:
        return 0.0
    if not ctypes.c_float(softmax_scale).value > 0:        # (1e-50 would be 0)
        raise ValueError(f"softmax_scale must be positive (a float32), got {softmax_scale}")
    return float(softmax_scale)


def make_packed_config(q, k, v, cu_seqlens, softmax_scale: float | None = None, flags: int = 0,
                       wait_limit_ns: int = 0) -> C.PackedConfig:
    """Configuration of packed attention from q [total, Hq, 128], k, v [total, Hkv, 128] and cu_seqlens
    [n_seqs + 1] int32; checks the tensors.  q, k and v may be strided (rows contiguous, 16-byte steps)."""
    dtype, dev = q.dtype, q.get_device()
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [total, heads, 128]")
    T, Hq, _ = q.shape
    Hkv = k.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} KV heads")
    qt, qh = _strides(q, "q", T, Hq, dtype, dev)
    kt, kh = _strides(k, "k", T, Hkv, dtype, dev)
    vt, vh = _strides(v, "v", T, Hkv, dtype, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [n_seqs + 1]")
    _flat(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, dev)
    return C.PackedConfig(Hq, Hkv, _D, cu_seqlens.shape[0] - 1, T, qt, qh, kt, kh, vt, vh, _DT[dtype], flags,
                          _scale(softmax_scale), 0, wait_limit_ns)


def _check_packed(cfg, q, k, v, cu_seqlens) -> None:
    """q, k, v and cu_seqlens are what cfg describes."""
    T, dtype, dev = cfg.total, q.dtype, q.get_device()
    if _DT.get(dtype) != cfg.dtype:
        raise ValueError(f"q has dtype {dtype}, which is not the configuration's")
    for t, name, H, st, sh in ((q, "q", cfg.Hq, cfg.q_stride_t, cfg.q_stride_h),
                               (k, "k", cfg.Hkv, cfg.k_stride_t, cfg.k_stride_h),
                               (v, "v", cfg.Hkv, cfg.v_stride_t, cfg.v_stride_h)):
        want, got = (st or H * _D, sh or _D), _strides(t, name, T, H, dtype, dev)
        if (T > 1 and got[0] != want[0]) or (T and H > 1 and got[1] != want[1]):
            raise ValueError(f"{name} has strides {got}, the configuration {want}")
    _flat(cu_seqlens, "cu_seqlens", (cfg.n_seqs + 1,), torch.int32, dev)


def _workspace(cfg, workspace, q, flags: int):
    """The caller's workspace (zeroed once, checked), or a new one whose status the call clears."""
    n = C.packed_workspace_size(cfg)
    if workspace is None:
        return q.new_empty(n, dtype=torch.uint8), flags | C.HGA_PACKED_CLEAR_STATUS
    dev = q.get_device()
    if workspace.get_device() != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.numel() < n:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {n} bytes on cuda:{dev}")
    return workspace, flags


def _with_flags(cfg, flags: int):
    if flags == cfg.flags:
        return cfg
    out = C.PackedConfig.from_buffer_copy(cfg)
    out.flags = flags
    return out


def packed_attn_fwd(cfg, q, k, v, cu_seqlens, o=None, lse=None, workspace=None, o_lo=None):
    """Forward, for a cfg of these tensors' shapes and strides (checked).  Rows of no sequence are left as they
    were in a given o / lse, and hold zeros / -inf in a new one.  o_lo: an output like o for a backward pass in
    bfloat16, what rounding took from o.  workspace: ``new_workspace(cfg, device)``, zeroed once
    (``read_status`` tells of a cu_seqlens that is not valid); without one the call makes its own."""
    _check_packed(cfg, q, k, v, cu_seqlens)
    return _fwd(cfg, q, k, v, cu_seqlens, o, lse, workspace, o_lo)


def _fwd(cfg, q, k, v, cu_seqlens, o=None, lse=None, workspace=None, o_lo=None):
    T, Hq, dev, flags = cfg.total, cfg.Hq, q.get_device(), cfg.flags
    if o is None and lse is None:
        flags |= C.HGA_PACKED_FILL_TAIL
        o = _like(q, (T, Hq, _D))
        lse = q.new_empty((Hq, T), dtype=torch.float32)
    elif o is None or lse is None:
        raise ValueError("o and lse are given together or not at all")
    else:
        _flat(o, "o", (T, Hq, _D), q.dtype, dev)
        _flat(lse, "lse", (Hq, T), torch.float32, dev)
    if o_lo is not None:
        _flat(o_lo, "o_lo", (T, Hq, _D), q.dtype, dev)
    workspace, flags = _workspace(cfg, workspace, q, flags)
    _launch(C.packed_attn_fwd, dev, _with_flags(cfg, flags), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            cu_seqlens.data_ptr(), o.data_ptr(), None if o_lo is None else o_lo.data_ptr(), lse.data_ptr(),
            workspace.data_ptr())
    return o, lse


def packed_attn_bwd(cfg, q, k, v, cu_seqlens, o, lse, d_o, dq=None, dk=None, dv=None, workspace=None, o_lo=None):
    """Gradients (contiguous) for d_o, from the forward's o, lse and, in bfloat16 for the accuracy of short
    sequences, o_lo.  Rows of no sequence: as in ``packed_attn_fwd`` (zeros in new gradients)."""
    _check_packed(cfg, q, k, v, cu_seqlens)
    return _bwd(cfg, q, k, v, cu_seqlens, o, lse, d_o, dq, dk, dv, workspace, o_lo)


def _bwd(cfg, q, k, v, cu_seqlens, o, lse, d_o, dq=None, dk=None, dv=None, workspace=None, o_lo=None):
    T, Hq, Hkv, dev, flags = cfg.total, cfg.Hq, cfg.Hkv, q.get_device(), cfg.flags
    if dq is None and dk is None and dv is None:
        flags |= C.HGA_PACKED_FILL_TAIL
        dq = _like(q, (T, Hq, _D))
        dk = _like(k, (T, Hkv, _D))
        dv = _like(v, (T, Hkv, _D))
    elif dq is None or dk is None or dv is None:
        raise ValueError("dq, dk and dv are given together or not at all")
    else:
        for t, n, h in ((dq, "dq", Hq), (dk, "dk", Hkv), (dv, "dv", Hkv)):
            _flat(t, n, (T, h, _D), q.dtype, dev)
    _flat(o, "o", (T, Hq, _D), q.dtype, dev)
    _flat(d_o, "d_o", (T, Hq, _D), q.dtype, dev)
    _flat(lse, "lse", (Hq, T), torch.float32, dev)
    if o_lo is not None:
        _flat(o_lo, "o_lo", (T, Hq, _D), q.dtype, dev)
    workspace, flags = _workspace(cfg, workspace, q, flags)
    _launch(C.packed_attn_bwd, dev, _with_flags(cfg, flags), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            cu_seqlens.data_ptr(), o.data_ptr(), None if o_lo is None else o_lo.data_ptr(), lse.data_ptr(),
            d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr())
    return dq, dk, dv


_NEW = C.HGA_PACKED_FILL_TAIL | C.HGA_PACKED_CLEAR_STATUS      # of calls with outputs and workspace of their own


def _new_flags(workspace) -> int:
    return _NEW if workspace is None else C.HGA_PACKED_FILL_TAIL      # (a given workspace keeps its status)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, softmax_scale, workspace):
        cfg = make_packed_config(q, k, v, cu_seqlens, softmax_scale, _new_flags(workspace))
        o_lo = _like(q, (cfg.total, cfg.Hq, _D)) if cfg.dtype == C.HGA_BF16 else None
        o, lse = _fwd(cfg, q, k, v, cu_seqlens, workspace=workspace, o_lo=o_lo)
        ctx.softmax_scale, ctx.workspace = softmax_scale, workspace
        ctx.save_for_backward(q, k, v, cu_seqlens, o, lse, o_lo)
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)
        return o, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o, _dlse):
        if d_o is None:
            return None, None, None, None, None, None
        # saved-tensor hooks may hand back tensors of the same values with other strides (save_on_cpu makes the slices of
        # a fused projection dense): the configuration describes what is here, not what the forward had
        q, k, v, cu_seqlens, o, lse, o_lo = ctx.saved_tensors
        cfg = make_packed_config(q, k, v, cu_seqlens, ctx.softmax_scale, _new_flags(ctx.workspace))
        o, lse, d_o = _dense(o), _dense(lse), _dense(d_o)
        o_lo = None if o_lo is None else _dense(o_lo)
        dq, dk, dv = _bwd(cfg, q, k, v, cu_seqlens, o, lse, d_o, workspace=ctx.workspace, o_lo=o_lo)
        return dq, dk, dv, None, None, None


def _check_accumulators(node, dev: int) -> None:
    """The gradient accumulator of a leaf belongs to the stream of the call that made it, for as long as an
    autograd graph holds it: noted at the first call, and compared in a capture."""
    stream = _raw_stream(dev)
    for acc, _ in node.next_functions:
        if acc is not None and acc.name() == _ACCUMULATE \
                and acc.metadata.setdefault("hga_stream", stream) != stream and acc.metadata["hga_stream"] == 0 \
                and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("packed_attention: an autograd graph of q, k or v made on the default stream is still alive; "
                               "its backward pass cannot be captured. Drop its outputs, or make them on the capture's stream")


_ACCUMULATE = "torch::autograd::AccumulateGrad"


def _tangents(*tensors) -> bool:
    """Within a level of forward-mode derivatives: whether one of them carries one, which only an autograd function refuses."""
    return any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


class _NoBackward(torch.autograd.Function):
    """Outputs of a kernel without a backward pass, in the graph of its input: a backward pass through them raises instead of
    leaving their part out."""

    @staticmethod
    def forward(ctx, x, name, fn):
        ctx.name = name
        out = fn(x)
        ctx.mark_non_differentiable(out[1])
        return out

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no backward pass")


def packed_attention(q, k, v, cu_seqlens, softmax_scale: float | None = None, workspace=None):
    """Causal attention over packed sequences: rows cu_seqlens[s] .. cu_seqlens[s+1] - 1 of q [total, Hq,
    128], k, v [total, Hkv, 128] are sequence s (int32, on the device, from 0, not decreasing, at most
    total).  Returns (o [total, Hq, 128], lse [Hq, total] float32); o is differentiable in q, k and v, backward
    and once (forward-mode derivatives are refused: RuntimeError), lse is not.
    Rows of no sequence give zeros and -inf, and zero gradients.

    q, k and v may be strided (slices of a fused projection, transposed head-major tensors); float32 or
    bfloat16.

    A cu_seqlens that is not valid gives zeros, -inf and zero gradients; after a device-side wait that expired, rows
    that were not finished hold anything.  Which of the two happened, if any, ``read_status(workspace)`` tells of a
    workspace that the caller gives (``new_workspace`` of a ``make_packed_config``, or larger): forward and backward
    record there and never clear it.  Calls that may overlap in time need one each.  Without one it goes unseen.

    Forward and backward can be captured into a CUDA graph.  Where q, k or v is a leaf, no autograd graph of it
    that was made on the default stream may be alive then: autograd would make that stream wait for the captured
    one, which the capture does not allow.  Where an earlier call of packed_attention made it, the call is refused
    (RuntimeError); graphs that other operations made of the leaf are not seen here."""
    if (torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad)) \
            or (forward_ad._current_level >= 0 and _tangents(q, k, v)):
        out = _PackedAttention.apply(q, k, v, cu_seqlens, softmax_scale, workspace)
        _check_accumulators(out[0].grad_fn, q.get_device())
        return out
    return _fwd(make_packed_config(q, k, v, cu_seqlens, softmax_scale, _new_flags(workspace)), q, k, v, cu_seqlens,
                workspace=workspace)


class PagedKVCache:
    """K/V of up to max_seqs growing sequences, in pages of a pool, over tensors of the caller:

    k_pool, v_pool [n_layers, n_pages, Hkv, page, 128] (pages contiguous; layers and pages may be strided),
    page_table int32 [max_seqs, max_pages], seq_len int32 [max_seqs], ref_count int32 [n_pages] (the last
    two zero in an empty cache).  ``PagedKVCache.new`` allocates them.

    Every call is asynchronous on the current stream; calls on one cache must not overlap in time (they share its
    workspace).  ``status()`` tells of what they could not do, as HGA_ERR_ARG or HGA_ERR_PAGES of ``_capi``:
    ``reserve``, ``fork``, ``free`` and ``copy_pages`` with a bad entry, or with too few free pages, change nothing;
    ``write`` and ``attend`` leave out the tokens (``attend``: the rows, pages) that a bad entry concerns and do the
    rest; ``compact`` leaves a page id outside the pool, and a row whose length is not valid, as they are and moves the
    other pages, so that such a row may name pages that have moved."""

    def __init__(self, k_pool, v_pool, page_table, seq_len, ref_count, wait_limit_ns: int = 0):
        if k_pool.dtype not in _DT:
            raise ValueError(f"unsupported dtype {k_pool.dtype}")
        if k_pool.dim() != 5 or page_table.dim() != 2:
            raise ValueError("k_pool must be [n_layers, n_pages, Hkv, page, 128], page_table [max_seqs, max_pages]")
        L, P, Hkv, page, D = k_pool.shape
        if tuple(v_pool.shape) != tuple(k_pool.shape) or v_pool.dtype != k_pool.dtype \
                or v_pool.stride() != k_pool.stride():
            raise ValueError("k_pool and v_pool must have one shape, dtype and strides")
        for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if P and L and not t[0, 0].is_contiguous():
                raise ValueError(f"{name}: a page of a layer must be contiguous")
            if (L > 1 and t.stride(0) == 0) or (P > 1 and t.stride(1) == 0):       # (to the library, 0 is contiguous)
                raise ValueError(f"{name}: layers and pages must not share memory, got strides {t.stride()}")
        dev = k_pool.get_device()
        if v_pool.get_device() != dev:
            raise ValueError(f"v_pool is on {v_pool.device}, expected {k_pool.device}")
        _flat(page_table, "page_table", page_table.shape, torch.int32, dev)
        _flat(seq_len, "seq_len", (page_table.shape[0],), torch.int32, dev)
        _flat(ref_count, "ref_count", (P,), torch.int32, dev)
        data = Hkv * page * D
        page_stride = k_pool.stride(1) if P > 1 else data
        layer_stride = k_pool.stride(0) if L > 1 else 0
        self.cfg = C.PagesConfig(L, P, page, Hkv, D, page_table.shape[0], page_table.shape[1], _DT[k_pool.dtype],
                                 layer_stride, page_stride, wait_limit_ns)
        self.k_pool, self.v_pool = k_pool, v_pool
        self.page_table, self.seq_len, self.ref_count = page_table, seq_len, ref_count
        self.device, self.dtype = k_pool.device, k_pool.dtype
        self._dev = dev
        self.workspace = torch.zeros(C.pages_workspace_size(self.cfg), dtype=torch.uint8, device=k_pool.device)
        self._ints = (page_table.data_ptr(), seq_len.data_ptr(), ref_count.data_ptr())
        self._pools = (k_pool.data_ptr(), v_pool.data_ptr())
        self._ws = self.workspace.data_ptr()

    @classmethod
    def new(cls, n_layers: int, n_pages: int, page: int, Hkv: int, max_seqs: int, max_seq_len: int,
            dtype=torch.bfloat16, device="cuda", **kw) -> "PagedKVCache":
        pools = [torch.zeros(n_layers, n_pages, Hkv, page, _D, dtype=dtype, device=device) for _ in range(2)]
        ints = [torch.zeros(s, dtype=torch.int32, device=device)
                for s in ((max_seqs, -(-max_seq_len // page)), (max_seqs,), (n_pages,))]
        return cls(*pools, *ints, **kw)

    def _entries(self, t, name: str, n: int = -1) -> int:
        """An int32 list of n entries (of any number: -1); returns their number."""
        shape = t.shape
        if len(shape) != 1 or (n >= 0 and shape[0] != n):
            raise ValueError(f"{name} has shape {tuple(shape)}, expected ({n if n >= 0 else 'n'},)")
        _flat(t, name, shape, torch.int32, self._dev)
        return shape[0]

    def _layer(self, layer: int) -> int:
        if not 0 <= layer < self.cfg.n_layers:
            raise ValueError(f"layer {layer} of {self.cfg.n_layers}")
        return layer

    def _call(self, fn, *args) -> None:
        _launch(fn, self._dev, self.cfg, *args, self._ws)

    def reserve(self, rows, add) -> torch.Tensor:
        """Room for add[i] tokens behind sequence row rows[i] (int32 [n]): takes the pages, grows seq_len.
        Returns pos [n], the position of each entry's first new token (-1: nothing was changed)."""
        n = self._entries(rows, "rows")
        self._entries(add, "add", n)
        pos = torch.empty_like(rows)
        self._call(C.pages_reserve, n, rows.data_ptr(), add.data_ptr(), pos.data_ptr(), *self._ints)
        return pos

    def write(self, layer: int, k, v, cu_new, rows, pos) -> None:
        """K/V rows of one layer into reserved places: rows cu_new[i] .. cu_new[i+1] - 1 of k, v [total, Hkv,
        128] (may be strided) become the tokens pos[i] .. of sequence row rows[i].  The cache holds values: no
        gradient goes through it."""
        n = self._entries(rows, "rows")
        self._entries(pos, "pos", n)
        self._entries(cu_new, "cu_new", n + 1)
        T, Hkv = k.shape[0], self.cfg.Hkv
        kt, kh = _strides(k, "k", T, Hkv, self.dtype, self._dev)
        vt, vh = _strides(v, "v", T, Hkv, self.dtype, self._dev)
        self._call(C.pages_write, self._layer(layer), n, rows.data_ptr(), pos.data_ptr(), cu_new.data_ptr(), T,
                   k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, *self._ints[:2], *self._pools)

    def attend(self, layer: int, q, rows, softmax_scale: float | None = None, o=None, lse=None):
        """Attention of one new token per sequence: q [n, Hq, 128] (rows may be strided), query i over all
        cached tokens of sequence row rows[i].  Returns (o [n, Hq, 128], lse [n, Hq] float32); an empty row
        gives zeros and -inf.

        For generation: there is no backward pass.  One through a new o, for a q that requires a gradient, raises
        RuntimeError, as a q with a forward-mode derivative does; given outputs hold values only."""
        if (q.requires_grad and o is None and torch.is_grad_enabled()) \
                or (forward_ad._current_level >= 0 and _tangents(q)):
            return _NoBackward.apply(q, "PagedKVCache.attend",
                                     lambda x: self._attend(layer, x, rows, softmax_scale, o, lse))
        return self._attend(layer, q, rows, softmax_scale, o, lse)

    def _attend(self, layer, q, rows, softmax_scale, o, lse):
        n = self._entries(rows, "rows")
        if q.dim() != 3:
            raise ValueError("q must be [n, heads, 128]")
        Hq = q.shape[1]
        sn, sh = _strides(q, "q", n, Hq, self.dtype, self._dev)
        if sh != _D or sn < Hq * _D:
            raise ValueError(f"q: the heads of a token must be contiguous, got strides {tuple(q.stride())}")
        if o is None:
            o = _like(q, (n, Hq, _D))
        else:
            _flat(o, "o", (n, Hq, _D), self.dtype, self._dev)
        if lse is None:
            lse = q.new_empty((n, Hq), dtype=torch.float32)
        else:
            _flat(lse, "lse", (n, Hq), torch.float32, self._dev)
        self._call(C.paged_attn, self._layer(layer), n, Hq, _scale(softmax_scale), rows.data_ptr(),
                   q.data_ptr(), sn, *self._ints[:2], *self._pools, o.data_ptr(), lse.data_ptr())
        return o, lse

    def fork(self, src, dst) -> None:
        """Empty sequence rows dst[i] become copies of rows src[i]: full pages are shared, a begun last page is
        copied in every layer."""
        n = self._entries(src, "src")
        self._entries(dst, "dst", n)
        self._call(C.pages_fork, n, src.data_ptr(), dst.data_ptr(), *self._ints, *self._pools)

    def free(self, rows) -> None:
        """Ends sequences: length 0, and their pages lose a reference."""
        n = self._entries(rows, "rows")
        self._call(C.pages_free, n, rows.data_ptr(), *self._ints)

    def compact(self) -> torch.Tensor:
        """Moves the pages in use to the front of the pool; returns their number (int32 [1], on the device)."""
        n_used = torch.empty(1, dtype=torch.int32, device=self.device)
        self._call(C.pages_compact, *self._ints, *self._pools, n_used.data_ptr())
        return n_used

    def copy_pages(self, src, dst) -> None:
        """Copies the K/V of pages src[i] to pages dst[i] in every layer; table and counts stay."""
        n = self._entries(src, "src")
        self._entries(dst, "dst", n)
        self._call(C.pages_copy, n, src.data_ptr(), dst.data_ptr(), *self._pools)

    def status(self) -> int:
        """Status of the calls since the last one, of those on the current stream and before it (synchronises that
        stream): HGA_OK, HGA_ERR_ARG, HGA_ERR_PAGES or HGA_ERR_TIMEOUT."""
        with torch.cuda.device(self._dev):
            return read_status(self.workspace)
