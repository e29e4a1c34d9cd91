"""The layer operators of libmuon.so (include/muon.h): 8-bit activation
checkpoints, the norm sites between blocks, and the weight gradients that the
optimizer step reads.

    site = layer.NormSite(branch, residual, w_pre, w_post=w, gate=g)
    site.forward()                          # site.y, site.h; checkpoints site.u, site.v
    ...                                     # the linear layer and what follows, on site.h
    site.backward(dy, dh)                   # site.d_residual, site.d_branch, site.d_w_pre, ...
    layer.WGrad([(dY, site.u, G, w_pre)]).run()   # G = dY^T (u * w_pre), for muon.Plan

Like the optimizer's plans, ``NormSite`` and ``WGrad`` take their tensors once
and keep them referenced; every call after that only launches kernels, on the
current stream or the one it is given (a torch stream or a raw handle). They may
be dropped while a stream still works on their buffers. Each has one set of
buffers: calls on two streams need an order between them, as any two writers of
a tensor do. Tensors are 2-D (weights 1-D) device tensors with unit column
stride, on the current device. There is no CPU fallback.
"""

from __future__ import annotations

import ctypes
from typing import Iterable, List, Optional, Sequence

import torch

from .muon import (MUON_BF16, MUON_F32, MuonError, check, lib, muon_norm_grads, muon_norm_site, muon_q8,
                   muon_wgrad_item)

GROUP = 32
KINDS = {"int8": 0, "e4m3": 1}
_CODES = {torch.bfloat16: MUON_BF16, torch.float32: MUON_F32}


def _bad(message: str):
    raise MuonError(-1, message)


def _kind(kind: str) -> int:
    if kind not in KINDS:
        raise MuonError(-4, f"kind must be one of {sorted(KINDS)}, not {kind!r}")
    return KINDS[kind]


def _code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise MuonError(-4, f"unsupported tensor dtype {t.dtype}")
    return code


def _matrix(t, name: str, shape=None, dtype=None, vector=False):
    """Checks one tensor of a call: where it is, its layout, shape and type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad(f"{name} must be a device tensor")
    if t.get_device() != torch.cuda.current_device():
        _bad(f"{name} is on {t.device}, not on the current device")
    size = t.shape
    if len(size) != (1 if vector else 2) or (t.stride(-1) != 1 and size[-1] > 1 and t.numel()):
        _bad(f"{name} must be a {1 if vector else 2}-D tensor with unit column stride")
    if shape is not None and size != shape:
        _bad(f"{name} must have shape {tuple(shape)}, not {tuple(size)}")
    if dtype is not None and t.dtype != dtype:
        _bad(f"{name} must be {dtype}, not {t.dtype}")
    return t


def _ld(t) -> int:
    """Row stride in elements; of one row or none, any will do."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _current_handle() -> int:
    """The current stream's handle: making a Stream object of it takes 3 us."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


class _Streams:
    """The streams that use a set of tensors, made on or ready for the stream
    that is current now. The tensors' memory is kept from reuse until every other
    stream that ever used it is done with it; that takes one record per tensor
    and stream, made when a stream comes up first."""

    def __init__(self, tensors: Iterable):
        self._tensors = tuple(tensors)
        self._seen = {_current_handle()}

    def use(self, stream, call: Sequence = ()) -> int:
        """The handle of the stream to launch on (None: the current one). Tensors
        of this call alone are recorded if the call names a stream that is not
        the current one: with the current one they are the caller's to keep, as
        with any torch operation."""
        now = _current_handle()
        handle = now if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        self.add(stream, handle)
        if handle != now:
            self._record(stream, call)
        return handle

    def add(self, stream, handle: int) -> None:
        """The stream, of this handle, uses the tensors from now on."""
        if handle not in self._seen:
            self._record(stream, self._tensors)
            self._seen.add(handle)

    @staticmethod
    def _record(stream, tensors) -> None:
        stream = torch.cuda.current_stream() if stream is None else _stream_object(stream)
        for t in tensors:
            t.record_stream(stream)  # nothing to do on the stream that the memory was made on


def _stream_object(stream):
    if hasattr(stream, "cuda_stream"):
        return stream
    # torch makes a stream of its own out of the handle 0, which is the default stream's
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class Q8:
    """An 8-bit checkpoint of a rows x cols matrix: bytes ``q`` (rows x a
    multiple of 16) and exponent bytes ``e`` (rows x ceil(cols / 32)), in
    groups of 32 columns. Given ``q`` and ``e`` (uint8 device tensors), it is a
    view of them; otherwise it allocates them."""

    def __init__(self, rows: int, cols: int, kind: str = "int8", *, q=None, e=None):
        if rows < 0 or cols < 1:
            _bad("a checkpoint needs rows >= 0 and cols >= 1")
        self.rows, self.cols, self.kind = int(rows), int(cols), kind
        code = _kind(kind)
        if (q is None) != (e is None):
            _bad("q and e go together")
        if q is None:
            dev = torch.device("cuda", torch.cuda.current_device())
            q = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=dev)
            e = torch.empty(rows, -(-cols // GROUP), dtype=torch.uint8, device=dev)
        _matrix(q, "q", dtype=torch.uint8)
        _matrix(e, "e", dtype=torch.uint8)
        if q.shape[0] != rows or e.shape[0] != rows:
            _bad("q and e must have one row per row of the checkpoint")
        if q.shape[1] < -(-cols // 16) * 16 or e.shape[1] < -(-cols // GROUP):
            _bad("q needs cols rounded up to a multiple of 16, e one byte per 32 columns")
        self.q, self.e = q, e
        self._streams = _Streams((q, e))
        ldq = _ld(q) if rows > 1 else -(-q.shape[1] // 16) * 16
        self._c = muon_q8(q.data_ptr(), e.data_ptr(), rows, cols, ldq, _ld(e), code, 0)

    def nbytes(self) -> int:
        return self.q.numel() + self.e.numel()


def q8_save(x, out: Q8, stream=None) -> Q8:
    """Saves x (bf16 or fp32) into the checkpoint ``out``."""
    _matrix(x, "x", (out.rows, out.cols))
    check(lib().muon_q8_save(x.data_ptr(), _ld(x), _code(x), ctypes.byref(out._c),
                             out._streams.use(stream, (x,))))
    return out


def q8_load(ckpt: Q8, out, stream=None):
    """Writes the values that the checkpoint stands for into ``out`` (bf16, which
    holds them exactly, or fp32)."""
    _matrix(out, "out", (ckpt.rows, ckpt.cols))
    check(lib().muon_q8_load(ctypes.byref(ckpt._c), out.data_ptr(), _ld(out), _code(out),
                             ckpt._streams.use(stream, (out,))))
    return out


class NormSite:
    """The norms after one block and before the next, with the gate and the
    residual scales between them (muon_norm_site):

        v = branch / rms(branch)        (branch itself without w_post)
        y = res_scale * residual + branch_scale * gate * w_post * v
        u = y / rms(y),   h = w_pre * u

    ``branch`` and ``residual`` are rows x cols, bf16 or fp32; the weights have
    their type. ``gate`` is None, one row (cols) or one per token (rows x cols).
    With a ``kind`` ("int8" or "e4m3") the forward pass keeps what the backward
    pass needs: checkpoints ``u`` and ``v`` and the norms ``rstd_y`` and
    ``rstd_b``; with None it keeps nothing. ``saved``: (u, v, rstd_y, rstd_b)
    to use in place of new buffers (v and rstd_b None where they are not
    needed).

    ``forward()`` writes ``y`` and ``h``. ``backward(dy, dh)`` writes
    ``d_residual``, ``d_branch``, ``d_w_pre``, ``d_w_post`` and ``d_gate``
    (None where the site has no such weight); these are allocated at its first
    call and reused. dy may be None: no gradient but through h."""

    def __init__(self, branch, residual, w_pre, *, w_post=None, gate=None, res_scale: float = 1.0,
                 branch_scale: float = 1.0, eps: float = 1e-6, kind: Optional[str] = "int8", saved=None):
        _matrix(branch, "branch")
        code, dt = _code(branch), branch.dtype
        rows, cols = branch.shape
        _matrix(residual, "residual", (rows, cols), dt)
        _matrix(w_pre, "w_pre", (cols,), dt, vector=True)
        if w_post is not None:
            _matrix(w_post, "w_post", (cols,), dt, vector=True)
        if gate is not None:
            vector = gate.dim() == 1
            _matrix(gate, "gate", (cols,) if vector else (rows, cols), dt, vector=vector)
            if not vector and _ld(gate) < cols:  # 0 would tell muon_norm_site that all rows share one gate
                _bad("gate's rows overlap; a gate that all rows share is 1-D")
        self.branch, self.residual, self.w_pre, self.w_post, self.gate = branch, residual, w_pre, w_post, gate
        self.y, self.h = torch.empty_like(branch, memory_format=torch.contiguous_format), \
            torch.empty_like(branch, memory_format=torch.contiguous_format)
        self.u = self.v = self.rstd_y = self.rstd_b = None
        if saved is not None:
            self.u, self.v, self.rstd_y, self.rstd_b = saved
        elif kind is not None:
            self.u = Q8(rows, cols, kind)
            self.rstd_y = torch.empty(rows, device=branch.device)
            if w_post is not None or gate is not None:
                self.v = Q8(rows, cols, kind)
            if w_post is not None:
                self.rstd_b = torch.empty(rows, device=branch.device)
        for t, name in ((self.rstd_y, "rstd_y"), (self.rstd_b, "rstd_b")):
            if t is not None:
                _matrix(t, name, (rows,), torch.float32, vector=True)
        self.d_residual = self.d_branch = self.d_w_pre = self.d_w_post = self.d_gate = None
        self._grads = self._workspace = self._grad_streams = None
        none = muon_q8()
        self._c = muon_norm_site(
            rows, cols, branch.data_ptr(), _ld(branch), residual.data_ptr(), _ld(residual), w_pre.data_ptr(),
            _ptr(w_post), _ptr(gate), _ld(gate) if gate is not None and gate.dim() == 2 else 0,
            self.y.data_ptr(), cols, self.h.data_ptr(), cols, _ptr(self.rstd_y), _ptr(self.rstd_b),
            self.u._c if self.u is not None else none, self.v._c if self.v is not None else none,
            res_scale, branch_scale, eps, code)
        self._streams = _Streams([t for t in (branch, residual, w_pre, w_post, gate, self.y, self.h, self.rstd_y, self.rstd_b)
                                  if t is not None] + [t for q in (self.u, self.v) if q is not None for t in (q.q, q.e)])

    def forward(self, stream=None) -> None:
        check(lib().muon_norm_forward(ctypes.byref(self._c), self._streams.use(stream)))

    def backward(self, dy, dh, stream=None) -> None:
        shape, dt = tuple(self.y.shape), self.y.dtype
        if self.u is None or self.rstd_y is None:
            _bad("the site keeps no checkpoints: make it with a kind")
        if dy is not None:
            _matrix(dy, "dy", shape, dt)
        _matrix(dh, "dh", shape, dt)
        if self._grads is None:
            # new memory belongs to the stream that uses it first
            with torch.cuda.stream(None if stream is None else _stream_object(stream)):
                self._make_grads()
        g = self._grads
        g.dy, g.ld_dy, g.dh, g.ld_dh = _ptr(dy), 0 if dy is None else _ld(dy), dh.data_ptr(), _ld(dh)
        handle = self._streams.use(stream, (dh,) if dy is None else (dy, dh))
        self._grad_streams.add(stream, handle)
        check(lib().muon_norm_backward(ctypes.byref(self._c), ctypes.byref(g), handle))

    def _make_grads(self) -> None:
        shape, dt = tuple(self.y.shape), self.y.dtype
        empty = lambda t: None if t is None else torch.empty(t.shape, dtype=dt, device=t.device)  # noqa: E731
        self.d_residual, self.d_branch = empty(self.y), empty(self.y)
        self.d_w_pre, self.d_w_post, self.d_gate = empty(self.w_pre), empty(self.w_post), empty(self.gate)
        need = ctypes.c_size_t()
        check(lib().muon_norm_backward_workspace(shape[0], shape[1], ctypes.byref(need)))
        self._workspace = torch.empty(need.value, dtype=torch.uint8, device=self.y.device)
        self._grads = muon_norm_grads(
            None, 0, None, 0, self.d_residual.data_ptr(), shape[1], self.d_branch.data_ptr(), shape[1],
            _ptr(self.d_w_pre), _ptr(self.d_w_post), _ptr(self.d_gate), shape[1], self._workspace.data_ptr(), need.value)
        self._grad_streams = _Streams([t for t in (self.d_residual, self.d_branch, self.d_w_pre, self.d_w_post, self.d_gate,
                                                   self._workspace) if t is not None])


class WGrad:
    """Weight gradients of linear layers, all in one go (muon_wgrad). Every
    item is ``(dY, ckpt, G[, scale[, beta[, C]]])``:

        G = dY^T (X * scale) + beta * C

    dY is rows x n (bf16 or fp32, the same for every item), ckpt a ``Q8`` of
    the layer's input X (rows x k, one kind for every item), G n x k (contiguous,
    bf16 or fp32: what ``muon.Plan`` takes), scale None or k elements of dY's
    type, C like G (default: G itself, to accumulate)."""

    def __init__(self, items: Iterable[Sequence]):
        tensors: List = []
        descs = []
        self._dtype = self._gdtype = None
        dts = None
        for item in items:
            dY, x, G = item[:3]
            scale, beta, C = (list(item[3:]) + [None, 0.0, None][len(item) - 3:])[:3]
            if not isinstance(x, Q8):
                _bad("the second entry of an item must be a Q8 checkpoint")
            if dts is None:
                self._dtype, self._gdtype, dts = _code(dY), _code(G), (dY.dtype, G.dtype)
            _matrix(G, "G", dtype=dts[1])
            if not G.is_contiguous():
                _bad("G must be contiguous")
            n, k = G.shape
            if k != x.cols:
                _bad(f"G has {k} columns, the checkpoint {x.cols}")
            _matrix(dY, "dY", (x.rows, n), dts[0])
            if scale is not None:
                _matrix(scale, "scale", (k,), dts[0], vector=True)
            C = G if C is None else C
            if C is not G:
                _matrix(C, "C", (n, k), dts[1])
                if not C.is_contiguous():
                    _bad("C must be contiguous")
            descs.append(muon_wgrad_item(dY.data_ptr(), _ld(dY), x._c, _ptr(scale), G.data_ptr(), C.data_ptr(), n,
                                         float(beta), 0))
            tensors += [t for t in (dY, x.q, x.e, G, C, scale) if t is not None]
        if not descs:
            _bad("no items")
        self._n = len(descs)
        self._items = (muon_wgrad_item * self._n)(*descs)
        need = ctypes.c_size_t()
        check(lib().muon_wgrad_workspace(self._items, self._n, self._dtype, self._gdtype, ctypes.byref(need)))
        self.workspace = torch.empty(need.value, dtype=torch.uint8, device=tensors[0].device)
        self._streams = _Streams(tensors + [self.workspace])

    def run(self, stream=None) -> None:
        check(lib().muon_wgrad(self._items, self._n, self._dtype, self._gdtype, self.workspace.data_ptr(),
                               self.workspace.numel(), self._streams.use(stream)))

    def info(self) -> List[dict]:
        """Per item: the edge of its output tiles, and the pieces of its sum over rows."""
        tile, pieces = (ctypes.c_int32 * self._n)(), (ctypes.c_int32 * self._n)()
        check(lib().muon_wgrad_info(self._items, self._n, self._dtype, self._gdtype, tile, pieces))
        return [{"tile": t, "pieces": p} for t, p in zip(tile, pieces)]
