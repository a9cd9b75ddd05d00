"""The operators on looked-up rows, on torch tensors (contracts: ``include/hkv.h``).

A training step on a table's rows is ``find`` -> ``mx_quantize`` ->
``mx_matmul`` -> ``preference_loss`` and its backward -> ``mx_matmul`` on the
copies along the other axis -> ``clip_grad_norm`` -> ``assign``; a serving step
scores hidden states against a 4-bit copy of rows.

Every function takes tensors of one CUDA device and raises ``ValueError`` for
a tensor it cannot take as it is (nothing is copied or cast behind the
caller's back) and ``HKVError`` for a status of the library.  ``stream``
(default: the current stream of the tensors' device) is the stream the
kernels run on and the one that results are allocated on; tensors made on
another stream are the caller's to order, as with any CUDA call.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

import hash_table_cache_gb300 as _abi

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _type(t, what):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{what}: float32, bfloat16 or float16, not {t.dtype}") from None


def _matrix(t, what):
    """(rows, columns, row stride) of a matrix with adjacent columns."""
    if t.dim() != 2:
        raise ValueError(f"{what}: a matrix, not {t.dim()} dimensions")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: columns have to be adjacent (stride 1)")
    stride = t.stride(0)
    if rows < 2:
        stride = max(stride, cols)
    elif stride < cols:
        raise ValueError(f"{what}: rows overlap")
    return rows, cols, stride


def _vector(t, n, dtype, what, device):
    if t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous values of {dtype}")
    _same(t, device, what)
    return t


def _same(t, device, what):
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, not {device}")


def _cuda(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor")
    return t.device


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _on(device, stream):
    """The stream handle to launch on, with its device current and the caching
    allocator on that stream."""
    if stream is None and torch.cuda.current_device() == device.index:
        return contextlib.nullcontext(torch.cuda.current_stream(device).cuda_stream)
    return _switched(device, stream)


def _ok(status, what):
    if status:
        raise _abi.HKVError(status, what)


class MXMatrix:
    """A 4-bit microscaled matrix (MXFP4) of ``rows`` x ``cols``: ``codes`` and
    ``scales`` are uint8 tensors in the layout of ``include/hkv.h``."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, rows, cols):
        rows, cols = int(rows), int(cols)
        device = _cuda(codes, "codes")
        _same(scales, device, "scales")
        need = (rows * -(-cols // 32) * 16, -(-rows // 128) * -(-cols // 128) * 512)
        for t, n, what in ((codes, need[0], "codes"), (scales, need[1], "scales")):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{what}: {n} contiguous bytes for {rows} x {cols}")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @classmethod
    def empty(cls, rows, cols, device):
        """Room for a matrix, not initialised."""
        m = cls.__new__(cls)
        m.codes = torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device)
        m.scales = torch.empty((-(-rows // 128), -(-cols // 128), 512), dtype=torch.uint8,
                               device=device)
        m.rows, m.cols = rows, cols
        return m

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def dequantize(self, dtype=torch.float32, out=None, stream=None):
        """The values the matrix stands for."""
        with _on(self.device, stream) as s:
            if out is None:
                out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.device)
            kind = _type(out, "out")
            _same(out, self.device, "out")
            rows, cols, stride = _matrix(out, "out")
            if (rows, cols) != self.shape:
                raise ValueError(f"out: {self.rows} x {self.cols}")
            _ok(_abi.load().hkv_mx_dequantize(rows, cols, self.codes.data_ptr(),
                                              self.scales.data_ptr(), out.data_ptr(), kind, stride,
                                              s), "hkv_mx_dequantize")
        return out


def mx_quantize(x, along="rows", stream=None):
    """The 4-bit copy of a matrix: of its rows (``along="rows"``), of its columns
    (``"columns"``: the copy of ``x.t()``), or both as a tuple (``"both"``, one read
    of ``x``)."""
    if along not in ("rows", "columns", "both"):
        raise ValueError(f"along: rows, columns or both, not {along!r}")
    device = _cuda(x, "x")
    kind = _type(x, "x")
    rows, cols, stride = _matrix(x, "x")
    with _on(device, stream) as s:
        q = MXMatrix.empty(rows, cols, device) if along != "columns" else None
        qt = MXMatrix.empty(cols, rows, device) if along != "rows" else None
        _ok(_abi.load().hkv_mx_quantize(
            rows, cols, x.data_ptr(), kind, stride,
            q.codes.data_ptr() if q else None, q.scales.data_ptr() if q else None,
            qt.codes.data_ptr() if qt else None, qt.scales.data_ptr() if qt else None, s),
            "hkv_mx_quantize")
    return (q, qt) if along == "both" else q or qt


def mx_matmul(a, b, dtype=torch.bfloat16, out=None, stream=None):
    """``a`` (m x k) times the transpose of ``b`` (n x k), both ``MXMatrix``: an
    m x n tensor of ``dtype``, or ``out``."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    device = a.device
    _same(b.codes, device, "b")
    with _on(device, stream) as s:
        if out is None:
            out = torch.empty((a.rows, b.rows), dtype=dtype, device=device)
        kind = _type(out, "out")
        _same(out, device, "out")
        m, n, stride = _matrix(out, "out")
        if (m, n) != (a.rows, b.rows):
            raise ValueError(f"out: {a.rows} x {b.rows}")
        _ok(_abi.load().hkv_mx_matmul(m, n, a.cols, a.codes.data_ptr(), a.scales.data_ptr(),
                                      b.codes.data_ptr(), b.scales.data_ptr(), out.data_ptr(), kind,
                                      stride, s), "hkv_mx_matmul")
    return out


class PreferenceLoss:
    """What ``preference_loss`` returns: ``losses`` [pairs], ``ratios`` [2 * pairs],
    ``logps`` [tokens], and what the backward call needs."""

    __slots__ = ("losses", "ratios", "logps", "logits", "labels", "lse", "row_grad", "row_pair")


def preference_loss(logits, labels, offsets, ref_logps=None, beta=0.1, label_smoothing=0.0,
                    average=False, stream=None):
    """The logistic loss of paired log ratios of token sequences.

    ``logits`` [tokens, vocab]; ``labels`` int64 [tokens], a value outside the
    vocabulary for tokens that are not counted; ``offsets`` int64
    [2 * pairs + 1] on the device, the chosen sequences first, then the
    rejected ones; ``ref_logps`` float32 [tokens], the reference model's log
    probabilities of the labels.  Returns a ``PreferenceLoss``."""
    device = _cuda(logits, "logits")
    kind = _type(logits, "logits")
    rows, vocab, stride = _matrix(logits, "logits")
    _vector(labels, rows, torch.int64, "labels", device)
    if offsets.dim() != 1 or offsets.numel() % 2 == 0:
        raise ValueError("offsets: 2 * pairs + 1 values")
    pairs = offsets.numel() // 2
    _vector(offsets, 2 * pairs + 1, torch.int64, "offsets", device)
    if ref_logps is not None:
        _vector(ref_logps, rows, torch.float32, "ref_logps", device)
    f = PreferenceLoss()
    f.logits, f.labels = logits, labels
    with _on(device, stream) as s:
        f.losses = torch.empty(pairs, dtype=torch.float32, device=device)
        f.ratios = torch.empty(2 * pairs, dtype=torch.float32, device=device)
        f.logps, f.lse, f.row_grad = (torch.empty(rows, dtype=torch.float32, device=device)
                                      for _ in range(3))
        f.row_pair = torch.empty(rows, dtype=torch.int32, device=device)
        _ok(_abi.load().hkv_preference_loss(
            pairs, rows, vocab, logits.data_ptr(), kind, stride, labels.data_ptr(),
            offsets.data_ptr(), ref_logps.data_ptr() if ref_logps is not None else None, beta,
            label_smoothing, int(bool(average)), f.losses.data_ptr(), f.ratios.data_ptr(),
            f.logps.data_ptr(), f.lse.data_ptr(), f.row_grad.data_ptr(), f.row_pair.data_ptr(), s),
            "hkv_preference_loss")
    return f


def preference_loss_backward(loss, dlosses=None, out=None, stream=None):
    """The gradient of ``(dlosses * loss.losses).sum()`` with respect to the
    logits, in their type, from what ``preference_loss`` returned.  ``out`` may be
    the logits themselves, which then hold the gradient."""
    logits = loss.logits
    device = logits.device
    rows, vocab, stride = _matrix(logits, "logits")
    pairs = loss.losses.numel()
    if dlosses is not None:
        _vector(dlosses, pairs, torch.float32, "dlosses", device)
    with _on(device, stream) as s:
        if out is None:
            out = torch.empty((rows, vocab), dtype=logits.dtype, device=device)
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError(f"out: {rows} x {vocab} of {logits.dtype}")
        _same(out, device, "out")
        _, _, dstride = _matrix(out, "out")
        _ok(_abi.load().hkv_preference_loss_backward(
            pairs, rows, vocab, logits.data_ptr(), _TYPES[logits.dtype], stride,
            loss.labels.data_ptr(), loss.lse.data_ptr(), loss.row_grad.data_ptr(),
            loss.row_pair.data_ptr(), dlosses.data_ptr() if dlosses is not None else None,
            out.data_ptr(), dstride, s), "hkv_preference_loss_backward")
    return out


def _dense(t):
    """Whether the tensor's elements fill one piece of memory, in any order."""
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != n:
            return False
        n *= size
    return True


def clip_grad_norm(grads, max_norm, outs="in place", stream=None):
    """The norm of all ``grads`` taken as one vector, as a float32 scalar tensor,
    and clipping to ``max_norm``: in place (the default, also ``outs=None``), into
    the tensors ``outs`` (of any of the three types), or not at all
    (``outs=()``: the norm alone).  Tensors have to be dense; an out tensor has
    its gradient's shape and strides."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if outs is None or isinstance(outs, str):
        if isinstance(outs, str) and outs != "in place":
            raise ValueError(f"outs: tensors, () or 'in place', not {outs!r}")
        targets = grads
    else:
        targets = [outs] if isinstance(outs, torch.Tensor) else list(outs)
        if targets and len(targets) != len(grads):
            raise ValueError(f"outs: {len(grads)} tensors")
    if not grads:
        raise ValueError("grads: at least one tensor")
    device = _cuda(grads[0], "grads")
    table = (_abi.Grad * len(grads))()
    for i, g in enumerate(grads):
        _same(g, device, "grads")
        if not _dense(g):
            raise ValueError("grads: tensors have to be dense")
        o = targets[i] if targets else None
        e = table[i]
        e.data, e.n, e.type = g.data_ptr(), g.numel(), _type(g, "grads")
        if o is not None:
            if o is not g:
                _same(o, device, "outs")
                if o.shape != g.shape or (o.stride() != g.stride() and not (
                        o.is_contiguous() and g.is_contiguous())):
                    raise ValueError("outs: the shapes and strides of the gradients")
            e.out, e.out_type = o.data_ptr(), _type(o, "outs")
    with _on(device, stream) as s:
        norm = torch.empty((), dtype=torch.float32, device=device)
        work = torch.empty(_abi.CLIP_WORK_BYTES, dtype=torch.uint8, device=device)
        _ok(_abi.load().hkv_clip_grad_norm(len(grads), ctypes.addressof(table), max_norm,
                                           norm.data_ptr(), work.data_ptr(), s),
            "hkv_clip_grad_norm")
    return norm
