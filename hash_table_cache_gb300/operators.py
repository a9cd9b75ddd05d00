"""The operators on looked-up rows, on torch tensors (contracts: ``include/hkv.h``).

A training step on a table's rows is ``find`` -> ``mx_quantize`` ->
``mx_matmul`` -> ``preference_loss`` and its backward -> ``mx_matmul`` on the
copies along the other axis -> ``clip_grad_norm`` -> ``assign``; a serving step
scores hidden states against a 4-bit copy of rows.  With an adapter for each user
(a row of the table) it is ``find`` -> ``mx_matmul`` -> ``adapter_matmul`` ->
``token_logps``, and learning goes back through ``token_logps_backward`` and
``adapter_matmul_backward``.

Every function takes tensors of one CUDA device and raises ``ValueError`` for
a tensor it cannot take as it is (nothing is copied or cast behind the
caller's back) and ``HKVError`` for a status of the library.  ``stream``
(default: the current stream of the tensors' device) is the stream the
kernels run on and the one that results are allocated on.  Work on other
streams that the call depends on is the caller's to order, as with any CUDA
call; tensors passed with a ``stream`` may be dropped right after the call, and
so may a call's result after another one that takes it, on any stream (what such
a result keeps for later calls is not a tensor of the caller's).

The operators are outside autograd: a result carries no gradient function,
also where an input requires a gradient (the backward passes are calls of
their own).  A tensor that a call writes counts as modified in place.

The smallest calls take a few microseconds on the GPU, so the host's share is
kept small: one allocation per result, and no context is entered unless the
stream or the device has to change.
"""
from __future__ import annotations

from array import array
from operator import attrgetter

import torch

import hash_table_cache_gb300 as _abi

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_dtype_of = attrgetter("dtype")


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
    stride, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: columns have to be adjacent (stride 1)")
    if stride < cols:
        if rows > 1:
            raise ValueError(f"{what}: rows overlap")
        stride = cols
    return rows, cols, stride


def _vector(t, n, dtype, what, device):
    if t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous values of {dtype}")
    _same(t, device, what)


def _same(t, device, what):
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, not {device}")


def _cuda(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor")
    return t.device


# the current device and the handle of its current stream, without a Stream
# object (2 us less per call) where torch offers it
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, stream, f, *args):
    """f(stream handle, *args) with the device current and the caching allocator
    on the stream."""
    if stream is None:
        index = device.index
        if _device_now() == index:
            return f(_current(index), *args)
    with torch.cuda.device(device):
        if stream is None:
            return f(_current(device.index), *args)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif stream.device != device:
            raise ValueError(f"stream: of {stream.device}, not {device}")
        with torch.cuda.stream(stream):
            result = f(stream.cuda_stream, *args)
        # their memory is not used again before the stream is done with it
        for t in _tensors(args):
            t.record_stream(stream)
        return result


def _tensors(args):
    for a in args:
        if isinstance(a, torch.Tensor):
            yield a
        elif isinstance(a, (list, tuple)):
            yield from _tensors(a)
        elif isinstance(a, MXMatrix):
            yield from (a._codes, a._scales) if a._base is None else a._base[:1]
        elif isinstance(a, PreferenceLoss):
            yield from (a.logits, a.labels, a._saved)
        elif isinstance(a, AdapterMatmul):
            yield from (t for t in (a.x, a.down, a.up, a.offsets, a.which, a.scales, a._hidden) if t is not None)
        elif isinstance(a, TokenLogps):
            yield from (t for t in (a.logits, a.labels, a.entropy, a._lse) if t is not None)


def _keep(s, f, *tensors):
    """`tensors` are f's own, allocated on the stream f._stream: where this call runs on
    another one, their memory is not used again before it is done."""
    if f._stream is not None and s != f._stream:
        now = torch.cuda.current_stream(tensors[0].device)
        for t in tensors:
            t.record_stream(now)


# For tensors of the caller's that a kernel has written: autograd counts what it
# sees written, and would otherwise use one that it had saved as if unchanged.
_written = torch.autograd.graph.increment_version


def _ok(status, what):
    if status:
        raise _abi.HKVError(status, what)


def _mx_bytes(rows, cols):
    """Bytes of the codes and of the scales of a 4-bit matrix."""
    return rows * -(-cols // 32) * 16, -(-rows // 128) * -(-cols // 128) * 512


class MXMatrix:
    """A 4-bit microscaled matrix (MXFP4) of ``rows`` x ``cols``: ``codes`` and
    ``scales`` are uint8 tensors in the layout of ``include/hkv.h``."""

    __slots__ = ("rows", "cols", "device", "_codes", "_scales", "_base", "_at", "_stream")

    def __init__(self, codes, scales, rows, cols):
        rows, cols = int(rows), int(cols)
        self.device = _cuda(codes, "codes")
        _same(scales, self.device, "scales")
        need = _mx_bytes(rows, cols)
        for t, n, what in ((codes, need[0], "codes"), (scales, need[1], "scales")):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{what}: {n} contiguous bytes for {rows} x {cols}")
        self.rows, self.cols = rows, cols
        self._codes, self._scales, self._base = codes, scales, None
        self._stream = None  # the caller's tensors
        self._at = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def _empty(cls, rows, cols, device, s):
        """A matrix to be written, codes and scales in one allocation of its own:
        of two copies from one call either may be kept without the other."""
        m = cls.__new__(cls)
        codes = -(-rows * -(-cols // 32) // 32) * 512  # in whole groups
        room = codes + -(-rows // 128) * -(-cols // 128) * 512
        base = torch.empty(room, dtype=torch.uint8, device=device)
        at = base.data_ptr()
        m.rows, m.cols, m.device = rows, cols, device
        m._codes = m._scales = None
        m._base = base, codes
        m._at = at, at + codes
        m._stream = s
        return m

    def _piece(self, skip, size, shape):
        base, codes = self._base
        start = codes if skip else 0
        return base[start:start + size].view(shape)

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._piece(False, _mx_bytes(self.rows, self.cols)[0],
                                      (self.rows, -(-self.cols // 32) * 16))
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._piece(True, _mx_bytes(self.rows, self.cols)[1],
                                       (-(-self.rows // 128), -(-self.cols // 128), 512))
        return self._scales

    @property
    def shape(self):
        return (self.rows, self.cols)

    def dequantize(self, dtype=torch.float32, out=None, stream=None):
        """The values the matrix stands for."""
        return _call(self.device, stream, _dequantize, self, dtype, out)


def _dequantize(s, q, dtype, out):
    given = out
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.device)
    kind = _type(out, "out")
    rows, cols, stride = _matrix(out, "out")
    if rows != q.rows or cols != q.cols:
        raise ValueError(f"out: {q.rows} x {q.cols}")
    _same(out, q.device, "out")
    if s != q._stream:
        _keep(s, q, *_tensors((q,)))
    codes, scales = q._at
    _ok(_abi.load().hkv_mx_dequantize(rows, cols, codes, scales, out.data_ptr(), kind, stride, s),
        "hkv_mx_dequantize")
    if given is not None:
        _written(given)
    return out


def mx_quantize(x, along="rows", stream=None):
    """The 4-bit copy of a matrix: of its rows (``along="rows"``), of its columns
    (``"columns"``: the copy of ``x.t()``), or both as a tuple (``"both"``, one read
    of ``x``)."""
    if along not in ("rows", "columns", "both"):
        raise ValueError(f"along: rows, columns or both, not {along!r}")
    return _call(_cuda(x, "x"), stream, _quantize, x, along)


def _quantize(s, x, along):
    kind = _type(x, "x")
    rows, cols, stride = _matrix(x, "x")
    device = x.device
    codes = scales = codes_t = scales_t = None
    if along != "columns":
        q = MXMatrix._empty(rows, cols, device, s)
        codes, scales = q._at
    if along != "rows":
        q_t = MXMatrix._empty(cols, rows, device, s)
        codes_t, scales_t = q_t._at
    _ok(_abi.load().hkv_mx_quantize(rows, cols, x.data_ptr(), kind, stride, codes, scales, codes_t,
                                    scales_t, s), "hkv_mx_quantize")
    return (q, q_t) if along == "both" else q if along == "rows" else q_t


def mx_matmul(a, b, dtype=torch.bfloat16, out=None, stream=None):
    """``a`` (m x k) times the transpose of ``b`` (n x k), both ``MXMatrix``: an
    m x n tensor of ``dtype``, or ``out``."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if a.device != b.device:
        raise ValueError(f"b: on {b.device}, not {a.device}")
    return _call(a.device, stream, _matmul, a, b, dtype, out)


def _matmul(s, a, b, dtype, out):
    m, n = a.rows, b.rows
    given = out
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=a.device)
        kind, stride = _type(out, "out"), n
    else:
        kind = _type(out, "out")
        rows, cols, stride = _matrix(out, "out")
        if rows != m or cols != n:
            raise ValueError(f"out: {m} x {n}")
        _same(out, a.device, "out")
    if s != a._stream or s != b._stream:
        _keep(s, a, *_tensors((a,)))
        _keep(s, b, *_tensors((b,)))
    at, bt = a._at, b._at
    _ok(_abi.load().hkv_mx_matmul(m, n, a.cols, at[0], at[1], bt[0], bt[1], out.data_ptr(), kind,
                                  stride, s), "hkv_mx_matmul")
    if given is not None:
        _written(given)
    return out


class PreferenceLoss:
    """What ``preference_loss`` returns: ``losses`` [pairs], ``ratios`` [2 * pairs],
    ``logps`` [tokens], and what the backward call needs."""

    __slots__ = ("losses", "ratios", "logps", "logits", "labels", "_saved", "_stream")


def preference_loss(logits, labels, offsets, ref_logps=None, beta=0.1, label_smoothing=0.0,
                    average=False, stream=None):
    """The logistic loss of paired log ratios of token sequences.

    ``logits`` [tokens, vocab]; ``labels`` int64 [tokens], a value outside the
    vocabulary for tokens that are not counted; ``offsets`` int64
    [2 * pairs + 1] on the device, the chosen sequences first, then the
    rejected ones; ``ref_logps`` float32 [tokens], the reference model's log
    probabilities of the labels.  Returns a ``PreferenceLoss``."""
    return _call(_cuda(logits, "logits"), stream, _loss, logits, labels, offsets, ref_logps, beta,
                 label_smoothing, average)


def _loss(s, logits, labels, offsets, ref_logps, beta, label_smoothing, average):
    device = logits.device
    kind = _type(logits, "logits")
    rows, vocab, stride = _matrix(logits, "logits")
    _vector(labels, rows, torch.int64, "labels", device)
    pairs, odd = divmod(offsets.numel(), 2)
    if not odd:
        raise ValueError("offsets: 2 * pairs + 1 values")
    _vector(offsets, 2 * pairs + 1, torch.int64, "offsets", device)
    if ref_logps is not None:
        _vector(ref_logps, rows, torch.float32, "ref_logps", device)
    f = PreferenceLoss()
    f.logits, f.labels, f._stream = logits, labels, s
    # what a caller may keep longer than the rest (the losses of every step, a
    # reference's logps) has memory of its own
    base = torch.empty(3 * pairs, dtype=torch.float32, device=device)
    f.losses, f.ratios = base.split_with_sizes((pairs, 2 * pairs))
    f.logps = torch.empty(rows, dtype=torch.float32, device=device)
    # lse, row_grad and row_pair of 4 bytes each
    f._saved = torch.empty(3 * rows, dtype=torch.float32, device=device)
    at, saved = base.data_ptr(), f._saved.data_ptr()
    _ok(_abi.load().hkv_preference_loss(
        pairs, rows, vocab, logits.data_ptr(), kind, stride, labels.data_ptr(), offsets.data_ptr(),
        None if ref_logps is None else ref_logps.data_ptr(), beta, label_smoothing,
        1 if average else 0, at, at + 4 * pairs, f.logps.data_ptr(), saved, saved + 4 * rows,
        saved + 8 * rows, s), "hkv_preference_loss")
    return f


def preference_loss_backward(loss, dlosses=None, out=None, stream=None):
    """The gradient of ``(dlosses * loss.losses).sum()`` with respect to the
    logits, in their type, from what ``preference_loss`` returned.  ``out`` may be
    the logits themselves, which then hold the gradient."""
    return _call(loss.logits.device, stream, _loss_backward, loss, dlosses, out)


def _loss_backward(s, loss, dlosses, out):
    logits = loss.logits
    device = logits.device
    rows, vocab, stride = _matrix(logits, "logits")
    pairs = loss.losses.numel()
    given = out
    if dlosses is not None:
        _vector(dlosses, pairs, torch.float32, "dlosses", device)
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=device)
        dstride = vocab
    else:
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError(f"out: {rows} x {vocab} of {logits.dtype}")
        _same(out, device, "out")
        dstride = _matrix(out, "out")[2]
    _keep(s, loss, loss._saved)
    saved = loss._saved.data_ptr()
    _ok(_abi.load().hkv_preference_loss_backward(
        pairs, rows, vocab, logits.data_ptr(), _TYPES[logits.dtype], stride, loss.labels.data_ptr(),
        saved, saved + 4 * rows, saved + 8 * rows, None if dlosses is None else dlosses.data_ptr(),
        out.data_ptr(), dstride, s), "hkv_preference_loss_backward")
    if given is not None:
        _written(given)
    return out


class TokenLogps:
    """What ``token_logps`` returns: ``logps`` [tokens] (None without labels),
    ``entropy`` [tokens], ``top_logps`` and int64 ``top_ids`` [tokens, top] (None where
    ``top`` is 0), and what the backward call needs."""

    __slots__ = ("logps", "entropy", "top_logps", "top_ids", "logits", "labels", "_lse", "_stream")


def token_logps(logits, labels=None, top=0, stream=None):
    """Log probabilities of given tokens, with the entropy and the ``top`` (at most
    32) largest entries of their rows of logits.

    ``logits`` [tokens, vocab]; ``labels`` int64 [tokens], a value outside the
    vocabulary for tokens that are not counted, or None: entropy and alternatives
    of every row.  Alternatives go from the largest down, equal ones by the lower
    index.  Returns a ``TokenLogps``."""
    return _call(_cuda(logits, "logits"), stream, _token_logps, logits, labels, top)


def _token_logps(s, logits, labels, top):
    device = logits.device
    kind = _type(logits, "logits")
    rows, vocab, stride = _matrix(logits, "logits")
    if not 0 <= top <= _abi.MAX_TOP or top > vocab:
        raise ValueError(f"top: 0 to {min(vocab, _abi.MAX_TOP)}, not {top}")
    empty, f32 = torch.empty, torch.float32
    f = TokenLogps()
    f.logits, f.labels, f._stream = logits, labels, s
    f.entropy = entropy = empty(rows, dtype=f32, device=device)
    f._lse = lse = empty(2 * rows, dtype=f32, device=device)
    f.logps = f.top_logps = f.top_ids = at_labels = at_logps = at_top = at_ids = None
    if labels is not None:
        _vector(labels, rows, torch.int64, "labels", device)
        f.logps = t = empty(rows, dtype=f32, device=device)
        at_labels, at_logps = labels.data_ptr(), t.data_ptr()
    if top:
        f.top_logps = t = empty((rows, top), dtype=f32, device=device)
        f.top_ids = u = empty((rows, top), dtype=torch.int64, device=device)
        at_top, at_ids = t.data_ptr(), u.data_ptr()
    _ok(_abi.load().hkv_token_logps(rows, vocab, logits.data_ptr(), kind, stride, at_labels, top,
                                    at_logps, entropy.data_ptr(), at_top, at_ids, lse.data_ptr(), s),
        "hkv_token_logps")
    return f


def token_logps_backward(f, dlogps=None, dentropy=None, out=None, stream=None):
    """The gradient of ``(dlogps * f.logps + dentropy * f.entropy).sum()`` with
    respect to the logits, in their type, from what ``token_logps`` returned.
    ``out`` may be the logits themselves, which then hold the gradient."""
    return _call(f.logits.device, stream, _token_logps_backward, f, dlogps, dentropy, out)


def _token_logps_backward(s, f, dlogps, dentropy, out):
    logits = f.logits
    device = logits.device
    rows, vocab, stride = _matrix(logits, "logits")
    given = out
    if dlogps is not None:
        if f.labels is None:
            raise ValueError("dlogps: there were no labels")
        _vector(dlogps, rows, torch.float32, "dlogps", device)
    if dentropy is not None:
        _vector(dentropy, rows, torch.float32, "dentropy", device)
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=device)
        dstride = vocab
    else:
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError(f"out: {rows} x {vocab} of {logits.dtype}")
        _same(out, device, "out")
        dstride = _matrix(out, "out")[2]
    _keep(s, f, f._lse, f.entropy)
    at = [None if t is None else t.data_ptr() for t in (f.labels, dlogps, dentropy)]
    _ok(_abi.load().hkv_token_logps_backward(
        rows, vocab, logits.data_ptr(), _TYPES[logits.dtype], stride, at[0], f._lse.data_ptr(),
        f.entropy.data_ptr(), at[1], at[2], out.data_ptr(), dstride, s), "hkv_token_logps_backward")
    if given is not None:
        _written(given)
    return out


class AdapterMatmul:
    """What ``adapter_matmul`` returns: ``out`` [tokens, n], and what the backward call
    needs."""

    __slots__ = ("out", "x", "down", "up", "offsets", "which", "scales", "_adapters", "_shape", "_hidden",
                 "_stream")


def adapter_matmul(x, down, up, offsets, which, scales=None, base=None, out=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection:
    ``base + scale * (x @ down[a].t()) @ up[a].t()`` for the rows of each request, with
    the request's adapter a.

    ``x`` [tokens, k]; ``down`` [adapters, rank, k] and ``up`` [adapters, n, rank] of
    its type, rank at most 64, each adapter's rows of adjacent columns (an adapter
    may be a row of a larger tensor, as of a table's rows); request s has the rows
    ``offsets[s]`` to ``offsets[s + 1]`` and the adapter ``which[s]`` (int64, on the
    device; a value outside the adapters for a request without one); ``scales``
    float32 [adapters]; ``base`` [tokens, n], the shared projection's result (None:
    zeros), which may be ``out``.  Rows without an adapter are ``base``'s.  Returns an
    ``AdapterMatmul``."""
    return _call(_cuda(x, "x"), stream, _adapter_matmul, x, down, up, offsets, which, scales, base, out)


def _given(t, shape, dtype, index, what):
    """The strides of a tensor that has to have that shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{what}: {' x '.join(map(str, shape))} of {dtype} on cuda:{index}")
    return t.stride()


def _row_stride(strides, shape, what):
    """The stride of a matrix's (or of each of some matrices') rows."""
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{what}: columns have to be adjacent (stride 1)")
    stride = strides[-2]
    if stride < shape[-1]:
        if shape[-2] > 1:
            raise ValueError(f"{what}: rows overlap")
        stride = shape[-1]
    return stride


def _adapter_matmul(s, x, down, up, offsets, which, scales, base, out):
    dtype, index = x.dtype, x.get_device()
    kind = _TYPES.get(dtype)
    if kind is None or x.dim() != 2 or down.dim() != 3 or up.dim() != 3 or which.dim() != 1:
        raise ValueError("x: a matrix of float32, bfloat16 or float16; down, up: adapters x rank x k and "
                         "adapters x n x rank; which: a vector")
    tokens, k = shape_x = x.shape
    x_stride = _row_stride(x.stride(), shape_x, "x")
    count, n, rank = shape_up = up.shape
    if not 1 <= rank <= _abi.MAX_RANK or not k or not n:
        raise ValueError(f"up: a rank of 1 to {_abi.MAX_RANK}, not {rank}, and k and n of at least 1")
    shape_down = count, rank, k
    strides = _given(down, shape_down, dtype, index, "down")
    down_step, down_stride = strides[0], _row_stride(strides, shape_down, "down")
    strides = _given(up, shape_up, dtype, index, "up")
    up_step, up_stride = strides[0], _row_stride(strides, shape_up, "up")
    requests, = shape = which.shape
    if (_given(which, shape, torch.int64, index, "which")[0] != 1 and requests > 1) or \
            (_given(offsets, (requests + 1,), torch.int64, index, "offsets")[0] != 1 and requests):
        raise ValueError("which, offsets: contiguous vectors")
    at_scales = at_base = None
    base_stride = 0
    if scales is not None:
        if _given(scales, (count,), torch.float32, index, "scales")[0] != 1 and count > 1:
            raise ValueError("scales: a contiguous vector")
        at_scales = scales.data_ptr()
    shape = tokens, n
    if base is not None:
        base_stride = _row_stride(_given(base, shape, dtype, index, "base"), shape, "base")
        at_base = base.data_ptr()
    f = AdapterMatmul()
    given = out
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        stride = n
    else:
        stride = _row_stride(_given(out, shape, dtype, index, "out"), shape, "out")
    f.out, f.x, f.down, f.up, f.offsets, f.which, f.scales = out, x, down, up, offsets, which, scales
    f._hidden = hidden = torch.empty(_abi.adapter_hidden_bytes(tokens, rank, kind), dtype=torch.uint8,
                                     device=x.device)
    # hkv_adapters
    f._adapters = adapters = array("Q", (count, down.data_ptr(), down_step, down_stride, up.data_ptr(),
                                         up_step, up_stride, at_scales or 0, rank))
    f._shape = tokens, k, n, kind, x_stride, requests, count, rank
    f._stream = s
    _ok(_abi.load().hkv_adapter_matmul(
        tokens, k, n, kind, adapters.buffer_info()[0], requests, offsets.data_ptr(), which.data_ptr(),
        x.data_ptr(), x_stride, at_base, base_stride, out.data_ptr(), stride, hidden.data_ptr(), s),
        "hkv_adapter_matmul")
    if given is not None:
        _written(given)
    return f


def adapter_matmul_backward(f, dout, base=None, out=None, stream=None):
    """The gradients of ``(dout * f.out).sum()``: (dx, ddown, dup), in the matrices'
    type, from what ``adapter_matmul`` returned.  ``base`` [tokens, k] is added to dx
    (the gradient through the shared projection), and may be ``out``, which takes dx.
    Beyond some thousands of adapters and requests the time grows with their product."""
    return _call(f.x.device, stream, _adapter_matmul_backward, f, dout, base, out)


def _adapter_matmul_backward(s, f, dout, base, out):
    x, adapters = f.x, f._adapters
    dtype, device = x.dtype, x.device
    index = device.index
    tokens, k, n, kind, x_stride, requests, count, rank = f._shape
    shape = tokens, n
    d_stride = _row_stride(_given(dout, shape, dtype, index, "dout"), shape, "dout")
    shape = tokens, k
    at_base, base_stride = None, 0
    if base is not None:
        base_stride = _row_stride(_given(base, shape, dtype, index, "base"), shape, "base")
        at_base = base.data_ptr()
    given = out
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        stride = k
    else:
        stride = _row_stride(_given(out, shape, dtype, index, "out"), shape, "out")
    ddown = torch.empty((count, rank, k), dtype=dtype, device=device)
    dup = torch.empty((count, n, rank), dtype=dtype, device=device)
    dhidden = torch.empty_like(f._hidden)
    _keep(s, f, f._hidden)
    _ok(_abi.load().hkv_adapter_matmul_backward(
        tokens, k, n, kind, adapters.buffer_info()[0], requests, f.offsets.data_ptr(), f.which.data_ptr(),
        x.data_ptr(), x_stride, dout.data_ptr(), d_stride, f._hidden.data_ptr(), at_base, base_stride,
        out.data_ptr(), stride, ddown.data_ptr(), dup.data_ptr(), dhidden.data_ptr(), s),
        "hkv_adapter_matmul_backward")
    if given is not None:
        _written(given)
    return out, ddown, dup


def _dense(t):
    """Whether the tensor's elements fill one piece of memory, in any order."""
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
    as many elements as its gradient, and lies in memory in the same order
    (both contiguous, or the same shape and strides).  What is written must not
    overlap another tensor of the call: the gradient of a parameter that is
    used twice is listed once."""
    if type(grads) is not list:
        grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError("grads: at least one tensor")
    if isinstance(outs, str) and outs != "in place":
        raise ValueError(f"outs: tensors, () or 'in place', not {outs!r}")
    if outs is None or isinstance(outs, str):
        outs = grads
    else:
        outs = [outs] if isinstance(outs, torch.Tensor) else list(outs)
        if outs and len(outs) != len(grads):
            raise ValueError(f"outs: {len(grads)} tensors")
    return _call(_cuda(grads[0], "grads"), stream, _clip, grads, outs, max_norm)


def _fields(tensors, what, device):
    """Addresses of dense tensors of one device, their types (one number where
    they share it), and whether all of them are contiguous.  One C call per
    tensor and field: hundreds of tensors are common here."""
    of = torch.Tensor
    if list(map(of.get_device, tensors)).count(device.index) != len(tensors):
        raise ValueError(f"{what}: tensors of {device}")
    plain = all(map(of.is_contiguous, tensors))
    if not plain and not all(map(_dense, tensors)):
        raise ValueError(f"{what}: tensors have to be dense")
    kinds = list(map(_dtype_of, tensors))
    try:
        if kinds.count(kinds[0]) == len(kinds):
            types = _TYPES[kinds[0]]
        else:
            types = list(map(_TYPES.__getitem__, kinds))
    except KeyError as e:
        raise ValueError(f"{what}: float32, bfloat16 or float16, not {e.args[0]}") from None
    return array("Q", list(map(of.data_ptr, tensors))), types, plain


def _both_types(types, out_types, n):
    """type | out_type << 32 of every gradient; a number stands for all of them."""
    if isinstance(types, int) and isinstance(out_types, int):
        return array("Q", (types | out_types << 32,)) * n
    types, out_types = ([t] * n if isinstance(t, int) else t for t in (types, out_types))
    return array("Q", [t | u << 32 for t, u in zip(types, out_types)])


def _clip(s, grads, outs, max_norm):
    device = grads[0].device
    n = len(grads)
    data, types, plain = _fields(grads, "grads", device)
    table = array("Q", bytes(32 * n))  # hkv_grad: data, out, n, type | out_type << 32
    table[0::4] = data
    sizes = array("Q", list(map(torch.Tensor.numel, grads)))
    table[2::4] = sizes
    if outs is grads:
        table[1::4] = data
        table[3::4] = _both_types(types, types, n)
    elif outs:
        to, out_types, out_plain = _fields(outs, "outs", device)
        same = array("Q", map(torch.Tensor.numel, outs)) == sizes
        if same and not (plain and out_plain):
            same = all(o.shape == g.shape and o.stride() == g.stride() for o, g in zip(outs, grads))
        if not same:
            raise ValueError("outs: the sizes and the order in memory of the gradients")
        table[1::4] = to
        table[3::4] = _both_types(types, out_types, n)
    else:
        table[3::4] = _both_types(types, 0, n)
    norm = torch.empty((), dtype=torch.float32, device=device)
    work = torch.empty(_abi.CLIP_WORK_BYTES, dtype=torch.uint8, device=device)
    _ok(_abi.load().hkv_clip_grad_norm(n, table.buffer_info()[0], max_norm, norm.data_ptr(),
                                       work.data_ptr(), s), "hkv_clip_grad_norm")
    if outs:
        _written(outs)
    return norm
