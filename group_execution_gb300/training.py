"""Training-step operators: layer norm, 8-bit activation checkpoints and the
gradients that read them, token log probabilities, the embedding of tokens, and
the cross entropy of a linear layer over the vocabulary.

Argument marshalling only, as everywhere in this package: the caller passes
every tensor, outputs included, and the library's kernels do the work (see
the training-step section of include/groupexec.h for what each computes).
Matrices are 2-D float32 or bfloat16 tensors whose rows are contiguous (any
row stride); vectors and row statistics are contiguous float32.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import FG_BF16, FG_EINVAL, FG_ESHAPE, FG_F32, FgError, OPCODES

_DTYPES = {torch.float32: FG_F32, torch.bfloat16: FG_BF16}


def _matrix(name, t, rows, cols, device):
    """(pointer, dtype, row pitch) of a matrix argument on `device`."""
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise FgError(FG_EINVAL, f"{name}: must be float32 or bfloat16")
    if t.get_device() != device:       # (-1: not a CUDA tensor)
        raise FgError(FG_EINVAL, f"{name}: must be on the handle's CUDA device")
    if t.shape != (rows, cols):
        raise FgError(FG_ESHAPE, f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise FgError(FG_EINVAL, f"{name}: a row's elements must be contiguous")
    if rows < 2 and ld < cols:
        ld = cols                      # the stride of a single row says nothing
    return t.data_ptr(), dt, ld


def _array(name, t, shape, device, dtype=torch.float32):
    """Pointer of a dense array argument (None passes through)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device:
        raise FgError(FG_EINVAL, f"{name}: must be of {dtype} on the handle's CUDA device")
    if t.shape != shape:
        raise FgError(FG_ESHAPE, f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise FgError(FG_EINVAL, f"{name}: must be contiguous")
    return t.data_ptr()


# The current stream's handle; making a torch.cuda.Stream object to ask takes
# longer (2.9 us) than all checks of a call.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def checkpoint_layout(rows, cols):
    """(pitch, scale offset, bytes) of a [rows, cols] checkpoint's buffer
    (host only)."""
    lib = _lib.load()
    v = [C.c_int64() for _ in range(3)]
    _lib.check(lib.ts_checkpoint_layout(rows, cols, *[C.byref(x) for x in v]))
    return tuple(x.value for x in v)


def linear_cross_entropy_workspace(rows, cols, vocab):
    """(least, most) workspace bytes of linear_cross_entropy and its gradient:
    below the first they are refused, with the second they take all rows and
    the whole vocabulary at once (host only)."""
    lib = _lib.load()
    v = [C.c_int64() for _ in range(2)]
    _lib.check(lib.ts_linear_cross_entropy_workspace(rows, cols, vocab, *[C.byref(x) for x in v]))
    return tuple(x.value for x in v)


class Checkpoint:
    """A [rows, cols] matrix in 8 bits: one byte buffer, allocated here unless
    given (checkpoint_layout says how it is laid out)."""

    def __init__(self, rows, cols, buf=None, device="cuda"):
        pitch = -(-cols // 128) * 128
        size = rows * pitch + rows * (pitch // 32)
        if rows < 0 or cols < 1:
            raise FgError(FG_ESHAPE, "rows must be at least 0 and columns at least 1")
        if buf is None:
            buf = torch.empty(size, dtype=torch.uint8, device=device)
        elif buf.dtype != torch.uint8 or not buf.is_cuda or not buf.is_contiguous() or buf.numel() < size:
            raise FgError(FG_EINVAL, f"checkpoint buffer: needs {size} contiguous CUDA bytes")
        self.rows, self.cols, self.buf = rows, cols, buf
        self.ptr, self.device = buf.data_ptr(), buf.get_device()


class TrainingOps:
    """A handle of the training-step operators on the current device.  Calls
    of one handle must be ordered (one stream, or streams that wait for each
    other); use one handle per concurrent stream.  wait_limit_ns bounds every
    device-side wait."""

    def __init__(self, workspace_bytes=0, wait_limit_ns=2_000_000_000, flags=0):
        self.lib = _lib.load()
        self.h = C.c_void_p()
        _lib.check(self.lib.ts_create(workspace_bytes, C.byref(self.h)))
        _lib.check(self.lib.ts_set_wait_limit(self.h, wait_limit_ns, flags))
        self.device = torch.cuda.current_device()

    def __del__(self):
        h = getattr(self, "h", None)
        if h:
            self.lib.ts_destroy(h)
            self.h = None

    def _stream(self, stream):
        if stream is None:
            return _current(self.device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def sync(self, stream=None):
        """Waits for the stream; raises FgError (FG_ETIMEOUT) if a kernel
        recorded an expired wait."""
        _lib.check(self.lib.ts_sync_status(self.h, self._stream(stream)))

    def layer_norm(self, x, gamma, beta, y, mean, rstd, eps=1e-5, ckpt=None, stream=None):
        """y = gamma (x - mean) rstd + beta by row; gamma, beta, mean, rstd may
        be None.  ckpt (a Checkpoint) receives the normalised rows."""
        dev = self.device
        rows, cols = x.shape
        px, tx, ldx = _matrix("x", x, rows, cols, dev)
        py, ty, ldy = _matrix("y", y, rows, cols, dev)
        _lib.check(self.lib.ts_layer_norm(
            self.h, px, tx, ldx, rows, cols, _array("gamma", gamma, (cols,), dev), _array("beta", beta, (cols,), dev),
            eps, py, ty, ldy, _array("mean", mean, (rows,), dev), _array("rstd", rstd, (rows,), dev),
            _saved(ckpt, rows, cols, dev), self._stream(stream)))

    def layer_norm_backward(self, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, accumulate=False, stream=None):
        """The gradient, from x, or from the Checkpoint of the normalised rows
        in its place (mean may then be None).  dgamma and dbeta may be None."""
        dev = self.device
        rows, cols = dy.shape
        pdy, tdy, lddy = _matrix("dy", dy, rows, cols, dev)
        pdx, tdx, lddx = _matrix("dx", dx, rows, cols, dev)
        if isinstance(x, Checkpoint):
            px, tx, ldx, pc = None, FG_F32, cols, _saved(x, rows, cols, dev)
        else:
            px, tx, ldx = _matrix("x", x, rows, cols, dev)
            pc = None
        _lib.check(self.lib.ts_layer_norm_backward(
            self.h, pdy, tdy, lddy, px, tx, ldx, pc, rows, cols, _array("gamma", gamma, (cols,), dev),
            _array("mean", mean, (rows,), dev), _array("rstd", rstd, (rows,), dev), pdx, tdx, lddx,
            _array("dgamma", dgamma, (cols,), dev), _array("dbeta", dbeta, (cols,), dev), accumulate,
            self._stream(stream)))

    def checkpoint_save(self, x, ckpt, stream=None):
        """x in 8 bits into ckpt."""
        dev = self.device
        px, tx, ldx = _matrix("x", x, ckpt.rows, ckpt.cols, dev)
        _lib.check(self.lib.ts_checkpoint_save(self.h, px, tx, ldx, ckpt.rows, ckpt.cols, _buffer(ckpt, dev),
                                               self._stream(stream)))

    def checkpoint_load(self, ckpt, y, stream=None):
        """ckpt's values into y."""
        dev = self.device
        py, ty, ldy = _matrix("y", y, ckpt.rows, ckpt.cols, dev)
        _lib.check(self.lib.ts_checkpoint_load(self.h, _buffer(ckpt, dev), ckpt.rows, ckpt.cols, py, ty, ldy,
                                               self._stream(stream)))

    def activation_backward(self, op, dy, ckpt, dx, stream=None):
        """dx = dy f'(x) for op "relu", "sigmoid" or "tanh", from the
        checkpoint of the activation's output."""
        dev = self.device
        pdy, tdy, lddy = _matrix("dy", dy, ckpt.rows, ckpt.cols, dev)
        pdx, tdx, lddx = _matrix("dx", dx, ckpt.rows, ckpt.cols, dev)
        _lib.check(self.lib.ts_activation_backward(self.h, OPCODES[op], pdy, tdy, lddy, _buffer(ckpt, dev), ckpt.rows,
                                                   ckpt.cols, pdx, tdx, lddx, self._stream(stream)))

    def weight_grad(self, ckpt, dy, dw, db=None, gamma=None, beta=None, accumulate=False, stream=None):
        """dw = X^T dy, X the checkpoint's values, or gamma * values + beta by
        column; db (may be None) receives dy's column sums."""
        dev = self.device
        n = dy.shape[1]
        pdy, tdy, lddy = _matrix("dy", dy, ckpt.rows, n, dev)
        pdw, tdw, lddw = _matrix("dw", dw, ckpt.cols, n, dev)
        if tdw != FG_F32:
            raise FgError(FG_EINVAL, "dw: must be float32")
        _lib.check(self.lib.ts_weight_grad(
            self.h, _buffer(ckpt, dev), ckpt.rows, ckpt.cols, _array("gamma", gamma, (ckpt.cols,), dev),
            _array("beta", beta, (ckpt.cols,), dev), pdy, tdy, lddy, n, pdw, lddw, _array("db", db, (n,), dev),
            accumulate, self._stream(stream)))

    def token_logprobs(self, logits, tokens, logprob, entropy, lse, top_logprob=None, top_id=None, stream=None):
        """Log probabilities of tokens (int64), the entropy and log-sum-exp of
        every row, and the k most likely columns, k = top_id.shape[1].  Any
        output may be None."""
        dev = self.device
        rows, vocab = logits.shape
        p, t, ld = _matrix("logits", logits, rows, vocab, dev)
        k = 0 if top_id is None else top_id.shape[-1]
        if (top_id is None) != (top_logprob is None):
            raise FgError(FG_EINVAL, "top_logprob and top_id go together")
        _lib.check(self.lib.ts_token_logprobs(
            self.h, p, t, ld, rows, vocab, _array("tokens", tokens, (rows,), dev, torch.int64),
            _array("logprob", logprob, (rows,), dev), _array("entropy", entropy, (rows,), dev),
            _array("lse", lse, (rows,), dev), k, _array("top_logprob", top_logprob, (rows, k), dev),
            _array("top_id", top_id, (rows, k), dev, torch.int32), self._stream(stream)))

    def token_logprobs_backward(self, logits, tokens, lse, entropy, g_logprob, g_entropy, dlogits, stream=None):
        """dlogits from the gradients of logprob and (may be None) entropy."""
        dev = self.device
        rows, vocab = logits.shape
        p, t, ld = _matrix("logits", logits, rows, vocab, dev)
        pd, td, ldd = _matrix("dlogits", dlogits, rows, vocab, dev)
        _lib.check(self.lib.ts_token_logprobs_backward(
            self.h, p, t, ld, rows, vocab, _array("tokens", tokens, (rows,), dev, torch.int64),
            _array("lse", lse, (rows,), dev), _array("entropy", entropy, (rows,), dev),
            _array("g_logprob", g_logprob, (rows,), dev), _array("g_entropy", g_entropy, (rows,), dev), pd, td, ldd,
            self._stream(stream)))

    def embedding(self, ids, table, y, scale=1.0, stream=None):
        """y = scale * table[ids] (ids int64); an id outside the table gives
        zeros."""
        dev = self.device
        rows, cols = y.shape
        vocab = table.shape[0]
        pt, tt, ldt = _matrix("table", table, vocab, cols, dev)
        py, ty, ldy = _matrix("y", y, rows, cols, dev)
        _lib.check(self.lib.ts_embedding(self.h, _array("ids", ids, (rows,), dev, torch.int64), rows, pt, tt, ldt,
                                         vocab, cols, scale, py, ty, ldy, self._stream(stream)))

    def embedding_backward(self, ids, dy, dtable, scale=1.0, accumulate=False, stream=None):
        """The table's gradient: row v is scale times the sum of dy over the
        tokens of id v (in an order that the ids, the sizes and the workspace
        fix).  accumulate adds to what dtable holds."""
        dev = self.device
        rows, cols = dy.shape
        vocab = dtable.shape[0]
        pdy, tdy, lddy = _matrix("dy", dy, rows, cols, dev)
        pd, td, ldd = _matrix("dtable", dtable, vocab, cols, dev)
        _lib.check(self.lib.ts_embedding_backward(
            self.h, _array("ids", ids, (rows,), dev, torch.int64), pdy, tdy, lddy, rows, vocab, cols, scale, pd, td,
            ldd, accumulate, self._stream(stream)))

    def linear_cross_entropy(self, x, w, targets, loss, lse, stream=None):
        """Cross entropy of the logits x w^T with targets (int64), and their
        log-sum-exp, by row; the logits are not kept.  Either may be None."""
        dev = self.device
        rows, cols = x.shape
        vocab = w.shape[0]
        px, pw, ldx, ldw = _operands(x, w, rows, cols, vocab, dev)
        _lib.check(self.lib.ts_linear_cross_entropy(
            self.h, px, ldx, pw, ldw, FG_BF16, rows, cols, vocab, _array("targets", targets, (rows,), dev, torch.int64),
            _array("loss", loss, (rows,), dev), _array("lse", lse, (rows,), dev), self._stream(stream)))

    def linear_cross_entropy_backward(self, x, w, targets, lse, g_loss, dx, dw, g_lse=None, accumulate=False,
                                      stream=None):
        """dx and dw (either may be None) from the gradients of loss and (may
        be None) lse.  accumulate adds to what dw holds."""
        dev = self.device
        rows, cols = x.shape
        vocab = w.shape[0]
        px, pw, ldx, ldw = _operands(x, w, rows, cols, vocab, dev)
        pdx, tdx, lddx = (None, FG_BF16, cols) if dx is None else _matrix("dx", dx, rows, cols, dev)
        pdw, tdw, lddw = (None, FG_BF16, cols) if dw is None else _matrix("dw", dw, vocab, cols, dev)
        _lib.check(self.lib.ts_linear_cross_entropy_backward(
            self.h, px, ldx, pw, ldw, FG_BF16, rows, cols, vocab, _array("targets", targets, (rows,), dev, torch.int64),
            _array("lse", lse, (rows,), dev), _array("g_loss", g_loss, (rows,), dev),
            _array("g_lse", g_lse, (rows,), dev), pdx, tdx, lddx, pdw, tdw, lddw, accumulate, self._stream(stream)))


def _operands(x, w, rows, cols, vocab, device):
    """The bf16 operands of a product over the vocabulary."""
    px, tx, ldx = _matrix("x", x, rows, cols, device)
    pw, tw, ldw = _matrix("w", w, vocab, cols, device)
    if tx != FG_BF16 or tw != FG_BF16:
        raise FgError(FG_EINVAL, "x and w: must be bfloat16")
    return px, pw, ldx, ldw


def _buffer(ckpt, device):
    if ckpt.device != device:
        raise FgError(FG_EINVAL, "checkpoint: must be on the handle's CUDA device")
    return ckpt.ptr


def _saved(ckpt, rows, cols, device):
    if ckpt is None:
        return None
    if ckpt.rows != rows or ckpt.cols != cols:
        raise FgError(FG_ESHAPE, f"checkpoint: shape {(ckpt.rows, ckpt.cols)}, expected {(rows, cols)}")
    return _buffer(ckpt, device)
