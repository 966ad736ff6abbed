"""8-bit logit checkpoints (format: ``include/kld_stats.h``).

    >>> base = pack_logits(base_logits)              # 1.03 bytes an entry
    >>> st.run_grad_packed(base, quant_logits)       # every step of a tuning run

The base model's rows are written once and read by every later pass
(:meth:`KLDStats.run_packed`, :meth:`KLDStats.run_grad_packed`); the quant
rows of a deferred backward pass can be kept the same way. This module
marshals arguments; the arithmetic runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

PACK_BLOCK = _lib.KLD_PACK_BLOCK

_DTYPES = {torch.float32: _lib.KLD_F32, torch.bfloat16: _lib.KLD_BF16, torch.float16: _lib.KLD_F16}


# The current stream's handle by device index: 0.2 us, where the Stream object
# that torch.cuda.current_stream builds takes 2.5 us, a seventh of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(stream, device) -> int:
    """The handle of the stream to launch on."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError("the stream must be on the tensors' device")
    return stream.cuda_stream


def _empty(stream, shape, dtype, device) -> torch.Tensor:
    """An output for a call on ``stream`` (None: the current one), allocated
    in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class PackedLogits:
    """[N, vocab] logits in 8 bits: ``codes`` [N, blocks * 128] uint8 and
    ``heads`` [N, blocks] int32, blocks = ceil(vocab / 128), both contiguous
    and on one device. A header is ``base << 9 | (some code is 0) << 8 |
    (e + 128)``; an entry is ``(base + code) * 2**e``, or -inf where its code
    is 0. ``rows(start, stop)`` gives views, so one large store can be filled
    and read in parts."""

    def __init__(self, codes: torch.Tensor, heads: torch.Tensor, vocab: int):
        vocab = int(vocab)
        blocks = -(-vocab // PACK_BLOCK)
        if vocab < 1 or codes.dim() != 2 or heads.dim() != 2:
            raise ValueError("codes and heads must be matrices and vocab positive")
        if codes.dtype != torch.uint8 or heads.dtype != torch.int32:
            raise TypeError("codes must be uint8 and heads int32")
        if codes.shape[1] != blocks * PACK_BLOCK or heads.shape[1] != blocks or codes.shape[0] != heads.shape[0]:
            raise ValueError(f"{vocab} columns take codes [N, {blocks * PACK_BLOCK}] and heads [N, {blocks}]")
        if not (codes.is_contiguous() and heads.is_contiguous()):
            raise ValueError("codes and heads must be contiguous")
        if codes.device != heads.device:
            raise ValueError("codes and heads must be on one device")
        if codes.data_ptr() % 16:
            raise ValueError("codes must be aligned to 16 bytes")
        self._hold(codes, heads, vocab)

    def _hold(self, codes: torch.Tensor, heads: torch.Tensor, vocab: int) -> "PackedLogits":
        self.codes, self.heads, self.vocab = codes, heads, vocab
        self.shape = (codes.shape[0], vocab)
        self.device = codes.device
        self._c = _lib.Packed(codes.data_ptr(), heads.data_ptr())
        return self

    @classmethod
    def empty(cls, n_rows: int, vocab: int, device=None) -> "PackedLogits":
        """An unwritten store for ``n_rows`` rows."""
        blocks = -(-int(vocab) // PACK_BLOCK)
        device = torch.device("cuda") if device is None else device
        return cls(torch.empty((n_rows, blocks * PACK_BLOCK), dtype=torch.uint8, device=device),
                   torch.empty((n_rows, blocks), dtype=torch.int32, device=device), vocab)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.heads.numel()

    def __len__(self) -> int:
        return self.codes.shape[0]

    def rows(self, start: int, stop: int) -> "PackedLogits":
        """Rows [start, stop) as a view."""
        if not 0 <= start <= stop <= len(self):
            raise ValueError("need 0 <= start <= stop <= rows")
        return PackedLogits(self.codes[start:stop], self.heads[start:stop], self.vocab)

    def to(self, device) -> "PackedLogits":
        """The same store on another device (a copy; the host counts too)."""
        return PackedLogits(self.codes.to(device), self.heads.to(device), self.vocab)

    def unpack(self, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        """The stored values as [N, vocab] logits: exact in float32, rounded
        to nearest in the 16-bit types. Asynchronous on the stream."""
        lib = _lib.load()
        if not self.codes.is_cuda:
            raise ValueError("the checkpoint must be on a CUDA device")
        s = _on(stream, self.device)
        if out is None:
            out = _empty(stream, self.shape, dtype, self.device)
        if out.dtype not in _DTYPES:
            raise TypeError(f"unsupported logit dtype {out.dtype}")
        if out.shape != self.shape or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out must be a contiguous [N, vocab] tensor on the checkpoint's device")
        if len(self):
            _lib.check(lib.kld_unpack_logits(ctypes.byref(self._c), len(self), self.vocab,
                                             out.data_ptr(), _DTYPES[out.dtype], self.device.index, s),
                       "kld_unpack_logits")
        return out


def pack_logits(logits: torch.Tensor, out: PackedLogits | None = None, stream=None,
                mask_at: float | None = None) -> PackedLogits:
    """The 8-bit checkpoint of contiguous [N, V] CUDA logits (float32,
    bfloat16 or float16), written to ``out`` (for instance ``store.rows(a, b)``)
    or to a new one. Asynchronous on the stream.

    Every block of 128 columns has one step, about 1/254 of what its entries
    span (-inf apart). So logits masked with a finite value need ``mask_at``:
    entries at or below it (as the logits' type holds it) are stored as -inf.
    Without it a mask of -1e9 leaves nothing of its block's other entries, and
    one of 2^126 or more in magnitude (``torch.finfo(dtype).min`` of float32
    and bfloat16) makes the row NONFINITE to the statistic."""
    lib = _lib.load()
    if logits.dtype not in _DTYPES:
        raise TypeError(f"unsupported logit dtype {logits.dtype}")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be a [N, V] tensor")
    if not logits.is_cuda or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA tensor")
    s = _on(stream, logits.device)
    if out is None:
        n, blocks = logits.shape[0], -(-logits.shape[1] // PACK_BLOCK)
        out = PackedLogits.__new__(PackedLogits)._hold(  # made to fit: no checks
            _empty(stream, (n, blocks * PACK_BLOCK), torch.uint8, logits.device),
            _empty(stream, (n, blocks), torch.int32, logits.device), logits.shape[1])
    elif out.shape != tuple(logits.shape) or out.device != logits.device:
        raise ValueError("out must hold as many rows and columns on the logits' device")
    if len(out) and mask_at is None:
        _lib.check(lib.kld_pack_logits(logits.data_ptr(), logits.shape[0], logits.shape[1],
                                       _DTYPES[logits.dtype], ctypes.byref(out._c), logits.device.index, s),
                   "kld_pack_logits")
    elif len(out):
        _lib.check(lib.kld_pack_logits_masked(logits.data_ptr(), logits.shape[0], logits.shape[1],
                                              _DTYPES[logits.dtype], float(mask_at), ctypes.byref(out._c),
                                              logits.device.index, s), "kld_pack_logits_masked")
    return out
