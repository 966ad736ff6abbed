"""Beam search over logit rows: selection and the reordering of states.

    >>> beam = BeamSearch(max_groups=16, max_beams=8)
    >>> states = beam.bind([(k_cache, 2), (v_cache, 2), (tokens, 1)])
    >>> scores, token, parent = beam.select(logits, scores, k=8)
    >>> beam.reorder(states, parent, lengths)         # in place

This module marshals arguments; the arithmetic runs in the library's CUDA
kernels (``include/kld_stats.h``: kld_beam_select, kld_beam_reorder).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .packed import _DTYPES, _empty, _on


def _ptr(t):
    return None if t is None else t.data_ptr()


def _span(t: torch.Tensor) -> tuple[int, int]:
    """Addresses [first, past the last) that a tensor's entries lie in."""
    if t.numel() == 0:
        return t.data_ptr(), t.data_ptr()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(a: tuple, b: tuple) -> bool:
    """Whether two states (span, layout, row count) share no byte. Layouts
    that interleave are told apart by the strides they have in common; states
    that this cannot show to be apart count as overlapping."""
    (x0, x1), s, rows = a
    (y0, y1), t, _ = b
    if x1 <= y0 or y1 <= x0:
        return True
    run_s, run_t = s.positions * s.position_bytes, t.positions * t.position_bytes

    def between(period, len_s, len_t):
        gap = (y0 - x0) % period  # from s on to the next t, and from there to the next s
        return gap >= len_s and period - gap >= len_t

    if rows > 1 and s.row_stride == t.row_stride:
        len_s = (s.outer - 1) * s.outer_stride + run_s
        len_t = (t.outer - 1) * t.outer_stride + run_t
        if between(s.row_stride, len_s, len_t):
            return True
    # all runs of both start whole multiples of their strides' common divisor apart
    steps = [u.row_stride for u in (s, t) if rows > 1] + [u.outer_stride for u in (s, t) if u.outer > 1]
    period = math.gcd(*steps)
    return period > 0 and between(period, run_s, run_t)


def _describe(t: torch.Tensor, time_dim: int | None) -> _lib.State:
    """A state's layout as runs of contiguous positions."""
    if not t.is_cuda or t.dim() < 1:
        raise ValueError("states must be CUDA tensors with one row per beam first")
    size = t.element_size()
    if t.numel() == 0:
        return _lib.State(t.data_ptr(), 0, 0, 0, 0, 0, 0, 0)
    d = 1 if time_dim is None else int(time_dim)
    if time_dim is not None and not 1 <= d < t.dim():
        raise ValueError("time_dim must be a dimension of the state other than the first")

    def joined(dims):
        """(count, stride) of dims (outermost first) that step as one."""
        count, stride = 1, 0
        for i in reversed(dims):
            if t.shape[i] == 1:
                continue
            if count == 1:
                stride = t.stride(i)
            elif t.stride(i) != count * stride:
                raise ValueError("a state's dimensions must be laid out in order")
            count *= t.shape[i]
        return count, stride

    if time_dim is None:
        positions, time_stride = 1, 0
        outer, outer_stride = 1, 0
        inner, inner_stride = joined(range(1, t.dim()))
    else:
        positions, time_stride = t.shape[d], t.stride(d)
        outer, outer_stride = joined(range(1, d))
        inner, inner_stride = joined(range(d + 1, t.dim()))
    if inner > 1 and inner_stride != 1:
        raise ValueError("the entries of a position must be contiguous")
    if positions > 1 and time_stride != inner:
        # [rows, heads, time, dim] viewed from [rows, time, heads, dim]: a
        # position's runs of all heads lie together
        if outer > 1 and outer_stride == inner and time_stride == outer * inner:
            inner, outer, outer_stride = outer * inner, 1, 0
        else:
            raise ValueError("positions must follow one another in memory")
    row = t.stride(0) * size if t.shape[0] > 1 else 0
    return _lib.State(t.data_ptr(), row, outer, outer_stride * size, positions, inner * size,
                      0 if time_dim is None else 1, 0)


def _holds(s: _lib.State, rows: int, a: int, b: int) -> bool:
    """Whether a state's runs hold any of the bytes [a, b), counted from its
    first one."""
    run = s.positions * s.position_bytes
    for r in range(rows if s.row_stride else 1):
        first = a - run - r * s.row_stride + 1  # the lowest start of a run that reaches a
        i = max(0, -(-first // s.outer_stride)) if s.outer > 1 else (0 if first <= 0 else 1)
        if i < s.outer and r * s.row_stride + i * s.outer_stride < b:
            return True
    return False


class BeamStates:
    """States that :meth:`BeamSearch.reorder` moves together, described once
    (it holds the tensors, whose memory must stay where it is)."""

    def __init__(self, states, device: torch.device):
        items = [s if isinstance(s, tuple) else (s, None) for s in states]
        self.tensors = [t for t, _ in items]
        rows = {t.shape[0] for t in self.tensors if t.dim()}
        if len(rows) > 1:
            raise ValueError("states must have the same number of rows")
        self.rows = rows.pop() if rows else None
        if any(t.device != device for t in self.tensors):
            raise ValueError("states must be on the handle's device")
        self.spans = [_span(t) for t in self.tensors]
        self.layouts = layouts = [_describe(t, d) for t, d in items]
        order = sorted(((span, layout, self.rows) for span, layout in zip(self.spans, layouts)
                        if span[0] < span[1]), key=lambda a: a[0])
        for i, a in enumerate(order):
            for b in order[i + 1:]:
                if b[0][0] >= a[0][1]:
                    break
                if not _apart(a, b):
                    raise ValueError("states may not overlap one another")
        self._c = (_lib.State * max(1, len(items)))(*layouts)

    def __len__(self) -> int:
        return len(self.tensors)

    def hold(self, t: torch.Tensor) -> bool:
        """Whether a contiguous tensor shares memory with a state (the gaps
        between a state's runs are not its own)."""
        a = t.data_ptr()
        b = a + t.numel() * t.element_size()
        for i, (x, y) in enumerate(self.spans):
            if a < y and x < b and _holds(self.layouts[i], self.rows, a - x, b - x):
                return True
        return False


class BeamSearch:
    """One handle of the library: workspace for selections of up to
    ``max_k`` candidates (default twice the beams) from ``max_groups`` groups
    of ``max_beams`` beams. Not thread-safe; use one per concurrent stream."""

    def __init__(self, max_groups: int, max_beams: int, max_k: int | None = None, device=None):
        self._lib = _lib.load()
        if device is None:
            device = torch.cuda.current_device()
        index = device if isinstance(device, int) else torch.device(device).index
        self.device = torch.device("cuda", torch.cuda.current_device() if index is None else index)
        self.max_groups, self.max_beams = int(max_groups), int(max_beams)
        self.max_k = min(_lib.KLD_BEAM_MAX_K, 2 * self.max_beams) if max_k is None else int(max_k)
        h = ctypes.c_void_p()
        _lib.check(self._lib.kld_beam_create(ctypes.byref(h), self.max_groups, self.max_beams, self.max_k,
                                             self.device.index), "kld_beam_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            self._lib.kld_beam_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def select(self, logits: torch.Tensor, scores: torch.Tensor, k: int,
               finished: torch.Tensor | None = None, eos: int | None = None,
               out: tuple | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """One step: of every group the ``k`` best continuations
        ``scores[g, w] + log_softmax(logits[g * beams + w])[j]``, best first,
        ties to the lowest ``w * V + j``.

        ``logits`` [groups * beams, V] (rows may be further apart than V),
        ``scores`` [groups, beams] float32 (-inf: no such beam); ``finished``
        [groups, beams] bool: those beams offer only token ``eos`` at their
        own score. Returns (or writes to ``out``) scores float32, tokens and
        parents int32, each [groups, k]; places without a candidate hold
        -inf, -1, -1. Asynchronous on the stream; see :meth:`status`."""
        if scores.dim() != 2 or scores.dtype != torch.float32 or not scores.is_contiguous():
            raise ValueError("scores must be a contiguous float32 [groups, beams] tensor")
        groups, beams = scores.shape
        if logits.dim() != 2 or logits.shape[0] != groups * beams:
            raise ValueError("logits must be a [groups * beams, V] tensor")
        if logits.dtype not in _DTYPES:
            raise TypeError(f"unsupported logit dtype {logits.dtype}")
        if logits.device != self.device or scores.device != self.device:
            raise ValueError("logits and scores must be on the handle's device")
        if (logits.shape[1] > 1 and logits.stride(1) != 1) or (
                logits.shape[0] > 1 and logits.stride(0) < logits.shape[1]):
            raise ValueError("logits rows must be contiguous and apart")
        if finished is not None:
            if finished.shape != scores.shape or finished.dtype not in (torch.bool, torch.uint8):
                raise ValueError("finished must be a bool [groups, beams] tensor")
            if finished.device != self.device or not finished.is_contiguous():
                raise ValueError("finished must be contiguous and on the handle's device")
            if eos is None or not 0 <= int(eos) < logits.shape[1]:  # before it is cut to 32 bits
                raise ValueError("finished beams need eos, a token of the vocabulary")
        s = _on(stream, self.device)
        k = int(k)
        if out is None:
            # one allocation: scores, tokens, parents
            top, tokens, parents = _empty(stream, (3, groups, k), torch.int32, self.device).unbind(0)
            out = (top.view(torch.float32), tokens, parents)
        else:
            for t, dt in zip(out, (torch.float32, torch.int32, torch.int32)):
                if t.shape != (groups, k) or t.dtype != dt or t.device != self.device or not t.is_contiguous():
                    raise ValueError("out must be contiguous float32, int32 and int32 [groups, k] tensors")
        ld = logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]
        _lib.check(self._lib.kld_beam_select(self._h, logits.data_ptr(), ld, _DTYPES[logits.dtype],
                                             scores.data_ptr(), _ptr(finished), 0 if finished is None else int(eos),
                                             groups, beams, logits.shape[1], k, out[0].data_ptr(),
                                             out[1].data_ptr(), out[2].data_ptr(), s), "kld_beam_select")
        return out

    def bind(self, states) -> BeamStates:
        """Describe the states of :meth:`reorder` once: tensors with one row
        per beam first, or (tensor, time_dim) pairs for those that lengths
        apply to. A position's entries must be contiguous and the positions
        of a run follow one another ([rows, heads, time, dim] and
        [rows, time, heads, dim] both do)."""
        return BeamStates(states, self.device)

    def reorder(self, states, parents: torch.Tensor, lengths: torch.Tensor | None = None,
                stream=None) -> None:
        """In place, beam w of group g takes over the states of beam
        ``parents[g, w]`` (int32 [groups, beams]; -1 leaves a beam as it is).
        ``lengths`` (int32, one per row): of the states with a time dimension
        only the parent's first ``lengths`` positions are copied, what lies
        behind stays as it was. ``states``: what :meth:`bind` gave, or what it
        takes. Asynchronous on the stream."""
        if not isinstance(states, BeamStates):
            states = self.bind(states)
        if parents.dim() != 2 or parents.dtype != torch.int32 or not parents.is_contiguous():
            raise ValueError("parents must be a contiguous int32 [groups, beams] tensor")
        rows = parents.shape[0] * parents.shape[1]
        if states.rows is not None and states.rows != rows:
            raise ValueError("states must have groups * beams rows")
        if lengths is not None and (lengths.dtype != torch.int32 or lengths.numel() != rows
                                    or not lengths.is_contiguous()):
            raise ValueError("lengths must be a contiguous int32 tensor with one value per row")
        for t in (parents, lengths):
            if t is None:
                continue
            if t.device != self.device:
                raise ValueError("parents and lengths must be on the handle's device")
            if states.hold(t):
                raise ValueError("parents and lengths may not lie in a state")
        _lib.check(self._lib.kld_beam_reorder(self._h, states._c, len(states.tensors), parents.data_ptr(),
                                              _ptr(lengths), parents.shape[0], parents.shape[1],
                                              _on(stream, self.device)), "kld_beam_reorder")

    def status(self) -> int:
        """Wait for this handle's last call and return (and clear) the
        ``BEAM_*`` bits its calls met: rows without a usable logit
        (BEAM_NONFINITE), NaN or +inf scores (BEAM_BAD_SCORE), parents
        outside the group (BEAM_BAD_PARENT)."""
        flags = ctypes.c_uint32()
        _lib.check(self._lib.kld_beam_status(self._h, ctypes.byref(flags)), "kld_beam_status")
        return flags.value
