"""Arguments of the logit checkpoints and of beam search are refused before
any GPU work. Runs without a GPU."""
import ctypes

import pytest
import torch

from logit_kl_divergence_b200 import _lib, PackedLogits, pack_logits
from logit_kl_divergence_b200.beam import BeamStates, _apart, _describe, _span

INVALID, DTYPE = _lib.KLD_ERR_INVALID_ARG, _lib.KLD_ERR_DTYPE
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _pk(codes=P, heads=P):
    return ctypes.byref(_lib.Packed(codes, heads))


def test_pack_and_unpack_refuse(lib):
    x = ctypes.c_void_p(P)
    for f in (lambda n=4, v=8, dt=0, x=x, pk=_pk(), dev=0: lib.kld_pack_logits(x, n, v, dt, pk, dev, None),
              lambda n=4, v=8, dt=0, x=x, pk=_pk(), dev=0: lib.kld_unpack_logits(pk, n, v, x, dt, dev, None)):
        assert f(n=0) == INVALID and f(v=0) == INVALID and f(v=1 << 31) == INVALID
        assert f(n=1 << 60) == INVALID and f(dt=3) == DTYPE and f(dev=-1) == INVALID
        assert f(x=None) == INVALID and f(x=ctypes.c_void_p(P + 2)) == INVALID
        assert f(pk=None) == INVALID and f(pk=_pk(codes=None)) == INVALID
        assert f(pk=_pk(heads=None)) == INVALID and f(pk=_pk(codes=P + 8)) == INVALID
        assert f(pk=_pk(heads=P + 2)) == INVALID


def test_pack_and_unpack_refuse_memory_that_overlaps(lib):
    # 4 rows of 8 columns: 512 bytes of codes, 16 of headers, 128 of logits
    at = lambda k: ctypes.c_void_p(P + k)
    for f in (lambda x, c, h: lib.kld_pack_logits(at(x), 4, 8, 0, _pk(P + c, P + h), 1 << 20, None),
              lambda x, c, h: lib.kld_unpack_logits(_pk(P + c, P + h), 4, 8, at(x), 0, 1 << 20, None)):
        assert f(0, 112, 4096) == INVALID and f(508, 0, 4096) == INVALID and f(0, 0, 4096) == INVALID
        assert f(0, 1024, 124) == INVALID and f(0, 1024, 1532) == INVALID and f(1552, 1024, 1540) == INVALID
        if not torch.cuda.is_available():  # apart: only the device is missing
            assert f(0, 128, 640) == _lib.KLD_ERR_NO_DEVICE and f(528, 0, 512) == _lib.KLD_ERR_NO_DEVICE


def test_packed_runs_and_beams_refuse_a_null_handle(lib):
    x = ctypes.c_void_p(P)
    assert lib.kld_stats_run_packed(None, _pk(), x, 0, None, None, 1, 1, None, None) == INVALID
    assert lib.kld_stats_run_grad_packed(None, _pk(), x, 0, None, None, 1, 1, x, 0, 1.0, None, None) == INVALID
    assert lib.kld_beam_select(None, x, 1, 0, x, None, 0, 1, 1, 1, 1, x, x, x, None) == INVALID
    assert lib.kld_beam_reorder(None, None, 0, x, None, 1, 1, None) == INVALID
    assert lib.kld_beam_status(None, ctypes.byref(ctypes.c_uint32())) == INVALID
    lib.kld_beam_destroy(None)


def test_beam_create_refuses_sizes(lib):
    h = ctypes.c_void_p()
    assert lib.kld_beam_create(None, 1, 1, 1, 0) == INVALID
    for groups, beams, k, dev in ((0, 1, 1, 0), (1, 0, 1, 0), (1, 65, 1, 0), (1, 1, 0, 0), (1, 1, 129, 0),
                                  (1, 1, 1, -1), (1 << 24, 2, 1, 0)):
        assert lib.kld_beam_create(ctypes.byref(h), groups, beams, k, dev) == INVALID
    if not torch.cuda.is_available():
        assert lib.kld_beam_create(ctypes.byref(h), 1, 1, 1, 0) == _lib.KLD_ERR_NO_DEVICE


def test_packed_logits_checks_its_tensors():
    c, h = torch.zeros((3, 256), dtype=torch.uint8), torch.zeros((3, 2), dtype=torch.int32)
    p = PackedLogits(c, h, 200)
    assert p.shape == (3, 200) and len(p) == 3 and p.nbytes == 3 * 256 + 24
    assert p.rows(1, 3).shape == (2, 200) and p.rows(2, 2).shape == (0, 200)
    assert p.rows(1, 3).codes.data_ptr() == c[1].data_ptr()
    for bad in ((c, h, 128), (c, h, 257), (c, h, 0), (c[:2], h, 200), (c.t(), h, 200)):
        with pytest.raises(ValueError):
            PackedLogits(*bad)
    with pytest.raises(TypeError):
        PackedLogits(c.int(), h, 200)
    with pytest.raises(TypeError):
        PackedLogits(c, h.long(), 200)
    with pytest.raises(ValueError):
        p.rows(2, 4)
    with pytest.raises(ValueError):
        p.unpack()  # not on a GPU
    with pytest.raises(ValueError):
        pack_logits(torch.zeros((2, 3)))
    with pytest.raises(TypeError):
        pack_logits(torch.zeros((2, 3), dtype=torch.float64))


class _Cuda:
    """A tensor's layout without its memory, for the host's description."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def _runs(t, time_dim):
    s = _describe(_Cuda(t), time_dim)
    return s.row_stride, s.outer, s.outer_stride, s.positions, s.position_bytes, s.timed


def test_states_are_described_as_runs():
    x = torch.zeros((6, 3, 10, 4))
    assert _runs(x, 2) == (480, 3, 160, 10, 16, 1)
    assert _runs(x, None) == (480, 1, 0, 1, 480, 0)
    assert _runs(x, 1) == (480, 1, 0, 3, 160, 1)
    y = torch.zeros((6, 10, 3, 4))
    assert _runs(y.transpose(1, 2), 2) == (480, 1, 0, 10, 48, 1)  # heads seen before time
    assert _runs(x[:, :, :7], 2) == (480, 3, 160, 7, 16, 1)       # part of a longer cache
    assert _runs(x[:, 1], 1) == (480, 1, 0, 10, 16, 1)
    assert _runs(torch.zeros((5,), dtype=torch.bfloat16), None) == (2, 1, 0, 1, 2, 0)
    assert _runs(torch.zeros((4, 0)), None)[3:5] == (0, 0)
    for bad, d in ((x[..., ::2], 2), (x[:, :, ::2], 2), (x.transpose(2, 3), 2), (x.transpose(1, 2), 1), (x, 0), (x, 4),
                   (x[:, :, :, :3], None)):
        with pytest.raises(ValueError):
            _describe(_Cuda(bad), d)


def test_bound_states_are_checked():
    with pytest.raises(ValueError):
        BeamStates([torch.zeros((2, 3))], torch.device("cpu"))  # not CUDA tensors
    with pytest.raises(ValueError):
        BeamStates([torch.zeros((2, 3)), torch.zeros((3, 3))], torch.device("cpu"))


def test_states_that_share_memory_are_told_from_those_that_interleave():
    def pair(x, y, dx=None, dy=None):
        x, y = _Cuda(x), _Cuda(y)
        return _apart((_span(x), _describe(x, dx), x.shape[0]), (_span(y), _describe(y, dy), y.shape[0]))

    kv = torch.zeros((6, 3, 2, 10, 4))       # rows, heads, k or v, time, dim
    assert pair(kv[:, :, 0], kv[:, :, 1], 2, 2) and pair(kv[:, 0, 0], kv[:, 1, 1], 1, 1)
    assert pair(kv[:, 0], kv[:, 1:], 2, None) and pair(kv[:3], kv[3:], 3, 3)
    assert not pair(kv[:, :, 0], kv[:, :, 0], 2, 2) and not pair(kv[:, :, 0, :6], kv[:, :, 0, 4:], 2, 2)
    assert pair(kv[:, :, 0, :6], kv[:, :, 0, 6:], 2, 2) and not pair(kv, kv[:, 2], 3, 2)
    assert not pair(kv[:, :, 0], kv[:, 0, 0], 2, 1) and not pair(kv[:4], kv[1:5], 3, 3)
    one = kv[:1]
    assert pair(one[:, :, 0], one[:, :, 1], 2, 2) and not pair(one[:, :, 0], one[:, :, 0, 1:], 2, 2)
    t = torch.zeros((3, 6, 2, 10, 4)).transpose(0, 1)  # rows between the runs of a head
    assert pair(t[:, :, 0], t[:, :, 1], 2, 2) and not pair(t[:, :, 0], t[:, :, 0, 2:], 2, 2)
    flat = torch.zeros(64)
    assert not pair(flat[:60].view(6, 10), flat[4:64].view(12, 5)[:6])
    assert pair(flat[:30].view(6, 5), flat[30:60].view(6, 5))


def test_masked_pack_refuses(lib):
    x = ctypes.c_void_p(P)
    f = lambda m, dt=0, pk=_pk(4 * P, 8 * P): lib.kld_pack_logits_masked(x, 4, 8, dt, m, pk, 1 << 20, None)
    assert f(float("nan")) == INVALID and f(float("inf")) == INVALID
    assert f(-1e9, dt=3) == DTYPE and f(-1e9, pk=None) == INVALID and f(-1e9, pk=_pk()) == INVALID
    if not torch.cuda.is_available():
        for m in (-1e9, 0.0, float("-inf")):
            assert f(m) == _lib.KLD_ERR_NO_DEVICE


def test_what_a_state_holds_is_told_from_the_gaps_in_it():
    """parents and lengths may lie between a state's rows or runs."""
    buf = torch.zeros((4, 3, 6, 10))                 # rows, heads, time, dim
    state = buf[:, :, :4]                            # two positions of every run are free

    def held(t, where):
        s = BeamStates.__new__(BeamStates)
        s.tensors, s.rows = [_Cuda(t)], t.shape[0]
        s.spans, s.layouts = [_span(t)], [_describe(_Cuda(t), 2 if t.dim() == 4 else None)]
        return s.hold(where)

    for r in range(4):
        for h in range(3):
            run = buf[r, h].view(-1)
            assert not held(state, run[40:60]) and held(state, run[39:60])
            assert held(state, run[:1]) and held(state, run[20:24])
            assert not held(buf[:, :2], run[:]) if h == 2 else held(buf[:, :2], run[:1])
            assert held(state, buf.view(-1)[(r * 3 + h) * 60 + 59 - (59 if (r, h) == (3, 2) else 0):][:2])
    assert not held(buf[1:3].view(2, -1), buf[3, 0, 0, :4]) and not held(buf[1:3].view(2, -1), buf[0, 2, 5, 6:])
    assert held(buf[1:3].view(2, -1), buf[2, 2, 5, 6:])
    one = buf[:1, :1]                                # one row, one run
    assert not held(one, buf[0, 1, 0]) and held(one, buf[0, 0, 5, 9:])
