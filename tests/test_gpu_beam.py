"""Beam search's selection and the reordering of its states on the GPU.

Selection: tokens and parents equal those of a 64-bit implementation (stable
sort: ties to the lowest beam * V + token); scores within one fp32 rounding
(2^-24 |s|) of it plus 2e-6, the fp32 part of a row's log-sum-exp: arguments
(x - m) L are rounded by 2^-23 |x - m| where the weight is e^-|x - m| (at most
0.4 * 2^-23 together), ex2.approx 2^-22, and a thread's sum of a few hundred
terms 2^-24 an addition (1.5e-6 for 25 tiles in the worst case).
Reordering copies bytes: equal to an indexed copy."""
import math

import numpy as np
import pytest
import torch

import packed_ref
from logit_kl_divergence_b200 import (BEAM_BAD_PARENT, BEAM_BAD_SCORE, BEAM_NONFINITE, BeamSearch,
                                      KLDError, KLDStats, PackedLogits, _lib, pack_logits)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _rows(rows, v, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, v), generator=g) * 2.5
    x[torch.arange(rows), torch.randint(0, v, (rows,), generator=g)] += 6.0
    return x


def _scores(groups, beams, seed):
    g = torch.Generator().manual_seed(seed)
    return -20.0 * torch.rand((groups, beams), generator=g)


def _check(x, scores, k, finished=None, eos=None, beam=None, logits=None):
    groups, beams = scores.shape
    own = beam is None
    beam = beam or BeamSearch(groups, beams, max_k=max(k, 1), device=DEV)
    got = beam.select(x.to(DEV) if logits is None else logits, scores.to(DEV), k,
                      finished=None if finished is None else finished.to(DEV), eos=eos)
    s, t, p = (z.cpu().numpy() for z in got)
    ws, wt, wp = packed_ref.select(x.float().numpy(), scores.numpy(), k,
                                   None if finished is None else finished.numpy(), eos or 0)
    assert np.array_equal(t, wt) and np.array_equal(p, wp)
    none = np.isneginf(ws)
    assert np.array_equal(np.isneginf(s), none)
    d = np.abs(np.where(none, 0.0, s.astype(np.float64)) - np.where(none, 0.0, ws))
    assert (d <= 2.0 ** -24 * np.abs(np.where(none, 0.0, ws)) + 2e-6).all(), d.max()
    if own:
        beam.close()
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("groups,beams,v,k", [(1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 5, 20), (1, 4, 32000, 8),
                                              (3, 5, 4099, 10), (8, 8, 1000, 16), (2, 64, 333, 128),
                                              (5, 2, 70001, 4), (40, 4, 9001, 8), (1, 16, 151936, 32)])
def test_selection(dtype, groups, beams, v, k):
    _check(_rows(groups * beams, v, v + k).to(DTYPES[dtype]), _scores(groups, beams, v), k)


def test_first_step_and_dead_beams():
    s = torch.full((3, 4), -math.inf)
    s[0, 0], s[1, 2] = 0.0, -1.5
    x = _rows(12, 5000, 1)
    _check(x, s, 8)  # group 2 has no beam at all
    x[0] = math.nan  # a dead beam's row is not looked at ...
    s[0] = torch.tensor([-math.inf, -2.0, -math.inf, -math.inf])
    with BeamSearch(3, 4, device=DEV) as beam:
        _check(x, s, 8, beam=beam)
        assert beam.status() == 0


def test_finished_beams_offer_their_eos():
    x, s = _rows(4 * 6, 2500, 2), _scores(4, 6, 3)
    done = torch.rand((4, 6), generator=torch.Generator().manual_seed(1)) < 0.5
    done[3] = True
    for k in (6, 12):
        _check(x, s, k, finished=done, eos=2)
    s[:, 1] = -math.inf
    _check(x, s, 12, finished=done, eos=2499)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ties_go_to_the_lowest_index(dtype):
    dt = DTYPES[dtype]
    x = torch.zeros((6, 12000))
    _check(x.to(dt), torch.zeros((2, 3)), 6)       # everything ties
    x[1, 4000:] = 1.0                              # 8000 ties at a row's top
    x[4, ::2] = 1.0
    _check(x.to(dt), torch.zeros((2, 3)), 6)
    y = _rows(1, 3000, 9).expand(4, 3000).contiguous()
    _check(y.to(dt), torch.full((1, 4), -3.0), 8)  # equal beams


def test_rising_and_falling_rows():
    x = torch.arange(20000).float().mul(1e-3).expand(4, 20000).clone()
    x[1] = x[1].flip(0)
    _check(x, _scores(1, 4, 5), 8)
    _check(x, _scores(2, 2, 5), 4)


def test_masks_and_bad_rows():
    x, s = _rows(8 * 2, 3000, 4), _scores(8, 2, 4)
    x[0, 10:] = -math.inf                            # fewer tokens than k
    x[1] = -math.inf
    x[2], x[3] = -math.inf, -math.inf                # a group with nothing to offer
    x[4, 100] = math.nan
    x[6, 5] = math.inf
    x[8] = torch.finfo(torch.float32).min            # the type's lowest value everywhere: uniform
    x[10, 7:] = torch.finfo(torch.float32).min
    x[12] = torch.finfo(torch.float32).min
    x[12, 2999] = 3.0
    with BeamSearch(8, 2, max_k=16, device=DEV) as beam:
        _check(x, s, 16, beam=beam)
        assert beam.status() == BEAM_NONFINITE
        assert beam.status() == 0
        s[7, 0], s[6, 1] = math.nan, math.inf
        _check(x, s, 4, beam=beam)
        assert beam.status() == BEAM_NONFINITE | BEAM_BAD_SCORE
        b = x.bfloat16()
        b[8] = torch.finfo(torch.bfloat16).min
        _check(b, _scores(8, 2, 4), 4, beam=beam)


def test_rows_apart_and_at_any_alignment():
    for dtype in DTYPES.values():
        x = _rows(6, 1003, 6).to(dtype)
        for shift, ld in ((0, 1003), (1, 1010), (3, 1024), (5, 2000)):
            flat = torch.full((shift + 6 * ld,), math.nan, dtype=dtype, device=DEV)
            view = torch.as_strided(flat, (6, 1003), (ld, 1), shift)
            view.copy_(x)
            _check(x, _scores(2, 3, 1), 6, logits=view)


def test_two_calls_replays_and_another_stream():
    x, s = _rows(4 * 4, 40000, 11).bfloat16().to(DEV), _scores(4, 4, 8).to(DEV)
    with BeamSearch(4, 4, device=DEV) as beam:
        want = [t.clone() for t in beam.select(x, s, 8)]
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(beam.select(x, s, 8), want))
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        got = beam.select(x, s, 8, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        moving = x.clone()
        with torch.cuda.graph(graph):
            out = beam.select(moving, s, 8)
        moving.copy_(x.flip(1))
        graph.replay()
        torch.cuda.synchronize()
        flipped = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(beam.select(x.flip(1).contiguous(), s, 8), flipped))
        moving.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# -------------------------------------------------------------- reordering

def _reorder(states, parents, lengths=None):
    """states: [(cpu tensor, time_dim or None)]."""
    groups, beams = parents.shape
    dev = [(t.to(DEV), d) for t, d in states]
    with BeamSearch(groups, beams, device=DEV) as beam:
        beam.reorder(dev, parents.to(DEV), None if lengths is None else lengths.to(DEV))
        flags = beam.status()
    for (t, d), (got, _) in zip(states, dev):
        want = packed_ref.reorder(t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.numpy(),
                                  parents.numpy(), None if lengths is None else lengths.numpy(), d)
        got = got.cpu()
        got = (got.view(torch.int16) if t.dtype == torch.bfloat16 else got).numpy()
        assert np.array_equal(got, want)
    return flags


@pytest.mark.parametrize("groups,beams", [(1, 1), (1, 2), (3, 4), (2, 5), (2, 8), (1, 13), (2, 16), (1, 31), (1, 64)])
def test_reorder(groups, beams):
    g = torch.Generator().manual_seed(beams)
    rows = groups * beams
    parents = torch.randint(0, beams, (groups, beams), generator=g, dtype=torch.int32)
    lengths = torch.randint(0, 41, (rows,), generator=g, dtype=torch.int32)
    states = [(torch.randn((rows, 3, 40, 24), generator=g).bfloat16(), 2),
              (torch.randn((rows, 40, 5), generator=g), 1),
              (torch.randint(0, 9, (rows, 40), generator=g, dtype=torch.int32), 1),
              (torch.randint(0, 255, (rows, 2, 40, 3), generator=g, dtype=torch.uint8), 2),
              (torch.randn((rows, 7), generator=g), None),
              (torch.randn((rows, 2, 5000), generator=g).half(), None),
              (torch.randn((rows,), generator=g), None)]
    _reorder(states, parents, lengths)
    _reorder(states, parents)


def test_reorder_of_cycles_and_forks():
    x = torch.arange(8 * 1000).view(8, 1000).float()
    for p in ([1, 2, 3, 4, 5, 6, 7, 0], [7, 6, 5, 4, 3, 2, 1, 0], [3] * 8, list(range(8)), [1, 0, 1, 0, 5, 4, 5, 4],
              [-1, 0, -1, 2, 2, -1, 0, 0]):
        _reorder([(x, None)], torch.tensor([p], dtype=torch.int32))


def test_reorder_leaves_bad_parents_and_lengths_alone():
    x = torch.randn((6, 2, 50, 8))
    p = torch.tensor([[1, 3, -2], [2 ** 30, 0, -1]], dtype=torch.int32)
    assert _reorder([(x, 2)], p, torch.tensor([5, -3, 50, 2 ** 30, 51, 0], dtype=torch.int32)) == BEAM_BAD_PARENT


def test_reorder_of_layouts():
    rows, heads, time, dim = 6, 3, 33, 16
    p = torch.tensor([[1, 0, 0], [2, 2, 1]], dtype=torch.int32)
    lengths = torch.tensor([33, 7, 12, 1, 20, 31], dtype=torch.int32)
    base = torch.randn((rows, time, heads, dim))
    with BeamSearch(2, 3, device=DEV) as beam:
        # [rows, heads, time, dim] seen from [rows, time, heads, dim]
        x = base.to(DEV)
        beam.reorder([(x.transpose(1, 2), 2)], p.to(DEV), lengths.to(DEV))
        assert np.array_equal(x.cpu().numpy(), packed_ref.reorder(base.numpy(), p.numpy(), lengths.numpy(), 1))
        # keys and values side by side, and a cache longer than the view
        kv = torch.randn((rows, 2, heads, time, dim))
        y = kv.to(DEV)
        beam.reorder([(y[:, 0, :, :20], 2), (y[:, 1], 2)], p.to(DEV), lengths.to(DEV))
        want = kv.numpy().copy()
        want[:, 0, :, :20] = packed_ref.reorder(want[:, 0, :, :20], p.numpy(), lengths.numpy(), 2)
        want[:, 1] = packed_ref.reorder(want[:, 1], p.numpy(), lengths.numpy(), 2)
        assert np.array_equal(y.cpu().numpy(), want)
        # layers first: one state per layer, rows apart
        z = torch.randn((4, rows, time))
        w = z.to(DEV)
        beam.reorder([(w[i], 1) for i in range(4)] + [(w.transpose(0, 1)[:, :0], None)], p.to(DEV), lengths.to(DEV))
        for i in range(4):
            assert np.array_equal(w[i].cpu().numpy(), packed_ref.reorder(z[i].numpy(), p.numpy(), lengths.numpy(), 1))


def test_reorder_of_many_states_replayed():
    g = torch.Generator().manual_seed(3)
    states = [torch.randn((8, 2, 30, 16), generator=g).to(DEV) for _ in range(100)]
    before = [t.clone() for t in states]
    p = torch.tensor([[1, 0, 2, 2], [0, 3, 3, 1]], dtype=torch.int32)
    dp, lengths = p.to(DEV), torch.full((8,), 30, dtype=torch.int32, device=DEV)
    with BeamSearch(2, 4, device=DEV) as beam:
        bound = beam.bind([(t, 2) for t in states])
        beam.reorder(bound, dp, lengths)
        torch.cuda.synchronize()
        for t, b in zip(states, before):
            t.copy_(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            beam.reorder(bound, dp, lengths)
        graph.replay()
        torch.cuda.synchronize()
        for t, b in zip(states, before):
            assert np.array_equal(t.cpu().numpy(), packed_ref.reorder(b.cpu().numpy(), p.numpy()))


# --------------------------------------------------- the operators together

def test_beams_decoded_then_scored_against_the_saved_logits():
    """A small decode as a user runs it: a toy base model gives logits from
    the last token and a state; every step's base logits are kept in 8 bits
    and travel with their beams; the quantised model's logits of the best
    sequences are then scored against them, and their gradient reduces KL."""
    g = torch.Generator().manual_seed(7)
    groups, beams, v, dim, steps = 2, 4, 777, 24, 6
    rows = groups * beams
    emb, mix, head = (torch.randn(s, generator=g) * c for s, c in (((v, dim), 0.5), ((dim, dim), 0.3), ((dim, v), 0.8)))
    demb, dmix, dhead = emb.to(DEV), mix.to(DEV), head.to(DEV)
    hidden = torch.zeros((rows, dim), device=DEV)
    tokens = torch.zeros((rows, steps + 1), dtype=torch.int32, device=DEV)
    tokens[:, 0] = 1
    store = PackedLogits.empty(rows * steps, v, DEV)
    codes, heads = store.codes.view(rows, steps, -1), store.heads.view(rows, steps, -1)
    scores = torch.full((groups, beams), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    with BeamSearch(groups, beams, device=DEV) as beam, KLDStats(rows * steps, DEV) as st:
        bound = beam.bind([hidden, (tokens, 1), (codes, 1), (heads, 1)])
        for i in range(steps):
            hidden.copy_(torch.tanh(hidden @ dmix + demb[tokens[:, i].long()]))
            logits = hidden @ dhead
            now = pack_logits(logits)
            codes[:, i], heads[:, i] = now.codes, now.heads
            scores, tok, parent = beam.select(logits, scores, beams)
            beam.reorder(bound, parent, torch.full((rows,), i + 1, dtype=torch.int32, device=DEV))
            tokens[:, i + 1] = tok.reshape(-1)
        assert beam.status() == 0
        # the sequences' log-probabilities, decoded again from scratch, are the scores
        h = torch.zeros((rows, dim), dtype=torch.float64)
        total = torch.zeros(rows, dtype=torch.float64)
        seq = tokens.cpu().long()
        saved = store.unpack().view(rows, steps, v).cpu()
        for i in range(steps):
            h = torch.tanh(h @ mix.double() + emb.double()[seq[:, i]])
            x = h @ head.double()
            total += torch.log_softmax(x, 1)[torch.arange(rows), seq[:, i + 1]]
            # the saved logits are those of the beam's own history: half a step of at
            # most (range / 128) plus the fp32 model's own rounding
            step = (x.amax(1) - x.amin(1)) / 127
            assert ((saved[:, i].double() - x).abs().amax(1) <= step / 2 + 1e-4).all()
        # fp32 model: six matrix products and tanh, ~1e-6 a step each
        assert (total - scores.cpu().double().view(-1)).abs().max() < 1e-4
        # score and tune a quantised model on the decoded sequences
        quant = (saved.view(rows * steps, v) + 0.1 * torch.randn((rows * steps, v), generator=g)).to(DEV)
        nxt = tokens[:, 1:].reshape(-1).contiguous()
        grad = st.run_grad_packed(store, quant, nxt, scale=1.0)
        first = st.result()
        st.run_packed(store, quant - 0.5 * grad, nxt)
        second = st.result()
        assert first["n_valid"] == rows * steps and second["mean_kld"] < first["mean_kld"]


def test_flags_and_tickets_are_cleared_before_the_next_call():
    """A handle made, or its flags read, right before a call on a stream that
    does not wait for the default one."""
    x = _rows(8, 4099, 3)
    x[2, 17] = math.nan
    x, scores = x.to(DEV), _scores(2, 4, 3).to(DEV)
    side = torch.cuda.Stream(DEV)
    big = torch.empty(64 << 20, device=DEV)
    torch.cuda.synchronize()
    want = None
    for _ in range(20):
        big.fill_(1.0)  # the default stream is busy
        with BeamSearch(2, 4, max_k=8, device=DEV) as beam:
            for _ in range(3):
                got = beam.select(x, scores, 8, stream=side)
                assert beam.status() == BEAM_NONFINITE
                got = [t.cpu() for t in got]
                want = want or got
                assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_over_inputs_are_refused():
    x, scores = _rows(4, 100, 1).to(DEV), _scores(2, 2, 1).to(DEV)
    free = [torch.empty((2, 2), dtype=dt, device=DEV) for dt in (torch.float32, torch.int32, torch.int32)]
    with BeamSearch(2, 2, max_k=4, device=DEV) as beam:
        for out in ((scores, free[1], free[2]), (free[0], free[1], free[1]),
                    (free[0], scores.view(torch.int32), free[2]), (x[3, 96:].view(2, 2), free[1], free[2])):
            with pytest.raises(KLDError):
                beam.select(x, scores, 2, out=out)
        done = torch.zeros((2, 2), dtype=torch.bool, device=DEV)
        assert beam.select(x, scores, 2, finished=done, eos=3, out=tuple(free))[0] is free[0]
        assert beam.status() == 0


def test_reorder_refuses_states_that_overlap_and_runs_past_a_grid():
    kv = torch.arange(4 * 3 * 2 * 5 * 8, dtype=torch.float32, device=DEV).view(4, 3, 2, 5, 8)
    parents = torch.tensor([[1, 0, 3, 3]], dtype=torch.int32, device=DEV)
    with BeamSearch(1, 4, device=DEV) as beam:
        for states in ([kv, kv], [(kv[:, :, 0], 2), (kv[:, :, 0, 1:], 2)], [kv, (kv[:, 1, 1], 1)]):
            with pytest.raises(ValueError):
                beam.reorder(states, parents)
        want = packed_ref.reorder(kv.cpu().numpy(), parents.cpu().numpy())
        beam.reorder([(kv[:, :, 0], 2), (kv[:, :, 1], 2)], parents,
                     torch.full((4,), 1 << 30, dtype=torch.int32, device=DEV))
        assert np.array_equal(kv.cpu().numpy(), want)
        # more runs than one launch takes: refused before the first state is moved
        many = [_lib.State(kv.data_ptr(), 960, 1, 0, 1, 960, 0, 0),
                _lib.State(kv.data_ptr(), 1 << 47, (1 << 31) - 1, 4096, 1, 2048 * 16, 0, 0)]
        many[1].outer_stride = 2048 * 16
        status = beam._lib.kld_beam_reorder(beam._h, (_lib.State * 2)(*many), 2, parents.data_ptr(), None, 1, 4, None)
        assert status == _lib.KLD_ERR_INVALID_ARG
        assert np.array_equal(kv.cpu().numpy(), want) and beam.status() == 0


@pytest.mark.parametrize("groups,beams,v,k", [(1, 1, 1000003, 128), (1, 64, 9001, 128), (600, 4, 130, 64),
                                              (2500, 1, 5000, 1), (3, 1, 257, 128)])
def test_many_and_few_lists(groups, beams, v, k):
    _check(_rows(groups * beams, v, k), _scores(groups, beams, k), k)


def test_lists_that_overflow_among_many_parts():
    x = _rows(8, 200000, 12)
    x[0] = 1.0                                     # one value everywhere
    x[1, ::2] = 12.0                               # half of the row at the maximum
    x[2] = torch.arange(200000).float() * 1e-4     # rising: every entry passes the bound before it
    x[3, 150000:] = 12.0
    for dt in (torch.float32, torch.bfloat16):
        _check(x.to(dt), _scores(2, 4, 2), 100)
        _check(x.to(dt), torch.zeros((1, 8)), 128)


def test_rows_past_32_bit_offsets():
    """Rows 2^28 elements apart: the last ones lie past 2^31 elements."""
    groups, beams, v, ld = 3, 3, 3000, 1 << 28
    x = _rows(groups * beams, v, 21).bfloat16()
    flat = torch.empty((groups * beams - 1) * ld + v, dtype=torch.bfloat16, device=DEV)
    view = torch.as_strided(flat, (groups * beams, v), (ld, 1))
    view.copy_(x)
    _check(x, _scores(groups, beams, 21), 6, logits=view)
    cache = torch.as_strided(flat, (groups * beams, 50, 8), (ld, 8, 1))
    cache.copy_(torch.arange(groups * beams * 400).view(groups * beams, 50, 8).remainder(251).bfloat16())
    parents = torch.tensor([[1, 0, 0], [2, 2, 1], [0, 1, 1]], dtype=torch.int32)
    lengths = torch.tensor([50, 7, 0, 1, 50, 9, 13, 3, 90], dtype=torch.int32)
    want = packed_ref.reorder(cache.float().cpu().numpy(), parents.numpy(), lengths.numpy(), 1)
    with BeamSearch(groups, beams, device=DEV) as beam:
        beam.reorder([(cache, 1)], parents.to(DEV), lengths.to(DEV))
        assert np.array_equal(cache.float().cpu().numpy(), want) and beam.status() == 0


@pytest.mark.parametrize("entries", [225, 240, 255, 256, 257, 288])
def test_finished_beams_at_the_merge_s_list_limit(entries):
    """So many entries that tie at the top of 32 live beams, and 32 finished
    beams that join them: the merge decides at 256 entries whether to look for
    a closer bound, before the finished beams' entries come in."""
    groups, beams, v, k = 4, 64, 333, 128
    x = torch.full((groups * beams, v), -math.inf)
    done = torch.zeros((groups, beams), dtype=torch.bool)
    done[:, 1::2] = True
    for g in range(groups):
        for i in range(entries):  # equal rows as far as they go
            x[g * beams + 2 * (i % 32), (7 * (i // 32)) % v] = 1.0
    s = torch.full((groups, beams), -2.0)
    s[:, 1::2] -= torch.arange(32) * 0.125
    with BeamSearch(groups, beams, max_k=k, device=DEV) as beam:
        for _ in range(20):
            _check(x, s, k, finished=done, eos=5, beam=beam)
        assert beam.status() == 0


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("v", [3001, 32003, 50257])
def test_equal_beams_tie_wherever_their_rows_start(dtype, v):
    """Equal rows that start at different offsets within 16 bytes have equal
    log-sum-exps, so their entries tie and the lowest beam comes first."""
    groups, beams = 20, 5
    x = _rows(groups, v, v).to(DTYPES[dtype])
    x = x[:, None].expand(groups, beams, v).reshape(groups * beams, v)
    s = torch.full((groups, beams), -3.0)
    s[3:] = _scores(groups, 1, 4)[3:].expand(-1, beams)
    _check(x, s, 10)
    for shift, ld in ((1, v), (5, v + 2), (0, v + 3)):
        flat = torch.full((shift + groups * beams * ld,), math.nan, dtype=x.dtype, device=DEV)
        view = torch.as_strided(flat, x.shape, (ld, 1), shift)
        view.copy_(x)
        _check(x, s, 10, logits=view)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_zeros_of_either_sign_tie(dtype):
    x = torch.zeros((4, 12000))
    x[:, ::2] = -0.0
    x[1] = -x[1]
    x[2, 500:] = -0.0
    x[3, :700] = -0.0
    x[3, 700:] = -1.0
    s = torch.tensor([[0.0, -0.0], [-0.0, 0.0]])
    for k in (1, 8, 100):
        _check(x.to(DTYPES[dtype]), s, k)
    # a single token: its score is the beam's own, zeros of either sign tie too
    _check(torch.zeros((4, 1), dtype=DTYPES[dtype]), s, 2)
    done = torch.tensor([[True, False], [False, True]])
    _check(torch.zeros((4, 1), dtype=DTYPES[dtype]), s, 2, finished=done, eos=0)


def test_parents_and_lengths_between_the_rows_of_a_state():
    """A state seen as part of wider rows, its parents and lengths kept in the
    rows' ends."""
    groups, beams = 2, 3
    wide = torch.arange(6 * 20, dtype=torch.int32).view(6, 20).to(DEV)
    p = torch.tensor([[1, 0, 0], [2, 2, 1]], dtype=torch.int32)
    lengths = torch.tensor([12, 3, 0, 5, 11, 7], dtype=torch.int32)
    parents, lens = wide[2, 14:20].view(groups, beams), wide[4, 13:19]
    parents.copy_(p), lens.copy_(lengths)
    before = wide.cpu().numpy()
    want = before.copy()
    want[:, :12] = packed_ref.reorder(before[:, :12], p.numpy(), lengths.numpy(), 1)
    with BeamSearch(groups, beams, device=DEV) as beam:
        beam.reorder([(wide[:, :12], 1)], parents, lens)
        assert np.array_equal(wide.cpu().numpy(), want)
        with pytest.raises(ValueError):
            beam.reorder([(wide[:, :15], 1)], parents, lens)
        with pytest.raises(ValueError):
            beam.reorder([(wide[:, :14], 1)], parents, lens)


def test_eos_outside_the_vocabulary_is_refused():
    x, s = _rows(4, 100, 1).to(DEV), _scores(2, 2, 1).to(DEV)
    done = torch.zeros((2, 2), dtype=torch.bool, device=DEV)
    with BeamSearch(2, 2, device=DEV) as beam:
        for eos in (None, -1, 100, (1 << 32) + 3, -(1 << 32)):
            with pytest.raises(ValueError):
                beam.select(x, s, 2, finished=done, eos=eos)
        beam.select(x, s, 2, finished=done, eos=99)
        beam.select(x, s, 2, eos=(1 << 40))  # not looked at
        assert beam.status() == 0


@pytest.mark.parametrize("rows,v", [(2400, 151936), (2400, 1 << 20), (64, 1 << 24)])
@pytest.mark.parametrize("down", [0.0, 0.6875, 1.90625, 3.09375])
def test_log_sum_exp_of_long_rows_of_two_values(rows, v, down):
    """Equal terms round alike, so that the errors of a long fp32 sum add up:
    the scores of rows that hold one value or two by turns."""
    x = torch.full((rows, v), 0.5, dtype=torch.bfloat16, device=DEV)
    x[:, 1::2] -= down
    with BeamSearch(rows, 1, device=DEV) as beam:
        s, t, _ = beam.select(x, torch.zeros((rows, 1), device=DEV), 1)
    assert (t == 0).all()
    want = math.log(v / 2 * (1.0 + math.exp(-down)))
    assert (s.double() + want).abs().max().item() <= 2.0 ** -24 * want + 2e-6
