"""8-bit logit checkpoints on the GPU.

Codes, headers and restored fp32 values: equal bit for bit to the format's
definition in 64 bits (its arithmetic is exact in fp32, so no tolerance).
16-bit restored values: the fp32 ones rounded to nearest.

Statistic from a checkpoint: that of the stored values by the fp64 oracle, at
the bars of gpu_helpers (per-row KL and NLL |d| <= 1e-6 + 1e-4 |ref|, argmaxes,
flags and counts equal).

Gradient: every element within |scale| * (4e-6 * (p + r) + 1e-12), p and r its
two softmax values. Each is an fp32 exponential: its argument u = x L - F is
one FMA (error <= |u| 2^-24, that is <= |u| ln2 2^-24 = 1.7e-6 relative at
|u| = 40, where the value is 1e-12), ex2.approx 2^-22, lambda - 1 = 1.4e-8
times |u|, the normaliser's sum (a few hundred fp32 terms whose partial sums
round by 2^-24 each, ~1e-6 in the worst case, and fp64 from there) and its
rounding 2^-24: <= 3.5e-6 together. Outputs in 16 bits add half a step, 2^-8
(bf16) or 2^-11 (fp16) of the value, and fp16's fixed step 2^-25 below its
normal range."""
import math
import threading

import numpy as np
import pytest
import torch

import oracle
import packed_ref
from logit_kl_divergence_b200 import KLDError, KLDStats, PackedLogits, pack_logits, rows_view, synth

from gpu_helpers import assert_rows_match, assert_stats_match

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _np(t):
    return t.detach().float().cpu().numpy()


def _pair(n, v, seed, masked=0):
    g = torch.Generator().manual_seed(seed)
    b = torch.randn((n, v), generator=g) * 2.5
    b[torch.arange(n), torch.randint(0, v, (n,), generator=g)] += 9.0
    q = b + torch.randn((n, v), generator=g) * 0.2
    if masked:
        b[:, v - masked:] = -math.inf
        q[:, v - masked:] = -math.inf
    tok = torch.randint(0, max(1, v - masked), (n,), generator=g, dtype=torch.int32)
    return b, q, tok


def _check_pack(x):
    p = pack_logits(x.to(DEV))
    codes, heads, value = packed_ref.pack(_np(x))
    assert np.array_equal(p.heads.cpu().numpy(), heads)
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    back = p.unpack()
    assert np.array_equal(_np(back), value.astype(np.float32), equal_nan=True)
    for dt in (torch.bfloat16, torch.float16):
        got = p.unpack(dt)
        want = back.to(dt)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    return p


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,v", [(1, 1), (3, 7), (2, 127), (5, 128), (4, 129), (7, 1000), (3, 4099),
                                 (2, 32003), (33, 512), (1, 70001)])
def test_pack_and_unpack_are_the_format(dtype, n, v):
    _check_pack(_pair(n, v, 3 * v + n)[0].to(DTYPES[dtype]))


def test_pack_of_masks_and_odd_values():
    b, _, _ = _pair(12, 1000, 5, masked=300)
    b[1] = -math.inf                       # a fully masked row
    b[2] = 1000.125                        # a constant: stored exactly
    b[3] = 0.0
    b[4] = torch.finfo(torch.float32).min  # magnitudes past the format's limit
    b[5, 17] = math.nan
    b[6, 130] = math.inf
    b[7] = torch.randn(1000) * 1e-42       # subnormals
    b[8] = torch.randn(1000) * 1e30
    b[9] = torch.where(torch.arange(1000) % 3 == 0, torch.tensor(-math.inf), b[9])
    b[10] = torch.arange(1000).float() * 254.0 / 127.0  # ends on whole steps
    b[11] = 2.0 ** 126 * torch.where(torch.arange(1000) == 5, 1.0, 0.999)
    p = _check_pack(b)
    assert torch.equal(p.unpack()[2].cpu(), b[2])


def test_pack_writes_parts_of_a_store_and_nothing_else():
    b, _, _ = _pair(6, 333, 8)
    store = PackedLogits.empty(10, 333, DEV)
    store.codes.fill_(77)
    store.heads.fill_(99)
    pack_logits(b.to(DEV), out=store.rows(2, 8))
    whole = pack_logits(b.to(DEV))
    assert torch.equal(store.codes[2:8], whole.codes) and torch.equal(store.heads[2:8], whole.heads)
    for part in (slice(0, 2), slice(8, 10)):
        assert (store.codes[part] == 77).all() and (store.heads[part] == 99).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_pack_of_a_row_that_starts_inside_a_vector(dtype):
    dt = DTYPES[dtype]
    b, _, _ = _pair(5, 1001, 9)
    for shift in range(1, 8):
        flat = torch.empty(5 * 1001 + 8, dtype=dt, device=DEV)
        x = flat[shift:shift + 5 * 1001].view(5, 1001)
        x.copy_(b)
        want = pack_logits(b.to(dt).to(DEV).clone())
        got = pack_logits(x)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.heads, want.heads)


# ---------------------------------------------------------- statistic, gradient

def _tolerance(p, r, ref, dtype, scale):
    tol = abs(scale) * (4e-6 * (np.nan_to_num(p) + np.nan_to_num(r)) + 1e-12)
    if dtype == torch.bfloat16:
        tol = tol + np.abs(ref) * 2.0 ** -8
    elif dtype == torch.float16:
        tol = tol + np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25)
    return tol


def _check(b, q, tok, quant="f32", grad=None, scale=1.0, out=None, pack_quant=False):
    n, v = b.shape
    base = pack_logits(b.to(DEV))
    qd = q.to(DTYPES[quant]).to(DEV)
    other = pack_logits(qd) if pack_quant else qd
    t = None if tok is None else tok.to(DEV)
    with KLDStats(n, DEV) as st:
        if grad is None:
            rows = st.run_packed(base, other, t, per_row=True)
            g = None
        else:
            g, rows = st.run_grad_packed(base, other, t, out=out, scale=scale, grad_dtype=DTYPES[grad],
                                         per_row=True)
        res = st.result()
        rec = {k: x.cpu().numpy() for k, x in rows_view(st.records()).items()}
    rec["flags"] = rec["flags"].astype(np.uint32)
    bv, qv = base.unpack().cpu(), (other.unpack() if pack_quant else qd.float()).cpu()
    ref_rows, ref = oracle.run(bv, qv, tok, oracle.F32)
    # rows of the type's lowest value: the oracle's q - lse_q absorbs ln V there
    # (it gives a negative KL), so they are taken relative to the maximum
    for i in np.nonzero((qv.amax(1) < -1e37).numpy() & ((ref_rows["flags"] & 3) == 0))[0]:
        ref_rows["kld"][i], lp, lr = packed_ref.relative_row(bv[i].numpy(), qv[i].numpy())
        if tok is not None and 0 <= tok[i] < v:
            ref_rows["nll"][i], ref_rows["nll_base"][i] = -lr[tok[i]], -lp[tok[i]]
        ref = oracle.reduce(ref_rows, tok is not None)
    assert_rows_match(rec, ref_rows)
    assert_stats_match(res, ref)
    for name in ("kld", "nll", "amax_b", "amax_q"):
        assert np.array_equal(rows[name].cpu().numpy(), rec[name], equal_nan=True)
    if g is not None:
        p, r = packed_ref.softmax(bv.numpy()), packed_ref.softmax(qv.numpy())
        keep = (ref_rows["flags"] & 3) == 0
        want = np.where(keep[:, None], (r - p) * scale, 0.0)
        got = _np(g).astype(np.float64)
        d = np.abs(got - want)
        tol = _tolerance(p, r, want, g.dtype, scale)
        assert (d <= tol).all(), (d / tol).max()
        assert (got[~keep] == 0).all()
    return rec


@pytest.mark.parametrize("quant", ["f32", "bf16", "f16", "packed"])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (5, 7), (4, 129), (9, 512), (3, 513), (2, 1000),
                                 (5, 4099), (2, 32003), (1, 151936), (3, 70001)])
def test_statistic_and_gradient(n, v, quant):
    b, q, tok = _pair(n, v, v + n)
    dt = "f32" if quant == "packed" else quant
    _check(b, q, tok, dt, None, pack_quant=quant == "packed")
    _check(b, q, tok, dt, dt, scale=1.0 / n, pack_quant=quant == "packed")


@pytest.mark.parametrize("quant,grad", [("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"),
                                        ("f16", "f32"), ("bf16", "f16"), ("packed", "f32"),
                                        ("packed", "bf16"), ("packed", "f16")])
@pytest.mark.parametrize("v", [1024, 2051])
def test_gradient_of_another_type(quant, grad, v):
    b, q, tok = _pair(6, v, v, masked=40)
    _check(b, q, tok, "f32" if quant == "packed" else quant, grad, scale=0.25, pack_quant=quant == "packed")


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
def test_many_rows_take_whole_and_split_launches(quant):
    for n, v in ((40, 20000), (300, 9001), (700, 1536)):
        b, q, tok = _pair(n, v, n)
        _check(b, q, tok, "f32" if quant == "packed" else quant, "f32", scale=1.0, pack_quant=quant == "packed")


def _edge_rows(v):
    b, q, tok = _pair(16, v, 77)
    b[0, v // 2:] = -math.inf
    q[0, v // 2:] = -math.inf                    # masks in both
    b[1, :v // 3] = -math.inf                    # masked in the base only
    q[2, 3] = -math.inf                          # KL = +inf
    b[3] = -math.inf                             # empty rows
    q[4] = -math.inf
    q[5, v - 1] = math.nan
    q[6, 0] = math.inf
    b[7, v // 2] = math.nan
    q[8] = b[8] + 1000.0                         # a constant shift
    q[9] = torch.finfo(torch.float32).min        # the type's lowest value everywhere
    q[10, ::2] = torch.finfo(torch.float32).min  # and as a mask
    b[10, ::2] = -math.inf
    b[11] = 0.0
    q[11] = 0.0                                  # ties everywhere
    b[12, 5] += 80.0
    q[12, 5] += 80.0                             # one-hot
    q[13] = b[13]
    tok[14], tok[15] = -1, v
    tok[0] = v - 1                               # a masked token
    tok[2] = 3
    return b, q, tok


@pytest.mark.parametrize("v", [40, 1500, 33000])
@pytest.mark.parametrize("grad", [None, "f32"])
def test_rows_at_the_edges(v, grad):
    b, q, tok = _edge_rows(v)
    _check(b, q, tok, "f32", grad)
    _check(b, q, None, "f32", grad)


@pytest.mark.parametrize("v", [40, 1500])
def test_rows_at_the_edges_with_both_packed(v):
    b, q, tok = _edge_rows(v)
    _check(b, q, tok, "f32", "f32", pack_quant=True)


def test_equal_rows_give_zero_exactly():
    b, _, tok = _pair(9, 5000, 4)
    base = pack_logits(b.to(DEV))
    with KLDStats(9, DEV) as st:
        g, rows = st.run_grad_packed(base, base.unpack(), tok.to(DEV), per_row=True)
        assert (g == 0).all() and (rows["kld"] == 0).all()
        g, rows = st.run_grad_packed(base, base, tok.to(DEV), per_row=True)
        assert (g == 0).all() and (rows["kld"] == 0).all()


@pytest.mark.parametrize("quant", ["f32", "bf16", "f16"])
def test_quant_rows_and_gradient_at_any_alignment(quant):
    dt = DTYPES[quant]
    n, v = 3, 1037
    b, q, tok = _pair(n, v, 12, masked=9)
    for shift in range(0, 8):
        flat = torch.empty(n * v + 16, dtype=dt, device=DEV)
        x = flat[shift:shift + n * v].view(n, v)
        x.copy_(q)
        store = torch.full((n * v + 32,), 7.0, dtype=torch.float32, device=DEV)
        out = store[8 + shift:8 + shift + n * v].view(n, v)
        base = pack_logits(b.to(DEV))
        with KLDStats(n, DEV) as st:
            got = st.run_grad_packed(base, x, tok.to(DEV), out=out)
            want = st.run_grad_packed(base, q.to(dt).to(DEV), tok.to(DEV), grad_dtype=torch.float32)
            # another order of the sums only: S differs by a few 2^-24
            p = np.abs(packed_ref.softmax(_np(base.unpack()))) + np.abs(packed_ref.softmax(_np(x)))
            assert (np.abs(_np(got) - _np(want)) <= 4e-6 * p + 1e-12).all()
        assert (store[:8 + shift] == 7).all() and (store[8 + shift + n * v:] == 7).all()


def test_gradient_agrees_with_differences():
    # d KL / d q by central differences of the oracle in fp64 over the stored values
    b, q, _ = _pair(1, 60, 3)
    base = pack_logits(b.to(DEV))
    with KLDStats(1, DEV) as st:
        g = st.run_grad_packed(base, q.to(DEV))[0].cpu().double()
    p = packed_ref.softmax(_np(base.unpack()))[0]
    x = q[0].double().numpy()

    def kl(z):
        r = packed_ref.softmax(z[None])[0]
        return float((p * (np.log(p) - np.log(r))).sum())

    h = 1e-5
    for j in range(60):
        e = np.zeros(60)
        e[j] = h
        d = (kl(x + e) - kl(x - e)) / (2 * h)
        # differences: h^2/6 of the third derivative (<= 1) + 1e-15 / h; gradient: as above
        assert abs(float(g[j]) - d) <= 4e-6 * 2 + 1e-9


def test_store_kept_across_steps_streams_and_graphs():
    b, q, tok = _pair(24, 3000, 21)
    base, t = pack_logits(b.to(DEV)), tok.to(DEV)
    quant = q.to(DEV)
    with KLDStats(24, DEV) as st:
        want, rows = st.run_grad_packed(base, quant, t, scale=0.5, per_row=True)
        want, kld = want.clone(), rows["kld"].clone()
        res = st.result()
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream(DEV))
        got, rows = st.run_grad_packed(base, quant, t, scale=0.5, per_row=True, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(rows["kld"], kld) and st.result() == res
        # captured and replayed on new quant rows
        out = torch.empty_like(want)
        moving = quant.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st.run_grad_packed(base, moving, t, out=out, scale=0.5)
        moving.copy_(quant.flip(1))
        want2 = st.run_grad_packed(base, quant.flip(1).contiguous(), t, scale=0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want2)
        moving.copy_(quant)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_packed_rows_leave_the_dense_path_as_it_was():
    w = synth.make_recipe("ctx", n=40, v=2049, dtype=synth.F32, seed=3)
    b, q, t = w.base.to(DEV), w.quant.to(DEV), w.token_ids.to(DEV)
    with KLDStats(40, DEV) as st:
        st.run(b, q, t)
        before = st.result()
        st.run_grad_packed(pack_logits(b), q, t)
        st.run(b, q, t)
        assert st.result() == before


def test_sizes_of_zero_rows():
    p = pack_logits(torch.empty((0, 300), device=DEV))
    assert p.shape == (0, 300) and p.unpack().shape == (0, 300)


@pytest.mark.parametrize("quant", ["f32", "bf16"])
@pytest.mark.parametrize("n,v", [(3, 40000), (1, 5), (700, 1003)])
def test_gradient_over_the_quant_rows_themselves(quant, n, v):
    """In place: the same gradient, rows done in fp64 (masked base entries
    with finite quant ones and the reverse, a NaN row) included."""
    b, q, tok = _pair(n, v, n + v)
    if n > 2:
        b[0, 1::2] = -math.inf
        q[1, ::3] = -math.inf
        q[2, v // 2] = math.nan
    q = q.to(DTYPES[quant]).to(DEV)
    base, tok = pack_logits(b.to(DEV)), tok.to(DEV)
    with KLDStats(n, device=DEV) as st:
        want, rows = st.run_grad_packed(base, q, tok, scale=0.5, per_row=True)
        over = q.clone()
        got, again = st.run_grad_packed(base, over, tok, out=over, scale=0.5, per_row=True)
        assert got.data_ptr() == over.data_ptr() and torch.equal(got, want)
        for name in rows:
            assert torch.equal(rows[name].nan_to_num(nan=-1.0), again[name].nan_to_num(nan=-1.0))


def test_outputs_over_inputs_are_refused():
    n, v = 4, 256
    mem = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)

    def at(byte, dtype, *shape):
        size = torch.empty((), dtype=dtype).element_size() * math.prod(shape)
        return mem[byte:byte + size].view(dtype).view(*shape)

    base = PackedLogits(at(0, torch.uint8, n, v), at(1024, torch.int32, n, 2), v)
    quant, tok = at(2048, torch.bfloat16, n, v), at(4096, torch.int32, n)
    with KLDStats(n, device=DEV) as st:
        for byte, dtype in ((2048, torch.float16), (2046, torch.bfloat16), (4094, torch.bfloat16),
                            (0, torch.bfloat16), (1022, torch.bfloat16), (1054, torch.float16), (4108, torch.float32)):
            with pytest.raises(KLDError):
                st.run_grad_packed(base, quant, tok, out=at(byte // 4 * 4 if dtype == torch.float32 else byte,
                                                            dtype, n, v))
        with pytest.raises(KLDError):
            st.run_grad_packed(base, base, out=at(1020, torch.float32, n, v))
        for byte in (0, 4112):  # before and behind all of them
            st.run_grad_packed(PackedLogits(at(8192, torch.uint8, n, v), at(9216, torch.int32, n, 2), v), quant,
                               tok, out=at(byte, torch.bfloat16, n, v))
        st.run_grad_packed(base, quant, tok, out=quant)
        st.result()


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
@pytest.mark.parametrize("n,v", [(1, 900001), (7, 300000), (800, 41000)])
def test_masks_in_every_block(n, v, quant):
    """Every chunk holds masked entries: more of them than a warp lists."""
    b, q, tok = _pair(n, v, n)
    for x in (b, q):
        x[:, 5::97] = -math.inf
    b[:, 40::1009] = -math.inf          # and some in the base only
    tok = torch.full((n,), 4, dtype=torch.int32)
    _check(b, q, tok, "f32" if quant == "packed" else quant, "bf16", scale=2.0, pack_quant=quant == "packed")


def test_bad_and_empty_rows_among_many():
    n, v = 1500, 515
    b, q, tok = _pair(n, v, 5)
    b[::7] = -math.inf
    q[3::11] = -math.inf
    q[5::13, 17] = math.nan
    b[6::17, ::2] = -math.inf           # finite quant entries there
    tok[::5] = v
    tok[1::5] = -7
    _check(b, q, tok, "bf16", "f32")
    _check(b, q, tok, "f32", "f32", pack_quant=True)


def test_rows_longer_than_32_bit_offsets():
    """70 rows of 2^25 + 1 columns: offsets past 2^31 in codes and logits."""
    n, v = 70, (1 << 25) + 1
    q = torch.zeros((n, v), dtype=torch.bfloat16, device=DEV)
    q[:, 77] = 3.0
    q[n - 1, v - 1] = 9.0
    base = pack_logits(q)
    # a block of one value has code 1 whatever the value; its header tells
    assert base.codes[n - 1, v - 1] == 1 and base.heads[n - 1, -1] != base.heads[n - 1, 1]
    assert base.unpack(torch.bfloat16)[n - 1, v - 3:].tolist() == [0.0, 0.0, 9.0]
    other = q.clone()
    other[n - 1, v - 1] = 0.0
    tok = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    with KLDStats(n, device=DEV) as st:
        g, rows = st.run_grad_packed(base, other, tok, per_row=True)
        assert (rows["kld"][:n - 1] == 0).all() and (g[:n - 1] == 0).all()
        z_b, z_q = v - 2 + math.exp(3.0) + math.exp(9.0), v - 1 + math.exp(3.0)
        kl = 9.0 * math.exp(9.0) / z_b - math.log(z_b) + math.log(z_q)
        assert abs(rows["kld"][n - 1].item() - kl) <= 1e-6 + 1e-4 * kl
        assert rows["amax_b"][n - 1] == v - 1 and (rows["amax_q"] == 77).all()
        want = 1.0 / z_q - math.exp(9.0) / z_b
        assert abs(g[n - 1, v - 1].item() - want) <= 2.0 ** -8 * abs(want) + 4e-6 * (1.0 / z_q + math.exp(9.0) / z_b)


def test_ties_go_to_even_whatever_the_base():
    """Blocks whose values lie halfway between two steps, at odd and even
    bases of either sign; some with masked entries between."""
    k = torch.arange(128).float()
    rows = []
    for base in (-300, -7, -4, 0, 1, 2, 1001, 4096):
        rows.append((base + 2 * k + torch.where(k % 3 == 0, 0.0, 0.5)).clone())  # range 254: steps of one
        x = rows[-1].clone()
        x[5::9] = -math.inf
        rows.append(x)
    _check_pack(torch.stack(rows))
    _check_pack(torch.cat(rows).view(2, -1)[:, :1019].contiguous())


def test_two_host_threads_with_handles_of_their_own():
    """Calls that need different amounts of shared memory of the same kernel,
    from two host threads at once, each with its own handle and stream."""
    sizes = [(2, 900), (2, 60000), (2, 3000), (2, 30000)]
    errors = []

    def work(i, n, v):
        try:
            b, q, _ = _pair(n, v, v)
            side = torch.cuda.Stream(DEV)
            with torch.cuda.stream(side), KLDStats(n, DEV) as st:
                base = pack_logits(b.to(DEV))
                quant = pack_logits(q.to(DEV))
                want = st.run_packed(base, quant, per_row=True)["kld"].clone()
                for _ in range(1500):
                    got = st.run_packed(base, quant, per_row=True)["kld"]
                assert torch.equal(got, want)
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i, *s)) for i, s in enumerate(sizes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def _peaked(n, v, peak, gap):
    """A token that the base model puts first and the quant rows hold `gap`
    nats below their own maximum (a token banned by a bias), which is in the
    same chunk, another warp's, or another CTA's of the cluster."""
    g = torch.Generator().manual_seed(v + int(gap))
    b = torch.randint(-4, 5, (n, v), generator=g) * 0.125
    q = torch.randint(-4, 5, (n, v), generator=g) * 0.125
    b[:, 5], q[:, 5], q[:, peak] = 30.0, 30.0 - gap, 30.0
    return b, q


PEAKS = [(1, 2048, 300), (1, 8192, 1500), (1, 70001, 60000), (900, 2048, 1500)]


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
@pytest.mark.parametrize("gap", [40.0, 85.0, 95.0, 100.0, 300.0])
@pytest.mark.parametrize("n,v,peak", PEAKS)
def test_statistic_of_quant_rows_that_peak_far_from_the_base_argmax(n, v, peak, gap, quant):
    b, q = _peaked(n, v, peak, gap)
    _check(b, q, torch.full((n,), 9, dtype=torch.int32), "f32" if quant == "packed" else quant,
           pack_quant=quant == "packed")
    # the peak's own NLL, about e^-25, at the bar of a row
    base, quant = pack_logits(b.to(DEV)), q.to(DEV) if quant != "packed" else pack_logits(q.to(DEV))
    with KLDStats(n, DEV) as st:
        rows = st.run_packed(base, quant, torch.full((n,), peak, dtype=torch.int32, device=DEV), per_row=True)
        assert (rows["nll"].abs() <= 1e-6).all()


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
@pytest.mark.parametrize("gap", [40.0, 85.0, 95.0, 100.0, 300.0])
@pytest.mark.parametrize("n,v,peak", PEAKS)
def test_gradient_of_quant_rows_that_peak_far_from_the_base_argmax(n, v, peak, gap, quant):
    b, q = _peaked(n, v, peak, gap)
    tok = torch.full((n,), 9, dtype=torch.int32)
    for scale in (1.0, 1.0 / 2048):
        _check(b, q, tok, "f32" if quant == "packed" else quant, "f32", scale=scale, pack_quant=quant == "packed")


def _wide_rows(v):
    """Rows whose blocks span up to 2^126: steps past 2^95."""
    b, q, tok = _pair(9, v, 31)
    for i, m in enumerate((-1e28, -1e30, -6e33, -1e36, -8.5e37)):
        b[i, 3::5] = m                       # masks that every block holds
        q[i, 3::5] = m
    b[5, 7] = -3e37                          # in one block
    q[5, 7] = -3e37
    b[6] = -8e37                             # everywhere
    q[6] = -8e37
    b[7] = torch.randn(v, generator=torch.Generator().manual_seed(1)).clamp(-2, 2) * 4e37
    q[7] = b[7]
    b[8, ::2], b[8, 1::2] = 8e37, -8e37
    q[8] = b[8]
    tok[:] = 0
    return b, q, tok


@pytest.mark.parametrize("v", [640, 1003, 9001])
def test_blocks_of_any_width_read_as_the_format(v):
    b, q, tok = _wide_rows(v)
    _check_pack(b)
    _check_pack(b[:, :512].contiguous())
    _check_pack(b.bfloat16())


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
@pytest.mark.parametrize("v", [640, 1003, 9001])
def test_rows_of_wide_blocks(v, quant):
    b, q, tok = _wide_rows(v)
    _check(b[:7], q[:7], tok[:7], "f32" if quant == "packed" else quant, "f32", pack_quant=quant == "packed")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("v", [1000, 4099])
def test_finite_masks_are_stored_as_none(dtype, v):
    """Rows masked by the type's lowest value or another finite one: with
    mask_at the checkpoint of the same rows masked by -inf."""
    dt = DTYPES[dtype]
    b = _pair(6, v, v)[0].to(dt)
    mask = torch.rand((6, v), generator=torch.Generator().manual_seed(2)) < 0.3
    mask[4], mask[5] = True, False
    mask[3, 128:256] = True
    none = b.masked_fill(mask, -math.inf)
    want = pack_logits(none.to(DEV))
    for mask_at in (torch.finfo(dt).min, -1e4, -60000.1) + ((-1e9,) if dtype != "f16" else ()):
        m = torch.tensor(mask_at, dtype=dt)
        x = b.masked_fill(mask, m.item())
        got = pack_logits(x.to(DEV), mask_at=mask_at)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.heads, want.heads)
        x[0, ::7] = -math.inf                        # masks of both kinds
        got, same = pack_logits(x.to(DEV), mask_at=mask_at), pack_logits(x.masked_fill(x <= m, -math.inf).to(DEV))
        assert torch.equal(got.codes, same.codes) and torch.equal(got.heads, same.heads)
    # NaN and +inf are not masks
    x = b.clone()
    x[1, 5], x[2, 7] = math.nan, math.inf
    got, same = pack_logits(x.to(DEV), mask_at=-1e4), pack_logits(x.to(DEV))
    assert torch.equal(got.codes, same.codes) and torch.equal(got.heads, same.heads)
    with pytest.raises(KLDError):
        pack_logits(b.to(DEV), mask_at=math.nan)


@pytest.mark.parametrize("quant", ["f32", "bf16"])
def test_rows_masked_by_the_type_s_lowest_value(quant):
    """KL and gradient of base rows masked by finfo.min, stored with mask_at,
    against those of the dense rows: the masked entries have no weight either
    way. A stored value is off by at most d = R / 254, R the row's span, so ln p
    by 2d and p by a factor within e^(+-2d); KL changes by sum p' (ln p' - ln p)
    + sum (p' - p) ln(p / r)."""
    dt = DTYPES[quant]
    n, v = 5, 3001
    b, q, tok = _pair(n, v, 8)
    low = torch.finfo(dt).min
    b[:, 7::3], q[:, 7::3] = low, low
    b, q, tok = b.to(dt), q.to(dt), torch.full((n,), 1, dtype=torch.int32)
    keep = (b > low).numpy()
    base = pack_logits(b.to(DEV), mask_at=low)
    with KLDStats(n, DEV) as st:
        g, rows = st.run_grad_packed(base, q.to(DEV), tok.to(DEV), grad_dtype=torch.float32, per_row=True)
        assert st.result()["n_valid"] == n
    x, y = b.double().numpy(), q.double().numpy()
    span = np.where(keep, x, np.nan)
    d = (np.nanmax(span) - np.nanmin(span)) / 254
    for i in range(n):
        lp = np.where(keep[i], x[i], -np.inf)
        lp = lp - np.logaddexp.reduce(lp)
        lr = np.where(keep[i], y[i], -np.inf)
        lr = lr - np.logaddexp.reduce(lr)
        p, r = np.exp(lp), np.exp(lr)
        gap = np.where(keep[i], np.abs(np.where(keep[i], lp, 0.0) - np.where(keep[i], lr, 0.0)), 0.0)
        kl = (p * np.where(keep[i], np.where(keep[i], lp, 0.0) - np.where(keep[i], lr, 0.0), 0.0)).sum()
        assert abs(rows["kld"][i].item() - kl) <= 2 * d + math.expm1(2 * d) * (p * gap).sum() + 1e-6 + 1e-4 * kl
        off = np.abs(g[i].cpu().double().numpy() - (r - p))
        assert (off <= p * math.expm1(2 * d) + 4e-6 * (p + r) + 1e-12).all()


@pytest.mark.parametrize("quant", ["f32", "packed"])
@pytest.mark.parametrize("noise", [0.05, 0.4])
def test_what_eight_bits_change(noise, quant):
    """KL and gradient from checkpoints against those of the logits that were
    stored. A stored value is off by at most d = max(R / 254, 2^-21 max|x|) in
    a block that spans R, so with d the row's largest (e for quant rows, 0 when
    dense) ln p moves by 2d, p by a factor within e^(+-2d), and
    KL by |sum p' ((ln p' - ln p) - (ln r' - ln r)) + sum (p' - p) ln(p / r)|
    <= 2d + 2e + (e^(2d) - 1) sum p |ln(p / r)|."""
    n, v = 8, 5003
    g = torch.Generator().manual_seed(17)
    b, _, tok = _pair(n, v, 17)
    q = b + noise * torch.randn((n, v), generator=g)

    def off(x):
        t = torch.nn.functional.pad(x, (0, -v % 128), value=math.nan).view(n, -1, 128).numpy()
        span = np.nanmax(t, 2) - np.nanmin(t, 2)
        return np.maximum(span / 254, 2.0 ** -21 * np.nanmax(np.abs(t), 2)).max(1).astype(np.float64)

    base = pack_logits(b.to(DEV))
    other = pack_logits(q.to(DEV)) if quant == "packed" else q.to(DEV)
    d, e = off(b), off(q) if quant == "packed" else np.zeros(n)
    stored = np.abs(_np(base.unpack()).astype(np.float64) - b.numpy())
    assert (stored.max(1) <= d).all()
    with KLDStats(n, DEV) as st:
        grad, rows = st.run_grad_packed(base, other, tok.to(DEV), grad_dtype=torch.float32, per_row=True)
    kld, grad = rows["kld"].cpu().numpy(), grad.cpu().double().numpy()
    p, r = packed_ref.softmax(b.numpy()), packed_ref.softmax(q.numpy())
    ratio = np.log(p) - np.log(r)
    kl = (p * ratio).sum(1)
    assert (np.abs(kld - kl) <= 2 * d + 2 * e + np.expm1(2 * d) * (p * np.abs(ratio)).sum(1) + 1e-6 + 1e-4 * kl).all()
    far = p * np.expm1(2 * d)[:, None] + r * np.expm1(2 * e)[:, None] + 4e-6 * (p + r) * np.exp(2 * (d + e))[:, None]
    assert (np.abs(grad - (r - p)) <= far + 1e-12).all()


@pytest.mark.parametrize("quant", ["f32", "bf16", "packed"])
def test_long_rows_of_random_logits(quant):
    """2^22 + 77 and 2^25 + 1 columns a row, taken by one CTA or a cluster:
    a lane adds 10^3 to 10^5 terms, whose sums keep the tolerances."""
    g = torch.Generator(device=DEV).manual_seed(5)
    for n, v in ((1, (1 << 25) + 1), (6, (1 << 22) + 77), (400, (1 << 20) + 3)):
        b = torch.randn((n, v), generator=g, device=DEV) * 2.0
        q = b + torch.randn((n, v), generator=g, device=DEV) * 0.3
        q = q.to(DTYPES["f32" if quant == "packed" else quant])
        base = pack_logits(b)
        other = pack_logits(q) if quant == "packed" else q
        del b
        tok = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
        with KLDStats(n, device=DEV) as st:
            grad, rows = st.run_grad_packed(base, other, tok, scale=1.0, grad_dtype=torch.float32, per_row=True)
        for i in range(0, n, 57):
            lp = torch.log_softmax(base.rows(i, i + 1).unpack()[0].double(), 0)
            lr = torch.log_softmax((other.rows(i, i + 1).unpack()[0] if quant == "packed" else q[i]).double(), 0)
            p, r = lp.exp(), lr.exp()
            kl, nll = (p * (lp - lr)).sum().item(), -lr[tok[i].long()].item()
            assert abs(rows["kld"][i].item() - kl) <= 1e-6 + 1e-4 * kl, (v, rows["kld"][i].item(), kl)
            assert abs(rows["nll"][i].item() - nll) <= 1e-6 + 1e-4 * nll
            off = ((grad[i].double() - (r - p)).abs() - 1e-12) / (p + r)
            assert off.max().item() <= 4e-6, (v, i, off.max().item())
        del grad, q, base, other


@pytest.mark.parametrize("value", [0.1, 0.3, 0.45, 5.3])
@pytest.mark.parametrize("n,v", [(400, 151936), (400, 1 << 20), (1, 1 << 22), (1, 1 << 25)])
def test_long_rows_of_equal_values(n, v, value):
    """Equal terms round alike, so that the errors of a long fp32 sum add up."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for step in (0.0, 0.7):
        b = torch.full((n, v), value, device=DEV)
        b[:, ::2] -= step
        base = pack_logits(b)
        q = b.fill_(value).add_(0.3 * torch.randn((1, v), generator=g, device=DEV))
        tok = torch.zeros(n, dtype=torch.int32, device=DEV)
        with KLDStats(n, device=DEV) as st:
            grad, rows = st.run_grad_packed(base, q, tok, per_row=True)
        for i in (0, n - 1):
            lp = torch.log_softmax(base.rows(i, i + 1).unpack()[0].double(), 0)
            lr = torch.log_softmax(q[i].double(), 0)
            p, r = lp.exp(), lr.exp()
            kl, nll = (p * (lp - lr)).sum().item(), -lr[0].item()
            assert abs(rows["kld"][i].item() - kl) <= 1e-6 + 1e-4 * kl
            assert abs(rows["nll"][i].item() - nll) <= 1e-6 + 1e-4 * nll
            off = ((grad[i].double() - (r - p)).abs() - 1e-12) / (p + r)
            assert off.max().item() <= 4e-6, (step, i, off.max().item())


@pytest.mark.parametrize("quant", ["f32", "packed"])
@pytest.mark.parametrize("kind", ["rising", "masked", "shifting"])
def test_long_rows_whose_frames_move(kind, quant):
    """More than 256 chunks a warp, so that sums move to fp64, with frames and
    centres that change between the moves, and with masks in every block."""
    n, v = 380, (1 << 20) + 5
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn((1, v), generator=g, device=DEV).expand(n, v).contiguous()
    at = torch.linspace(0.0, 1.0, v, device=DEV)
    if kind == "rising":
        x += 80.0 * at
        q = x + 0.3 * torch.randn((1, v), generator=g, device=DEV)
    elif kind == "masked":
        x[:, 3::97] = -math.inf
        q = x + 0.3 * torch.randn((1, v), generator=g, device=DEV)
    else:  # the log-ratio drifts by 12 nats, past the polynomial's range
        x += 20.0 * at
        q = x - 12.0 * at + 0.3 * torch.randn((1, v), generator=g, device=DEV)
    base = pack_logits(x)
    other = pack_logits(q) if quant == "packed" else q
    tok = torch.full((n,), 1, dtype=torch.int32, device=DEV)
    with KLDStats(n, device=DEV) as st:
        grad, rows = st.run_grad_packed(base, other, tok, per_row=True)
    for i in (0, n - 1):
        lp = torch.log_softmax(base.rows(i, i + 1).unpack()[0].double(), 0)
        lr = torch.log_softmax((other.rows(i, i + 1).unpack()[0] if quant == "packed" else q[i]).double(), 0)
        p, r = lp.exp(), lr.exp()
        kl, nll = (p * (lp - lr)).nan_to_num(nan=0.0).sum().item(), -lr[1].item()
        assert abs(rows["kld"][i].item() - kl) <= 1e-6 + 1e-4 * kl
        assert abs(rows["nll"][i].item() - nll) <= 1e-6 + 1e-4 * nll
        assert ((grad[i].double() - (r - p)).abs() <= 4e-6 * (p + r) + 1e-12).all()
