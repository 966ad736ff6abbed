"""Operators over logit rows that stand around the KL statistic: 8-bit logit
checkpoints with the statistic and the gradient read from them, and beam
search's selection with the reordering of its states.

``listed()`` gives the cases, ``draw()`` more of the same ranges,
``prepare()`` the inputs a program has in hand, ``run()`` one pass and
``exact()`` the same outputs in 64 bits. With ``own`` false, ``run`` computes
every operator in elementary torch operations; with ``own`` true it makes
the calls a user of this package makes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128  # columns that share one header of an 8-bit checkpoint
EOS = 2


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The base model's logits of one 2048-token sequence go into the
        # checkpoint of a tuning run and are restored from it.
        {"name": "pack 2048x151936 bf16", "op": "pack", "n": 2048, "v": 151936, "dtype": "bf16", "pad": 0},
        # A short chunk with a ragged vocabulary whose last entries are padding
        # masks, kept in fp32.
        {"name": "pack 200x32003 f32 ragged", "op": "pack", "n": 200, "v": 32003, "dtype": "f32", "pad": 61},
        # Scoring one 8192-token context against saved base logits.
        {"name": "score 8192x151936 bf16", "op": "score", "n": 8192, "v": 151936, "quant": "bf16", "pad": 0},
        # A few positions over a large vocabulary: latency counts.
        {"name": "score 16x262144 f32", "op": "score", "n": 16, "v": 262144, "quant": "f32", "pad": 0},
        # A tuning step on one 2048-token sequence: loss and gradient against
        # the saved base logits.
        {"name": "grad 2048x151936 bf16", "op": "grad", "n": 2048, "v": 151936, "quant": "bf16", "grad": "bf16", "pad": 0},
        # The same with a ragged fp32 vocabulary and padding masks.
        {"name": "grad 512x32003 f32 ragged", "op": "grad", "n": 512, "v": 32003, "quant": "f32", "grad": "f32", "pad": 61},
        # A deferred backward pass: both models' logits come from checkpoints.
        {"name": "grad 2048x131072 packed", "op": "grad", "n": 2048, "v": 131072, "quant": "packed", "grad": "bf16", "pad": 1024},
        # One prompt, four beams: the smallest selection.
        {"name": "select 1x4x32000 bf16", "op": "select", "groups": 1, "beams": 4, "v": 32000, "dtype": "bf16", "k": 8, "done": 0},
        # Several prompts, some beams finished, a ragged vocabulary.
        {"name": "select 8x5x32003 f16", "op": "select", "groups": 8, "beams": 5, "v": 32003, "dtype": "f16", "k": 10, "done": 7},
        # A full serving batch.
        {"name": "select 32x8x151936 bf16", "op": "select", "groups": 32, "beams": 8, "v": 151936, "dtype": "bf16", "k": 16, "done": 0},
        # Caches of a short decode: one prompt, four beams.
        {"name": "reorder 1x4, 4 states", "op": "reorder", "groups": 1, "beams": 4, "layers": 2, "heads": 4, "time": 256, "dim": 64, "dtype": "bf16", "pattern": 1},
        # Caches of a full serving batch, every group at a length of its own.
        {"name": "reorder 16x8, 8 states", "op": "reorder", "groups": 16, "beams": 8, "layers": 4, "heads": 8, "time": 1024, "dim": 128, "dtype": "bf16", "pattern": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack", "score", "grad", "select", "reorder"])
    if op in ("pack", "score", "grad"):
        v = rng.choice([32000, 131072, 151936, 262144, _log(rng, 1000, 200000), _log(rng, 1000, 200000) | 1])
        most = 8192 * 151936 // 4  # elements; a quarter of the largest listed case
        n = _log(rng, 1, max(2, min(8192, most // v)))
        pad = rng.choice([0, 0, rng.randrange(1, 900)])
        if op == "pack":
            return {"op": op, "n": n, "v": v, "dtype": rng.choice(["f32", "bf16", "f16"]), "pad": pad}
        quant = rng.choice(["f32", "bf16", "f16", "packed"])
        if op == "score":
            return {"op": op, "n": n, "v": v, "quant": quant, "pad": pad}
        grad = rng.choice(["f32", "bf16"]) if quant == "packed" else rng.choice([quant, quant, "f32"])
        return {"op": op, "n": n, "v": v, "quant": quant, "grad": grad, "pad": pad}
    if op == "select":
        beams = rng.randrange(1, 17)
        groups = _log(rng, 1, max(2, 256 // beams))
        v = rng.choice([32000, 131072, 151936, _log(rng, 1000, 200000), _log(rng, 1000, 200000) | 1])
        k = rng.choice([beams, 2 * beams])
        return {"op": op, "groups": groups, "beams": beams, "v": v, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "k": k, "done": rng.choice([0, 0, rng.randrange(0, max(1, groups * beams // 2))])}
    beams = rng.randrange(2, 17)
    return {"op": op, "groups": _log(rng, 1, 64 // beams + 1), "beams": beams, "layers": rng.randrange(1, 5),
            "heads": rng.choice([1, 2, 4, 8]), "time": _log(rng, 16, 1500), "dim": rng.choice([40, 64, 96, 128]),
            "dtype": rng.choice(["bf16", "f16", "f32"]), "pattern": rng.randrange(1 << 20)}


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _pairs(n, v, pad, g):
    """Rows of base and quant logits, 512 at a time: N(0, 2.5^2) plus a boost
    by rank 12 r^-1.1 on a random permutation of the vocabulary; the quant
    rows differ by N(0, s^2), s one of 0.05, 0.15, 0.4 a row. The last `pad`
    columns are masked in both."""
    perm = torch.randperm(v, generator=g, device=DEV)
    boost = torch.empty(v, device=DEV)
    boost[perm] = 12.0 * torch.arange(1, v + 1, device=DEV, dtype=torch.float64).pow(-1.1).float()
    sigma = torch.tensor([0.05, 0.15, 0.4], device=DEV)
    for r in range(0, n, 512):
        m = min(512, n - r)
        b = torch.randn((m, v), generator=g, device=DEV).mul_(2.5).add_(boost)
        s = sigma[torch.randint(0, 3, (m, 1), generator=g, device=DEV)]
        q = torch.randn((m, v), generator=g, device=DEV).mul_(s).add_(b)
        if pad:
            b[:, v - pad:] = -math.inf
            q[:, v - pad:] = -math.inf
        yield r, r + m, b, q


def _blocks(x):
    """[N, V] -> fp32 [N, blocks, 128], -inf past V."""
    n, v = x.shape
    nb = -(-v // BLOCK)
    return torch.nn.functional.pad(x.float(), (0, nb * BLOCK - v), value=-math.inf).view(n, nb, BLOCK)


def _two(e):
    """2^e in fp32 for whole e in [-126, 127], by its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """Codes [N, blocks * 128] uint8, headers [N, blocks] int32 and the values
    they stand for (fp32 [N, V]). A block's step is the smallest power of two
    2^e, e >= floor(log2 max|x|) - 20, that spans it in 254 steps; codes count
    from one step below its least entry, 0 stands for -inf. A header holds
    base * 512 + (a code is 0) * 256 + e + 128. Scaling by powers of two and
    rounding to integers below 2^24 are exact in fp32."""
    t = _blocks(x)
    there = t != -math.inf
    some = there.any(-1)
    lo = torch.where(there, t, math.inf).amin(-1)
    lo = torch.where(some, lo, 0.0)
    hi = torch.where(some, t.amax(-1), 0.0)
    big = torch.maximum(lo.abs(), hi.abs())
    least = torch.where(big > 0, torch.frexp(big)[1] - 21, -126).clamp(min=-126)
    width = torch.where(hi > lo, torch.frexp(hi - lo)[1] - 8, -126)
    e = torch.maximum(width, least)
    up = _two(-e)
    e = e + (torch.round(hi * up) - torch.round(lo * up) > 254).int()
    up = _two(-e)
    base = torch.round(lo * up) - 1
    count = torch.where(there, torch.round(torch.where(there, t, 0.0) * up[..., None]) - base[..., None], 0.0)
    value = torch.where(there, (base[..., None] + count) * _two(e)[..., None], -math.inf)
    head = base.int() * 512 + (~there.all(-1)).int() * 256 + e.int() + 128
    head = torch.where(some, head, 256)
    n, v = x.shape
    return count.to(torch.uint8).view(n, -1), head, value.view(n, -1)[:, :v]


def _decode(codes, heads, v):
    """The fp32 values of [N, blocks * 128] codes."""
    n, nb = heads.shape
    c = codes.view(n, nb, BLOCK).float()
    step = _two(((heads & 255) - 128).clamp(min=-126))
    value = ((heads >> 9).float()[..., None] + c) * step[..., None]
    return torch.where(c > 0, value, -math.inf).view(n, -1)[:, :v]


def _forks(case):
    """Parents and lengths of a beam search that keeps each surviving beam in
    its slot and forks survivors into the slots of the dropped ones (the
    assignment that moves least): [groups][beams] and one length a group."""
    r = random.Random(case["pattern"])
    parents, lengths = [], []
    for _ in range(case["groups"]):
        w = case["beams"]
        live = sorted(r.sample(range(w), max(1, (w + 1) // 2)))
        parents.append([i if i in live else r.choice(live) for i in range(w)])
        lengths.append(r.randrange(case["time"] // 2, case["time"] + 1))
    return parents, lengths


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"op": op}
    if op in ("pack", "score", "grad"):
        n, v = case["n"], case["v"]
        s["v"] = v
        if op == "pack":
            s["x"] = torch.empty((n, v), dtype=TYPES[case["dtype"]], device=DEV)
            for r0, r1, b, _ in _pairs(n, v, case["pad"], g):
                s["x"][r0:r1] = b
            return s
        nb = -(-v // BLOCK)
        both = case["quant"] == "packed"
        s["codes"] = torch.empty((n, nb * BLOCK), dtype=torch.uint8, device=DEV)
        s["heads"] = torch.empty((n, nb), dtype=torch.int32, device=DEV)
        s["quant"] = (torch.empty_like(s["codes"]), torch.empty_like(s["heads"])) if both else torch.empty(
            (n, v), dtype=TYPES[case["quant"]], device=DEV)
        for r0, r1, b, q in _pairs(n, v, case["pad"], g):
            s["codes"][r0:r1], s["heads"][r0:r1], _ = _encode(b)
            if both:
                s["quant"][0][r0:r1], s["quant"][1][r0:r1], _ = _encode(q)
            else:
                s["quant"][r0:r1] = q
        s["tokens"] = torch.randint(0, max(1, v - case["pad"]), (n,), generator=g, device=DEV, dtype=torch.int32)
        s["scale"] = 1.0 / n
        s["grad"] = TYPES[case["grad"]] if op == "grad" else None
        if own:
            from logit_kl_divergence_b200 import KLDStats, PackedLogits
            s["handle"] = KLDStats(n)
            s["base"] = PackedLogits(s["codes"], s["heads"], v)
            s["other"] = PackedLogits(*s["quant"], v) if both else s["quant"]
        return s
    groups, beams = case["groups"], case["beams"]
    if op == "select":
        v = case["v"]
        s.update(k=case["k"], v=v)
        s["logits"] = torch.empty((groups * beams, v), dtype=TYPES[case["dtype"]], device=DEV)
        for r0, r1, b, _ in _pairs(groups * beams, v, 0, g):
            s["logits"][r0:r1] = b
        s["scores"] = torch.rand((groups, beams), generator=g, device=DEV).mul_(-20.0)
        s["done"] = None
        if case["done"]:
            s["done"] = torch.zeros(groups * beams, dtype=torch.bool, device=DEV)
            s["done"][torch.randperm(groups * beams, generator=g, device=DEV)[:case["done"]]] = True
            s["done"] = s["done"].view(groups, beams)
    else:
        parents, lengths = _forks(case)
        rows, dt = groups * beams, TYPES[case["dtype"]]
        shape = (rows, case["heads"], case["time"], case["dim"])
        s["states"] = [torch.randn(shape, generator=g, device=DEV).to(dt) for _ in range(2 * case["layers"])]
        s["tokens"] = torch.randint(0, 32000, (rows, case["time"]), generator=g, device=DEV, dtype=torch.int32)
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=DEV)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV).repeat_interleave(beams)
    if own:
        from logit_kl_divergence_b200 import BeamSearch
        s["handle"] = BeamSearch(groups, beams)
        if op == "reorder":
            s["bound"] = s["handle"].bind([(x, 2) for x in s["states"]] + [(s["tokens"], 1)])
    return s


# -------------------------------------------------------------- plain form

def _plain_rows(b, q, tokens):
    """KL, NLL of the tokens, both argmaxes (lowest index) and both softmaxes."""
    mb, mq = b.amax(1, keepdim=True), q.amax(1, keepdim=True)
    eb, eq = torch.exp(b - mb), torch.exp(q - mq)
    sb, sq = eb.sum(1, keepdim=True), eq.sum(1, keepdim=True)
    p, r = eb / sb, eq / sq
    ratio = ((b - mb) - (q - mq)) - (torch.log(sb) - torch.log(sq))
    kld = torch.where(p > 0, p * ratio, 0.0).sum(1)
    at = tokens.long()[:, None]
    nll = (mq + torch.log(sq) - q.gather(1, at))[:, 0]
    cols = torch.arange(b.shape[1], device=b.device, dtype=torch.int32)
    first = [torch.where(x == m, cols, b.shape[1]).amin(1) for x, m in ((b, mb), (q, mq))]
    return {"kld": kld, "nll": nll, "amax_b": first[0], "amax_q": first[1]}, p, r


def _plain_select(logits, scores, done, k):
    groups, beams = scores.shape
    x = logits.double()
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    s = scores.double().view(-1, 1) + (x - lse)
    if done is not None:
        only = torch.where(torch.arange(x.shape[1], device=x.device) == EOS, scores.double().view(-1, 1), -math.inf)
        s = torch.where(done.view(-1, 1), only, s)
    v = x.shape[1]
    order = torch.sort(s.view(groups, beams * v), dim=1, descending=True, stable=True)
    top, at = order.values[:, :k], order.indices[:, :k]
    none = top == -math.inf
    return (top.float(), torch.where(none, -1, at % v).int(),
            torch.where(none, -1, torch.div(at, v, rounding_mode="floor")).int())


def _plain_reorder(states, dims, parents, lengths):
    groups, beams = parents.shape
    rows = (parents.long() + torch.arange(groups, device=parents.device)[:, None] * beams).view(-1)
    for x, d in zip(states, dims):
        shape = [1] * x.dim()
        shape[d] = x.shape[d]
        at = torch.arange(x.shape[d], device=x.device).view(shape)
        keep = at < lengths.long()[rows].view([-1] + [1] * (x.dim() - 1))
        x.copy_(torch.where(keep, x[rows], x))
    return states


# --------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if own:
        return _own(state, op)
    if op == "pack":
        return _encode(state["x"])[2]
    if op in ("score", "grad"):
        b = _decode(state["codes"], state["heads"], state["v"])
        q = state["quant"]
        q = _decode(*q, state["v"]) if isinstance(q, tuple) else q.float()
        rows, p, r = _plain_rows(b, q, state["tokens"])
        if op == "grad":
            rows["grad"] = ((r - p) * state["scale"]).to(state["grad"])
        return rows
    if op == "select":
        return _plain_select(state["logits"], state["scores"], state["done"], state["k"])
    return _plain_reorder(state["states"] + [state["tokens"]], [2] * len(state["states"]) + [1], state["parents"],
                          state["lengths"])


def _own(state, op):
    if op == "pack":
        from logit_kl_divergence_b200 import pack_logits
        return pack_logits(state["x"]).unpack(torch.float32)
    h = state["handle"]
    if op in ("score", "grad"):
        base, quant = state["base"], state["other"]
        if op == "score":
            rows = h.run_packed(base, quant, state["tokens"], per_row=True)
        else:
            grad, rows = h.run_grad_packed(base, quant, state["tokens"], scale=state["scale"],
                                           grad_dtype=state["grad"], per_row=True)
            rows["grad"] = grad
        rows["kld"], rows["nll"] = rows["kld"].float(), rows["nll"].float()
        return rows
    if op == "select":
        return h.select(state["logits"], state["scores"], state["k"], finished=state["done"], eos=EOS)
    h.reorder(state["bound"], state["parents"], lengths=state["lengths"])
    return state["states"] + [state["tokens"]]


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("pack", "score", "grad"):
        n, v = case["n"], case["v"]
        nb = -(-v // BLOCK)
        packed = n * (v + 4 * nb)
        if op == "pack":  # read, checkpoint written and read back, values written
            return {"bytes": n * v * SIZE[case["dtype"]] + 2 * packed + 4 * n * v, "flops": 8 * n * v}
        quant = packed if case["quant"] == "packed" else n * v * SIZE[case["quant"]]
        rows = 28 * n
        if op == "score":
            return {"bytes": packed + quant + rows, "flops": 10 * n * v}
        return {"bytes": packed + quant + rows + n * v * SIZE[case["grad"]], "flops": 14 * n * v}
    if op == "select":
        live = case["groups"] * case["beams"] - case["done"]
        return {"bytes": live * case["v"] * SIZE[case["dtype"]] + 12 * case["groups"] * case["k"] + 4 * live,
                "flops": 4 * live * case["v"]}
    parents, lengths = _forks(case)
    per = 2 * case["layers"] * case["heads"] * case["dim"] * SIZE[case["dtype"]] + 4
    total = 0
    for p, n in zip(parents, lengths):
        moved = [x for i, x in enumerate(p) if x != i]
        total += (len(moved) + len(set(moved))) * n * per
    return {"bytes": total + 8 * case["groups"] * case["beams"], "flops": 0}


# ------------------------------------------------------------------- exact

def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, heads, v):
    heads = heads.long()
    e = (heads % 256 - 128).double()
    base = torch.div(heads, 512, rounding_mode="floor").double()
    c = codes.reshape(codes.shape[0], -1, BLOCK).double()
    x = (c + base[:, :, None]) * _two64(e)[:, :, None]
    x[c == 0] = -math.inf
    return x.flatten(1)[:, :v]


def _exact_pack(x):
    """Every block's step and codes from their definition in 64 bits."""
    n, v = x.shape
    full = torch.full((n, -(-v // BLOCK) * BLOCK), -math.inf, dtype=torch.float64, device=x.device)
    full[:, :v] = x
    t = full.view(n, -1, BLOCK)
    masked = torch.isinf(t)
    lo = t.masked_fill(masked, math.inf).min(2).values
    hi = t.max(2).values
    empty = masked.all(2)
    lo[empty] = 0.0
    hi[empty] = 0.0
    big = torch.maximum(lo.abs(), hi.abs())
    e = torch.floor(torch.log2(big.clamp(min=2.0 ** -160))).sub(20).clamp(min=-126)
    spread = torch.floor(torch.log2((hi - lo).clamp(min=2.0 ** -200))) - 8
    e = torch.maximum(e, spread)  # at least two steps finer than what can span the block, unless the floor holds it
    for _ in range(4):
        wide = torch.round(hi * _two64(-e)) - torch.round(lo * _two64(-e)) > 254
        e = e + wide.double()
    y = torch.round(t.masked_fill(masked, 0.0) * _two64(-e)[..., None]) * _two64(e)[..., None]
    return y.masked_fill(masked, -math.inf).flatten(1)[:, :v]


def exact(case, seed):
    op = case["op"]
    if op == "reorder":
        return None
    s = prepare(case, seed)
    if op == "pack":
        return torch.cat([_exact_pack(x.double()) for x in s["x"].split(256)])
    if op == "select":
        x = s["logits"].double()
        x = x - torch.logsumexp(x, 1, keepdim=True) + s["scores"].double().reshape(-1, 1)
        if s["done"] is not None:
            d = s["done"].reshape(-1)
            x[d] = -math.inf
            x[d, EOS] = s["scores"].double().reshape(-1)[d]
        best = torch.topk(x.view(case["groups"], -1), case["k"], dim=1).values
        return best, None, None
    out = {"kld": [], "nll": [], "grad": []}
    for r in range(0, case["n"], 256):
        c = slice(r, r + 256)
        b = torch.log_softmax(_exact_values(s["codes"][c], s["heads"][c], s["v"]), 1)
        q = s["quant"]
        q = _exact_values(q[0][c], q[1][c], s["v"]) if isinstance(q, tuple) else q[c].double()
        q = torch.log_softmax(q, 1)
        p = b.exp()
        out["kld"].append((p * (b - q)).masked_fill(p == 0, 0.0).sum(1))
        out["nll"].append(-q[torch.arange(q.shape[0], device=q.device), s["tokens"][c].long()])
        if op == "grad":
            out["grad"].append((q.exp() - p) * s["scale"])
    return {k: torch.cat(v) if v else None for k, v in out.items()}
