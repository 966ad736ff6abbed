"""Plain numpy implementations in 64 bits that the tests of the logit
checkpoints and of beam search compare against. They share no code with the
package."""
import numpy as np

BLOCK = 128


def pack(x: np.ndarray):
    """Codes, headers and values of the 8-bit format (include/kld_stats.h),
    block by block from its definition: the smallest e that fits."""
    n, v = x.shape
    nb = -(-v // BLOCK)
    t = np.full((n, nb * BLOCK), -np.inf)
    t[:, :v] = x.astype(np.float64)
    t = t.reshape(n * nb, BLOCK)
    bad = (np.isnan(t) | (t == np.inf) | (np.isfinite(t) & (np.abs(t) >= 2.0 ** 126))).any(1)
    there = np.isfinite(t)
    some = there.any(1)
    lo = np.where(some, np.where(there, t, np.inf).min(1), 0.0)
    hi = np.where(some, np.where(there, t, -np.inf).max(1), 0.0)
    big = np.maximum(np.abs(lo), np.abs(hi))
    with np.errstate(divide="ignore"):
        e = np.where(big > 0, np.floor(np.log2(big)) - 20, -126)
    e = np.maximum(e, -126).astype(np.int64)
    for _ in range(400):
        scale = np.ldexp(1.0, -e)
        wide = (np.rint(hi * scale) - np.rint(lo * scale) > 254) & ~bad
        if not wide.any():
            break
        e = e + wide
    scale = np.ldexp(1.0, -e)
    base = np.rint(lo * scale) - 1
    code = np.where(there, np.rint(np.where(there, t, 0.0) * scale[:, None]) - base[:, None], 0)
    value = np.where(there, (base[:, None] + code) * np.ldexp(1.0, e)[:, None], -np.inf)
    head = base.astype(np.int64) * 512 + (~there.all(1)) * 256 + e + 128
    head = np.where(some, head, 256)
    head = np.where(bad, 511, head)
    code = np.where(bad[:, None], 0, code)
    value = np.where(bad[:, None], np.nan, value)
    head = ((head + 2 ** 31) % 2 ** 32 - 2 ** 31).astype(np.int32)
    return (code.astype(np.uint8).reshape(n, -1), head.reshape(n, nb),
            value.reshape(n, -1)[:, :v])


def softmax(x: np.ndarray) -> np.ndarray:
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
        return e / e.sum(1, keepdims=True)


def relative_row(b: np.ndarray, q: np.ndarray):
    """KL of one row pair and ln softmax of both, from differences to the
    rows' maxima: also right for rows near the type's lowest value, where
    x - lse in fp64 loses lse's logarithm."""
    x, y = b.astype(np.float64) - float(b.max()), q.astype(np.float64) - float(q.max())
    lp, lr = x - np.log(np.exp(x).sum()), y - np.log(np.exp(y).sum())
    p = np.exp(lp)
    return float((p[p > 0] * (lp - lr)[p > 0]).sum()), lp, lr


def select(logits: np.ndarray, scores: np.ndarray, k: int, finished=None, eos=0):
    """Beam selection of [groups * beams, V] logits: scores (fp64), tokens and
    parents, each [groups, k]."""
    groups, beams = scores.shape
    v = logits.shape[1]
    out = (np.full((groups, k), -np.inf), np.full((groups, k), -1), np.full((groups, k), -1))
    x = logits.astype(np.float64).reshape(groups, beams, v)
    for g in range(groups):
        cand = np.full((beams, v), -np.inf)
        for w in range(beams):
            s = float(scores[g, w])
            if not -np.inf < s < np.inf:
                continue
            if finished is not None and finished[g, w]:
                cand[w, eos] = s
                continue
            row = x[g, w]
            m = row.max()
            if np.isnan(row).any() or m == np.inf or m == -np.inf:
                continue
            rel = row - m
            cand[w] = s + (rel - np.log(np.exp(rel).sum()))
        flat = cand.reshape(-1)
        order = np.argsort(-flat, kind="stable")[:k]
        order = order[flat[order] > -np.inf]
        out[0][g, :len(order)] = flat[order]
        out[1][g, :len(order)] = order % v
        out[2][g, :len(order)] = order // v
    return out


def reorder(x: np.ndarray, parents: np.ndarray, lengths=None, time_dim=None) -> np.ndarray:
    """What in-place reordering leaves in a state [groups * beams, ...]."""
    groups, beams = parents.shape
    y = x.copy()
    for g in range(groups):
        for w in range(beams):
            p = int(parents[g, w])
            if not 0 <= p < beams:
                continue
            src, dst = g * beams + p, g * beams + w
            if lengths is None or time_dim is None:
                y[dst] = x[src]
            else:
                n = min(max(int(lengths[src]), 0), x.shape[time_dim])
                at = (slice(None),) * (time_dim - 1) + (slice(0, n),)
                y[dst][at] = x[src][at]
    return y
