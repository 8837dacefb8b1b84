"""Plain references of the beam search operators (numpy, fp64), and the bound on the scores."""
import numpy as np

# A score is cum + (x - max) - log(sum). The sum is off by at most one 2^-24 for each of the 32 values that a
# thread adds one after another and each of the few dozen joins behind it, plus the exponential's 2^-22 and its
# argument's rounding (2^-23 times the distance to the maximum, which its factor exp(-distance) <= 1/distance
# outweighs): below 2^-17 of the sum, hence of the logarithm. fp32 scores add half a step.
LSE_BOUND = 2.0 ** -17


def select(logits, scores, K, *, rows=None, finished=None, eos=-1):
    """logits: [R, V] fp64 values; returns scores (fp64), parents, tokens [batch, K], and for each batch entry the
    sorted (score, beam) list one past K, for a test to see how close its choices are."""
    batch, beams = scores.shape
    V = logits.shape[1]
    out = np.full((batch, K), -np.inf), np.full((batch, K), -1), np.full((batch, K), -1)
    margins = []
    for b in range(batch):
        found = []
        for j in range(beams):
            cum = float(scores[b, j])
            if not cum > -np.inf:
                continue
            if finished is not None and finished[b, j]:
                found.append((cum, j, 0.0, eos))
                continue
            x = logits[b * beams + j if rows is None else rows[b, j]]
            x = np.where(np.isnan(x), -np.inf, x)
            top = x.max()
            if top == -np.inf:
                continue
            term = (x == top).astype(np.float64)
            rest = (x != top) & (x > -np.inf)
            if top < np.inf:
                term[rest] = np.exp(x[rest] - top)
            norm = np.log(term.sum())
            best = np.lexsort((np.arange(V), -x))[:K + 1]
            for t in best:
                if x[t] > -np.inf and not (top == np.inf and x[t] != top):
                    found.append((cum + ((0.0 if x[t] == top else x[t] - top) - norm), j, -x[t], int(t)))
        found.sort(key=lambda f: (-f[0], f[1], f[2], f[3]))
        margins.append([(f[0], f[1]) for f in found[:K + 1]])
        for k, f in enumerate(found[:K]):
            out[0][b, k], out[1][b, k], out[2][b, k] = f[0], f[1], f[3]
    return *out, margins


def clear(margins):
    """Whether no two neighbours of different beams are so close that rounding could swap them."""
    return all(a[1] == b[1] or a[0] == b[0] or a[0] - b[0] > 4 * LSE_BOUND for m in margins for a, b in zip(m, m[1:]))


def reorder(slots, parents):
    """New slots, and the (source, destination) copies."""
    new, copies = np.empty_like(slots), []
    for b, (row, par) in enumerate(zip(slots, parents)):
        n = len(row)
        taken = {int(p) for p in par if 0 <= p < n}
        free = [int(row[j]) for j in range(n) if j not in taken]
        seen = set()
        for j, p in enumerate(par):
            p = int(p)
            if 0 <= p < n and p not in seen:
                seen.add(p)
                new[b, j] = row[p]
            else:
                new[b, j] = free.pop(0)
                if 0 <= p < n:
                    copies.append((int(row[p]), int(new[b, j])))
    return new, copies
