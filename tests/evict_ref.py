"""Plain 64-bit forms of the operators that bound a paged cache (numpy), on the batches of tests/paged_ref.py."""
import numpy as np

from tests.paged_ref import F32_STEP


def rows_of(b, d, n=None):
    """(page, slot) of the first n positions of sequence d."""
    pos = np.arange(b.lens[d][1] if n is None else n)
    return b.table[d, pos // b.page], pos % b.page


def random_weights(rng, b, ties=False):
    w = np.exp(rng.standard_normal((b.num_pages, b.n_kv, b.page)) - 2).astype(np.float32)
    if ties:
        w = np.round(w * 8) / 8
    w[rng.random(w.shape) < 0.1] = 0.0
    return w.astype(np.float32)


def weigh(b, q, lse, weights, group, sm_scale):
    """weights after the call and a bound of what FP32 loses: products are exact, sums FP32.

    With lse as given, a logit minus it is off by dl = scale (D + 2) 2^-23 sum |q k| + 2^-22 (|logit| + |lse| + 1) (the
    sum, the scalings to base 2, their difference), its exponential by expm1(dl) + 2^-21, the sum of n by n 2^-23."""
    out, tol = weights.astype(np.float64), np.zeros(weights.shape)
    K = b.rows["k"]
    for d, (t, s) in enumerate(b.lens):
        if t == 0:
            continue
        page, slot = rows_of(b, d)
        for h in range(b.n_kv):
            k = K[b.cu_k[d]:b.cu_k[d] + s, h]
            total, err = np.zeros(s), np.zeros(s)
            for i in range(t):
                for g in range(group):
                    r, hh = b.cu_q[d] + i, h * group + g
                    if lse[r, hh] == -np.inf:
                        continue
                    lg = sm_scale * (k @ q[r, hh])
                    mag = sm_scale * (np.abs(k) @ np.abs(q[r, hh]))
                    see = np.arange(s) <= s - t + i
                    w = np.where(see, np.exp(np.where(see, lg - lse[r, hh], -np.inf)), 0.0)
                    dl = (b.D + 2) * F32_STEP * mag + 2.0 ** -22 * (np.abs(lg) + abs(lse[r, hh]) + 1)
                    total += w
                    err += w * (np.expm1(dl) + 2.0 ** -21)
            old = np.where(np.arange(s) < s - t, out[page, h, slot], 0.0)
            out[page, h, slot] = old + total
            tol[page, h, slot] = err * 1.01 + (t * group + 2) * F32_STEP * total + F32_STEP * (old + total)
    return out, tol


def select(b, weights, budget, sinks, recent, shared):
    """kept, kept_len"""
    heads = 1 if shared else b.n_kv
    kept = np.full((len(b.lens), heads, budget), -1, np.int32)
    for d, (_, s) in enumerate(b.lens):
        page, slot = rows_of(b, d)
        w = np.stack([weights[page, h, slot] for h in range(b.n_kv)]).astype(np.float32)
        if shared:
            total = w[0]
            for h in range(1, b.n_kv):
                total = (total + w[h]).astype(np.float32)
            w = total[None]
        for h in range(heads):
            order = sorted(range(s), key=lambda i: (not (i < sinks or i >= s - recent), np.isnan(w[h, i]),
                                                    0.0 if np.isnan(w[h, i]) else -float(w[h, i]), i))
            best = sorted(order[:budget])
            kept[d, h, :len(best)] = best
    return kept, np.array([min(s, budget) for _, s in b.lens], np.int32)


def compact(b, tensors, kept, kept_len):
    """Copies of the tensors [pages, heads, page, ...] with the kept rows moved."""
    out = {n: t.copy() for n, t in tensors.items()}
    for d in range(len(b.lens)):
        n = int(kept_len[d])
        page, slot = rows_of(b, d, n)
        for h in range(b.n_kv):
            src = kept[d, h if kept.shape[1] > 1 else 0, :n]
            for name, t in tensors.items():
                out[name][page, h, slot] = t[b.table[d, src // b.page], h, src % b.page]
    return out
