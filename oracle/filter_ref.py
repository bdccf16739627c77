"""Temperature, top-k, top-p and min-p (test infrastructure only).

"解码：采样、束搜索和推测性解码": the sampling strategies of its first sections
(temperature divides the logits; top-k keeps the k most probable tokens; top-p the
smallest set of the most probable tokens whose probabilities reach p) and "Gumbel
Max技巧" for the draw. Readings: tokens of equal logits count in index order; the
scaled logit is the float32 product with the float32 reciprocal of the temperature,
as in sample_ref; top-p counts within what top-k leaves; min-p keeps tokens of at
least m times the largest probability; a logit of -inf is masked and never kept.
Sums are long doubles.
"""

import math

import numpy as np


def _order(x):
    """Indices by (value descending, index ascending), NaN first."""
    first = np.where(np.isnan(x), 1, 0)
    value = np.where(np.isnan(x), 0, x).astype(np.float64) + 0.0
    return np.lexsort((np.arange(len(x)), -value, -first))


def filter_ref(logits, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (keep bool [V], scaled float32 [V], weights float128 [V] of all
    tokens relative to the largest, margin). margin is how far the top-p border's
    sum is from its target, as a share of the whole (inf where top-p is off): where
    it is tiny, an evaluation with rounded weights may put the border elsewhere (inf too
    where all weights that count are equal)."""
    x = np.asarray(logits, np.float32)
    v = len(x)
    keep = np.zeros(v, bool)
    order = _order(x)
    if temperature == 0:
        if not x[order[0]] == -np.inf:
            keep[order[0]] = True
        return keep, x, keep.astype(np.longdouble), math.inf
    inv = np.float32(1.0) / np.float32(temperature)
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.multiply(x, inv, dtype=np.float32)
    allowed = ~(x == -np.inf)
    if not allowed.any():
        return keep, s, np.zeros(v, np.longdouble), math.inf
    top = s[order[0]]
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        if np.isfinite(top):
            w = np.exp(s.astype(np.longdouble) - np.longdouble(top))
        else:
            w = (np.isnan(s) if np.isnan(top) else s == top).astype(np.longdouble)
    w = np.where(allowed, w, 0)
    n = int(allowed.sum())                    # masked tokens come last in the order
    if top_k and top_k < v:
        n = min(n, top_k)
    margin = math.inf
    if top_p < 1:
        sums = np.cumsum(w[order[:n]])
        target = np.longdouble(np.float32(top_p)) * sums[-1]
        m = int(np.searchsorted(sums, target, side="left")) + 1      # the first sum that reaches it
        m = min(m, n)
        near = [abs(sums[i] - target) / sums[-1] for i in (m - 2, m - 1) if 0 <= i < n - 1]
        some = w[order[:len(sums)]]
        equal = bool(((some == some[0]) | (some < 2.0 ** -70)).all())   # sums of one weight are exact everywhere
        margin = float(min(near)) if near and np.isfinite(top) and not equal else math.inf
        n = m
    keep[order[:n]] = True
    if min_p > 0:
        if np.isfinite(top):
            with np.errstate(invalid="ignore"):
                keep &= s.astype(np.float64) - np.float64(top) >= math.log(np.float32(min_p))
        else:
            keep &= w > 0
    return keep, s, w, margin


def draw_ref(keep, scaled, weights, gumbel):
    """(token, logp) from what is kept: the first argmax of the float32 sums; a
    row that keeps nothing gives token 0 and -inf."""
    if not keep.any():
        return 0, -math.inf
    with np.errstate(invalid="ignore"):
        got = np.add(scaled, np.asarray(gumbel, np.float32), dtype=np.float32)
    at = np.nonzero(keep)[0]
    token = int(at[_order(got[at])[0]])
    total = weights[keep].sum()
    return token, float(np.log(weights[token]) - np.log(total)) if weights[token] > 0 else -math.inf
