"""float64 oracle of what stands in front of the experts: the residual norm, its gradient, and the
softmax router with groups.  The definitions, in numpy.
"""
import numpy as np


def rms_norm(s, weight, eps):
    """(y, r) of the rows s (after the residual's addition)."""
    r = 1.0 / np.sqrt((s * s).mean(-1) + eps)
    return s * r[..., None] * weight, r


def rms_norm_backward(dy, s, weight, eps, dsum=0.0):
    """(dx, dweight): y_i = w_i s_i r and dr/ds_i = -s_i r^3 / H."""
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    along = (dy * weight * s).mean(-1, keepdims=True)
    return dsum + dy * weight * r - s * r ** 3 * along, (dy * s * r).sum(0)


def route_softmax_grouped(logits, top_k, groups, selected, top_two, renormalize, scale, bias=None):
    """(idx [T, k], w [T, k]); ties go to the lower group and expert.  Rows with a NaN, a +inf or only
    -inf, and all rows with a NaN bias: ids 0..k-1 and NaN."""
    T, E = logits.shape
    idx = np.tile(np.arange(top_k), (T, 1))
    w = np.full((T, top_k), np.nan)
    for t, x in enumerate(logits.astype(np.float64)):
        m = x.max()
        if np.isnan(x).any() or not np.isfinite(m) or (bias is not None and np.isnan(bias).any()):
            continue
        z = np.exp(x - m)
        p = z / z.sum()
        c = p if bias is None else p + bias.astype(np.float64)
        # without a bias the exact softmax's ranking is the logits'
        rank = x if bias is None else c
        parts = np.sort(c.reshape(groups, -1), -1)[:, ::-1]
        if top_two:
            score = np.where(parts[:, 0] == np.inf, np.inf, parts[:, 0] + parts[:, 1])
        else:
            score = rank.reshape(groups, -1).max(-1)
        kept = np.argsort(-score, kind="stable")[:selected]
        ids = np.flatnonzero(np.isin(np.arange(E) // (E // groups), kept))
        idx[t] = ids[np.argsort(-rank[ids], kind="stable")[:top_k]]
        chosen = x[idx[t]]
        if renormalize:
            with np.errstate(invalid="ignore"):
                q = np.exp(chosen - chosen.max())
            w[t] = q / q.sum() * scale
        else:
            w[t] = p[idx[t]] * scale
    return idx, w
