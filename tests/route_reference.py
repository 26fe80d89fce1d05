"""Routing to experts in 64 bits, from its definition, one token at a time."""
import numpy as np


def route(logits, k, score, bias=None, n_groups=1, top_groups=1, top2=False, renorm=True, scale=1.0):
    """(ids [T][k], gates [T][k] in 64 bits) of logits [T][E] (any float array)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.zeros((T, k), np.int64)
    gates = np.zeros((T, k))
    with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
        for t in range(T):
            l = np.where(np.isnan(logits[t]), -np.inf, logits[t])
            live = l > -np.inf
            if score == "sigmoid":
                s = np.where(live, 1 / (1 + np.exp(-l)), 0.0)
            else:
                e = np.where(live, np.exp(l - (l.max() if live.any() else 0.0)), 0.0)
                s = e / e.sum() if live.any() else e
            v = s + (0.0 if bias is None else np.asarray(bias, np.float64))
            c = l if bias is None else v
            stay = np.ones(E, bool)
            if n_groups > 1:
                n = E // n_groups
                g = []
                for h in range(n_groups):
                    of = np.sort((v if top2 else c)[h * n:(h + 1) * n][live[h * n:(h + 1) * n]])[::-1]
                    g.append(-np.inf if not len(of) else of[:2].sum() if top2 else of[0])
                order = np.argsort(-np.array(g), kind="stable")
                stay[:] = False
                for h in order[:top_groups]:
                    stay[h * n:(h + 1) * n] = True
            rank = np.argsort(-np.where(live & stay, c, -np.inf), kind="stable")
            rank = [e for e in rank if live[e] and stay[e]] + [e for e in range(E) if stay[e] and not live[e]]
            ids[t] = rank[:k]
            chosen = s[ids[t]]
            if renorm:
                if score == "softmax" or l[ids[t]].max() < -600:  # quotients of what 64 bits lose, too
                    top = l[ids[t]].max()
                    chosen = np.where(live[ids[t]], np.exp(l[ids[t]] - top), 0.0) if top > -np.inf else chosen
                total = chosen.sum()
                chosen = chosen / total if total > 0 else chosen
            gates[t] = chosen * scale
    return ids, gates


def gate_tolerance(logits, ids, gates):
    """How far fp32 gates may be off.  In steps of 2^-24 of the gate: the difference of two logits |d| (its rounding
    is an error of the exponent), expf 4, the sum over all experts 70 (its terms as the numerator, the mean of |d| at
    most ln 1024, 37 additions), the k chosen 12 more, quotient and scale 2: 96 + |d|.  
    Gates below 2^-126 may be lost."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    top = l.max(1, keepdims=True)
    of = np.take_along_axis(l, ids, 1)
    with np.errstate(invalid="ignore"):
        d = np.where(of > -np.inf, np.abs(top - of), 0.0)
    d = np.where(np.isfinite(d), d, 0.0)
    return np.abs(gates) * (96 + d) * 2.0 ** -24 + 2.0 ** -126 * (gates > 0)
