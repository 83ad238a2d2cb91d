"""Plain numpy float64 forms of the serving operators around the quantised
layers (test infrastructure), and their tolerances.

A rounding to a type is off by at most half a step, HALF[t] relative (below the
type's normal range half of its smallest step, TINY[t]); F32 bounds what the
float32 arithmetic before it adds, stated where it is used."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10, "f32": 2.0 ** -150}
MIN_SCALE = 2.0 ** -100


def e4m3_values(codes):
    """E4M3 codes -> float64 values."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def rms_norm(x, r, w, eps):
    """float64 rows -> (s, y)."""
    s = x.astype(np.float64) if r is None else x.astype(np.float64) + r.astype(np.float64)
    big = np.maximum(np.abs(s).max(-1, keepdims=True), 1.0)  # far from float64's range all the same
    mean = ((s / big) ** 2).mean(-1, keepdims=True) * big * big
    y = s / np.sqrt(mean + eps)
    return s, y if w is None else y * w.astype(np.float64)


def route(logits, topk, scoring="softmax", bias=None, n_group=1, topk_group=1, group_score="max", renormalize=True,
          routed_scale=1.0):
    """One row at a time: (weights float64 [M, topk], ids int32 [M, topk])."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    weights, ids = np.zeros((M, topk)), np.zeros((M, topk), np.int32)
    for m in range(M):
        row = l[m]
        if scoring == "softmax":
            if row.max() == -np.inf:
                s = np.zeros(E)
            else:
                ex = np.exp(row - row.max())
                s = ex / ex.sum()
        else:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-row))
        c = (s if bias is None else s + np.asarray(bias, np.float64)).astype(np.float32)
        order = row if bias is None else c.astype(np.float64)
        open_ = list(range(E))
        if n_group > 1:
            per = E // n_group
            value = []
            for g in range(n_group):
                if group_score == "max":
                    value.append(order[g * per:(g + 1) * per].max())
                else:
                    best = np.sort(c[g * per:(g + 1) * per])[::-1]
                    value.append(np.float32(best[0] + best[1]))
            chosen = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            open_ = [e for e in range(E) if e // per in chosen]
        sel = sorted(open_, key=lambda e: (-order[e], e))[:topk]
        if scoring == "softmax" and renormalize:
            top = row[sel].max()  # not through scores that underflow
            w = np.zeros(topk) if top == -np.inf else np.exp(row[sel] - top)
        else:
            w = s[sel]
        if renormalize and w.sum() > 0:
            w = w / w.sum()
        weights[m], ids[m] = w * routed_scale, sel
    return weights, ids
