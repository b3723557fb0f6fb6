"""fp64 definition of the general routing, the router losses and their gradient in the
logits (test-only, CPU, numpy). Conventions as stated in include/moe.h."""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def clean(logits) -> np.ndarray:
    """fp64 logits with NaN as -inf and +inf as the largest float."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, FLT_MAX)


def softmax(l: np.ndarray) -> np.ndarray:
    m = l.max(axis=1, keepdims=True)
    x = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
    s = x.sum(axis=1, keepdims=True)
    return x / np.where(s > 0, s, 1.0)


def sigmoid(l: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return np.where(np.isneginf(l), 0.0, 1.0 / (1.0 + np.exp(-l)))


def scores(l, scoring: str) -> np.ndarray:
    return sigmoid(l) if scoring == "sigmoid" else softmax(l)


def _first_largest(values, open_) -> int:
    """Index of the largest open value, the lowest index among equal ones."""
    best = -1
    for i, v in enumerate(values):
        if open_[i] and (best < 0 or v > values[best]):
            best = i
    return best


def route(logits, k: int, scoring="softmax", num_groups=1, topk_groups=1, group_top=1,
          renormalize=True, scale=1.0, bias=None):
    """(idx [T, k], w [T, k]): the definition, one token and one choice at a time."""
    l = clean(logits)
    t_count, e_count = l.shape
    s = scores(l, scoring)
    # without a bias experts are compared by their logits (both scores rise with them), and
    # so are groups by one expert each
    c = l if bias is None else s + np.asarray(bias, dtype=np.float64)
    c = np.where(np.isnan(c), -np.inf, c)
    by_group = s if bias is None and group_top > 1 else c
    gs = e_count // num_groups
    idx = np.empty((t_count, k), dtype=np.int32)
    for t in range(t_count):
        open_ = np.ones(e_count, dtype=bool)
        if num_groups > 1:
            value = []
            for g in range(num_groups):
                v = np.sort(by_group[t, g * gs:(g + 1) * gs])[::-1][:group_top]
                value.append(np.inf if np.isposinf(v).any() else v.sum())
            free = np.ones(num_groups, dtype=bool)
            for _ in range(topk_groups):
                free[_first_largest(value, free)] = False
            open_ = np.repeat(~free, gs)
        for j in range(k):
            idx[t, j] = _first_largest(c[t], open_)
            open_[idx[t, j]] = False
    return idx, weights(l, idx, scoring, renormalize, scale)


def weights(logits, idx, scoring="softmax", renormalize=True, scale=1.0) -> np.ndarray:
    """w [T, k] of the chosen experts (idx outside [0, E): weight 0)."""
    l = clean(logits)
    ok = (idx >= 0) & (idx < l.shape[1])
    at = np.where(ok, idx, 0)
    ls = np.where(ok, np.take_along_axis(l, at, 1), -np.inf)
    if scoring == "softmax" and renormalize:
        return softmax(ls) * scale
    s = np.where(ok, np.take_along_axis(scores(l, scoring), at, 1), 0.0)
    if renormalize:
        tot = s.sum(axis=1, keepdims=True)
        s = s / np.where(tot > 0, tot, 1.0)
    return s * scale


def probs(l, scoring: str) -> np.ndarray:
    s = scores(l, scoring)
    tot = s.sum(axis=1, keepdims=True)
    return s / np.where(tot > 0, tot, 1.0)


def logsumexp(l: np.ndarray) -> np.ndarray:
    m = l.max(axis=1)
    dead = np.isneginf(m)
    x = np.exp(l - np.where(dead, 0.0, m)[:, None])
    return np.where(dead, 0.0, m + np.log(np.where(dead, 1.0, x.sum(axis=1))))


def losses(logits, idx, scoring="softmax", mask=None, counts=None):
    """(losses [2], counts [E + 1], P [E])."""
    l = clean(logits)
    e_count = l.shape[1]
    keep = np.ones(l.shape[0], dtype=bool) if mask is None else np.asarray(mask).astype(bool)
    n = int(keep.sum())
    if counts is None:
        named = np.asarray(idx)[keep].ravel()
        named = named[(named >= 0) & (named < e_count)]
        counts = np.concatenate([np.bincount(named, minlength=e_count), [n]]).astype(np.int64)
    p = probs(l, scoring)[keep].sum(axis=0) / max(n, 1)
    balance = e_count * float((counts[:e_count] / max(n, 1) * p).sum())
    z = float((logsumexp(l[keep]) ** 2).sum()) / max(n, 1) if n else 0.0
    return np.array([balance, z]), counts, p


def route_backward(logits, idx, scoring="softmax", renormalize=True, scale=1.0, d_w=None,
                   counts=None, d_losses=None, mask=None):
    """(gradient [T, E], size [T, E]): the gradient, and the sum of the magnitudes of the
    terms that are added up in it (what rounding errors are relative to)."""
    l = clean(logits)
    t_count, e_count = l.shape
    s, soft = scores(l, scoring), softmax(l)
    live = ~np.isneginf(l)
    grad, size = np.zeros_like(s), np.zeros_like(s)
    rest = np.where(live, sigmoid(-np.where(live, l, 0.0)), 0.0)      # 1 - sigmoid
    for t in range(t_count):
        if d_w is not None:
            slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < e_count]
            g = np.array([scale * float(d_w[t, j]) for j in slots])
            at = np.array([idx[t, j] for j in slots], dtype=int)
            if len(slots):
                if renormalize:
                    u = weights(l[t:t + 1], idx[t:t + 1], scoring, True, 1.0)[0][slots]
                    term, mag = u * (g - (g * u).sum()), u * (abs(g) + (abs(g) * u).sum())
                    if scoring == "sigmoid":
                        term, mag = term * rest[t, at], mag * rest[t, at]
                elif scoring == "sigmoid":
                    term = s[t, at] * rest[t, at] * g
                    mag = abs(term)
                else:
                    u = s[t, at]
                    term, mag = u * g, abs(u * g)
                    grad[t] -= s[t] * (u * g).sum()
                    size[t] += s[t] * abs(u * g).sum()
                np.add.at(grad[t], at, term)
                np.add.at(size[t], at, mag)
        if d_losses is not None and (mask is None or mask[t]):
            n = max(int(counts[e_count]), 1)
            c = float(d_losses[0]) * e_count * np.asarray(counts[:e_count], dtype=np.float64) / n ** 2
            z = 2.0 * float(d_losses[1]) / n * logsumexp(l[t:t + 1])[0] * soft[t]
            if scoring == "sigmoid":
                tot = s[t].sum() if s[t].sum() > 0 else 1.0
                term = s[t] * rest[t] * (c - (c * s[t]).sum() / tot) / tot
                mag = s[t] * rest[t] * (abs(c) + (abs(c) * s[t]).sum() / tot) / tot
            else:
                term = s[t] * (c - (c * s[t]).sum())
                mag = s[t] * (abs(c) + (abs(c) * s[t]).sum())
            grad[t] += term + z
            size[t] += mag + abs(z)
    return grad, size
