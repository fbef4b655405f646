"""Oracle: the router of the MoE layer, forward and backward in fp64.

The pages do not describe the router; the definition is the library's: the k
largest keys logit + bias (one fp32 addition), ties to the lower expert, keys
of -inf or NaN never chosen; softmax weights over the chosen logits ("topk")
or over all experts ("all")."""

import numpy as np


def select(logits, bias, k):
    """Ids [T, k] int32 (-1 where nothing is left) of fp32 logits."""
    logits = np.asarray(logits, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        key = logits + (np.zeros(logits.shape[1], np.float32) if bias is None else np.asarray(bias, np.float32))
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k].astype(np.int32)
    return np.where(np.take_along_axis(key, ids, 1) > -np.inf, ids, -1)


def _softmax(x, axis=-1):
    """Softmax in fp64; a row of -inf gives zeros."""
    x = np.asarray(x, np.float64)
    m = x.max(axis=axis, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(x - m)
    s = e.sum(axis=axis, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def weights(logits, ids, score, scale):
    l = np.asarray(logits, np.float64)
    got = ids >= 0
    at = np.where(got, ids, 0)
    if score == "topk":
        return scale * np.where(got, _softmax(np.where(got, np.take_along_axis(l, at, 1), -np.inf)), 0.0)
    return scale * np.where(got, np.take_along_axis(_softmax(l), at, 1), 0.0)


def lse(logits):
    l = np.asarray(logits, np.float64)
    m = l.max(axis=1)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(np.isneginf(m), -np.inf, m + np.log(np.exp(l - np.where(np.isneginf(m), 0, m)[:, None]).sum(1)))


def prob_sum(logits):
    return _softmax(logits).sum(axis=0)


def _times(p, x):
    """p x, 0 where p is 0 (a masked expert), whatever x is there."""
    return np.where(p == 0, 0.0, p * np.where(p == 0, 0.0, x))


def backward(logits, ids, score, scale, dw, dlse=None, dsum=None):
    """d logits (fp64) of sum(w dw) + sum(lse dlse) + sum(prob_sum dsum)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    p = _softmax(l)
    d = np.zeros((T, E))
    u = scale * np.asarray(dw, np.float64)
    for t in range(T):
        on = ids[t] >= 0
        e = ids[t][on]
        if score == "topk":
            if e.size:
                q = _softmax(l[t, e])
                np.add.at(d[t], e, q * (u[t, on] - (q * u[t, on]).sum()))
        else:
            np.add.at(d[t], e, p[t, e] * u[t, on])
            d[t] -= p[t] * (p[t, e] * u[t, on]).sum()
    if dlse is not None:
        d += _times(p, np.asarray(dlse, np.float64)[:, None])
    if dsum is not None:
        s = np.asarray(dsum, np.float64)
        d += _times(p, s[None, :] - _times(p, s).sum(axis=1, keepdims=True))
    return d
