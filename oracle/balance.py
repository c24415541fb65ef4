"""Balance and z losses of a softmax top-k router (test infrastructure only).

Sequence b holds the tokens [offs[b], offs[b+1]) whose mask is set and that have
a logit above -inf; with p_t = softmax(l_t), n the sequence's counted tokens and
c_e the ids e among theirs:
    probs_e = sum_t p_te / n,   loss = E / (k n) sum_e c_e probs_e,
    z = sum_t logsumexp(l_t)^2 / n;  0 where n = 0.
The gradient takes c for a constant; with f_e = E c_e / (k n):
    d l_te = p_te (d_loss / n (f_e - sum_i p_ti f_i) + 2 d_z / n logsumexp(l_t)).

Pins (tests/test_oracle_balance.py): even and one-expert routing in closed form,
a hand-written example, differences of the loss with c held.
"""
from __future__ import annotations

import numpy as np


def softmax(logits):
    """float64 probabilities, logsumexp, and whether some logit is above -inf."""
    l = np.asarray(logits, np.float64)
    live = ~(l == -np.inf).all(axis=1)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        top = np.where(live, l.max(axis=1, initial=-np.inf), 0.0)[:, None]
        ex = np.exp(l - top)
        total = ex.sum(axis=1, keepdims=True)
        return ex / np.where(total == 0, 1.0, total), (top + np.log(total))[:, 0], live


def members(n, offs, mask, live):
    """The counted tokens of each sequence."""
    offs = [0, n] if offs is None else [int(v) for v in offs]
    keep = live if mask is None else live & np.asarray(mask, bool)
    return [np.nonzero(keep[lo:hi])[0] + lo for lo, hi in zip(offs[:-1], offs[1:])]


def balance(logits, idx, offs=None, mask=None):
    """-> dict of loss, z_loss, counts, probs, tokens (float64, int64)."""
    logits, idx = np.asarray(logits), np.asarray(idx)
    n, e = logits.shape
    k = idx.shape[1]
    p, lse, live = softmax(logits)
    seqs = members(n, offs, mask, live)
    b = len(seqs)
    out = dict(loss=np.zeros(b), z_loss=np.zeros(b), counts=np.zeros((b, e), np.int64),
               probs=np.zeros((b, e)), tokens=np.array([t.size for t in seqs]))
    for i, t in enumerate(seqs):
        if not t.size:
            continue
        ids = idx[t].reshape(-1)
        out["counts"][i] = np.bincount(ids[(ids >= 0) & (ids < e)], minlength=e)
        out["probs"][i] = p[t].sum(0) / t.size
        out["loss"][i] = e / (k * t.size) * (out["counts"][i] * out["probs"][i]).sum()
        out["z_loss"][i] = (lse[t] ** 2).sum() / t.size
    return out


def balance_backward(logits, counts, tokens, k, d_loss, d_z, offs=None, mask=None):
    logits = np.asarray(logits)
    n, e = logits.shape
    p, lse, live = softmax(logits)
    grad = np.zeros((n, e))
    for i, t in enumerate(members(n, offs, mask, live)):
        m = int(tokens[i])
        if not t.size or m < 1:
            continue
        f = np.asarray(counts[i], np.float64) * e / (k * m)
        q = p[t]
        inner = f - (q * f).sum(1, keepdims=True)
        grad[t] = q * (d_loss[i] / m * inner + (2.0 * d_z[i] / m * lse[t])[:, None])
    return grad
