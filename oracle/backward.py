"""Gradients of the token path (test infrastructure only).

Each function is the derivative of a forward oracle, written as the formula in
float64:

* combine, out[t] = sum_j w[t, j] y[dst_pos[t*k + j]]:
      d_y[p] = w[t, j] d_out[t] for the pair whose row is p,
      d_w[t, j] = <d_out[t], y[p]>;
* dispatch, rows[dst_pos[t*k + j]] = x[t]:  d_x[t] = sum_j d_rows[dst_pos[t*k + j]];
* routing weights, w = softmax over the selected logits (renormalize) or the
  selected entries of the full softmax p, with S = sum_j w_j d_j:
      renormalize: d_l[idx_j] = w_j (d_j - S), else 0;
      otherwise:   d_l[e] = sum_{j: idx_j = e} w_j d_j - p_e S.

Positions outside [0, NK) and ids outside [0, E) hold no pair.

Pins (tests/test_oracle_backward.py): central differences of the forward
oracles (combine_f64, dispatch, route_topk_brute's softmax); the gradient of a
constant shift of the logits is zero; a dispatch whose rows are summed back.
"""
from __future__ import annotations

import numpy as np


def combine_backward(d_out, y, dst_pos, w, k):
    """-> (d_y float64 [NK, D], zero where no pair names the row; d_w float64
    [N, k]; |d_w| magnitude float64 [N, k], the sum of its terms' absolute values)."""
    d_out = np.asarray(d_out, np.float64)
    y = np.asarray(y, np.float64)
    w = np.asarray(w, np.float64).reshape(-1, k)
    pos = np.asarray(dst_pos, np.int64).reshape(-1, k)
    nk = pos.size
    d_y = np.zeros((nk, d_out.shape[1]))
    d_w = np.zeros(pos.shape)
    mag = np.zeros(pos.shape)
    for j in range(k):
        t = np.nonzero((pos[:, j] >= 0) & (pos[:, j] < nk))[0]
        p = pos[t, j]
        d_y[p] = w[t, j:j + 1] * d_out[t]
        terms = d_out[t] * y[p]
        d_w[t, j] = terms.sum(1)
        mag[t, j] = np.abs(terms).sum(1)
    return d_y, d_w, mag


def dispatch_backward(d_rows, dst_pos, k):
    """-> (d_x float64 [N, D], sum of the terms' absolute values)."""
    d_rows = np.asarray(d_rows, np.float64)
    pos = np.asarray(dst_pos, np.int64).reshape(-1, k)
    out = np.zeros((pos.shape[0], d_rows.shape[1]))
    mag = np.zeros_like(out)
    for j in range(k):
        t = np.nonzero((pos[:, j] >= 0) & (pos[:, j] < pos.size))[0]
        out[t] += d_rows[pos[t, j]]
        mag[t] += np.abs(d_rows[pos[t, j]])
    return out, mag


def route_backward(topk_idx, w, d_w, n_experts, renormalize=True, logits=None):
    """-> (d_logits float64 [N, E], scale float64 [N, E]: |w_j d_j| of the
    expert's slots plus its probability times sum_j |w_j d_j|, the size of the
    terms that its rounding errors are relative to)."""
    idx = np.asarray(topk_idx, np.int64)
    w = np.asarray(w, np.float64)
    d = np.asarray(d_w, np.float64)
    n, k = idx.shape
    ok = (idx >= 0) & (idx < n_experts)
    wd = np.where(ok, w * d, 0.0)
    s = wd.sum(1, keepdims=True)
    sa = np.abs(wd).sum(1, keepdims=True)
    out = np.zeros((n, n_experts))
    scale = np.zeros((n, n_experts))
    if renormalize:
        p = np.zeros((n, n_experts))
        for j in range(k):
            t = np.nonzero(ok[:, j])[0]
            p[t, idx[t, j]] += w[t, j]
    else:
        l = np.asarray(logits, np.float64)
        with np.errstate(invalid="ignore"):
            p = np.exp(l - l.max(1, keepdims=True))
            p = p / p.sum(1, keepdims=True)
    out -= p * s
    scale += p * sa
    for j in range(k):
        t = np.nonzero(ok[:, j])[0]
        out[t, idx[t, j]] += wd[t, j]
        scale[t, idx[t, j]] += np.abs(wd[t, j])
    return out, scale
