"""References and error bounds of the calls over chosen blocks, in fp64.

The bounds are derived from the arithmetic, not fitted:

  scores   a coefficient (scale * q, or scale * q * L) is rounded at most twice,
           then 8 products are summed by fused multiply-adds and the lanes' sums
           in 5 additions: each term meets fewer than 16 roundings of 2^-24.
  decode   a logit sums at most 256 products with fp16 hi + lo parts of the
           query (2^-22 each) through 16 tensor-core steps, whose fp32 sums may
           be cut instead of rounded (2^-23 of the running sum each): within
           16 * 2^-23 + 2^-21 < 2^-18 of A = scale * sum_c |q_c| (|k_hat_c| + |z_c|).
           A probability is then off by a factor exp(delta) with delta = 2^-18 A
           plus the exponential's own 2^-21; numerator and denominator both
           carry it, so the output moves by at most 2 delta max|v|.  The value
           sums round like the logits' (2^-18 of max|v| + max|z|), and the
           result once to fp16 (half a step: 2^-11 of it, 2^-25 below 2^-14).
"""
from __future__ import annotations

import math

import numpy as np

from oracle.attention import decode_attention


def block_tokens(blocks, G):
    """Token indices of the listed blocks (negative entries skipped)."""
    return np.concatenate([np.arange(b * G, (b + 1) * G) for b in blocks if b >= 0] or [np.zeros(0, np.int64)])


def ref_scores(oc, q, bits, scale=None):
    """(scores [blocks], bound [blocks]) of one oracle slot for its group's queries q [nq][D]."""
    s, z = oc.k_s[0, 0].astype(np.float64), oc.k_z[0, 0].astype(np.float64)      # [blocks][D]
    q = q.astype(np.float64)[:, None]
    L = 2 ** bits - 1
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    u = scale * (q * z + L * np.maximum(q, 0) * s).sum(-1)
    size = scale * (np.abs(q * z) + L * np.maximum(q, 0) * s).sum(-1)
    return u.max(0), 16 * 2.0 ** -24 * size.max(0)


def ref_decode(oc, q, blocks, G, scale=None):
    """(out [nq][D], bound [nq][D]) of attention of q [nq][D] over the listed
    blocks (with repeats) and the residual of one oracle slot."""
    K, V = oc.keys_hat()[0, 0], oc.values_hat()[0, 0]
    at = np.concatenate([block_tokens(blocks, G), np.arange(oc.n_quant, K.shape[0])])
    K, V = K[at], V[at]
    o, _ = decode_attention(q[None], K[None, None], V[None, None], scale)
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    zk = np.abs(oc.k_z[0, 0].astype(np.float64)).max(0) if oc.n_quant else 0.0
    zv = float(np.abs(oc.v_z[0, 0].astype(np.float64)).max()) if oc.n_quant else 0.0
    A = scale * (np.abs(q.astype(np.float64)) @ (np.abs(K).max(0) + zk))            # [nq]
    vmax = float(np.abs(V).max())
    delta = 2.0 ** -18 * A + 2.0 ** -20
    bound = 2.0 ** -11 * np.abs(o[0]) + 2.0 ** -25 + 2 * delta[:, None] * vmax + 2.0 ** -18 * (vmax + zv)
    return o[0], bound


def ref_select(scores, n_keep, keep_first):
    """The selection of kivi_select_blocks for scores [rows][cols], int32 [rows][n_keep]."""
    out = np.full((scores.shape[0], n_keep), -1, np.int32)
    for r, row in enumerate(np.asarray(scores, np.float64)):
        n = np.arange(row.size)
        ok = row > -np.inf
        first = (n < keep_first) & ok
        key = np.where(ok, row, -np.inf)
        order = np.lexsort((n, -key, ~first))          # the kept ones, then by score, then by index
        # among the always-kept columns the index decides
        head = n[first]
        rest = [c for c in order if ok[c] and not first[c]]
        pick = np.sort(np.concatenate([head, rest])[:n_keep].astype(np.int64))
        out[r, :pick.size] = pick
    return out


def assert_within(got, ref, bound, what=""):
    got = np.asarray(got, np.float64)
    over = np.abs(got - ref) - bound
    assert not np.isnan(got).any(), f"{what}: NaN"
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - ref).max():.3e}, bound {bound.ravel()[over.argmax()]:.3e}"
