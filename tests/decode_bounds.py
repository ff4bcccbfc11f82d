"""fp64 reference of a decode over one cache slot, with an error bound per output
that follows the inputs' scales: every term is relative to a value of the call itself.

From the tensor-core kernels' arithmetic (a rounding to fp32: 2^-24 of the value; to fp16: 11
significant bits, and a last bit worth 2^-24 at least):

  query    x = scale log2(e) q is held times a power of two that puts the head's largest
           |x| into [2^8, 2^9), as fp16 hi + lo parts: each channel is off by at most
           2^-22 of itself, or by half of the last bit.  The parts carry the channel's
           code scale (2^-6 at least), so that half is worth 2^-25 2^6 2^-8 = 2^-27 of
           the head's largest |x|.
  keys     steps times 2^-f, f from the largest step S of the warp's blocks so far: 2^f
           <= max(S / 16, 2^-15).  A product x step is h + l per unit of code, h a multiple
           of 1, 2 or its own last bit, l what is left (at most 1, or 2^-11 of the product),
           off by 2^-11 of that size: per unit of code 2^-11 (times code scale in both)
           where 1 is worth `one` = max|x| 2^-8 2^f; beside 2^-22 of the product.
  MMAs     the codes are fp16 subnormals, which the tensor cores multiply without
           normalizing them: of a step's 16 products and its running sum, bits below
           2^-15 of the largest factor per unit of code are cut (measured with single
           products).  The h have no such bits; the l are at most 2^-12 of the
           largest product of 2^15, 8: 17 2^-12 a step.  fp16 rows: 17 2^-25 of the
           largest product, of numbers below 2^-14 as if they were that.
  logits   16 steps' fp32 sums, cut as well (2^-23 of the running sum), the zero
           points' sum, times the unit: with the 2^-21 above less than 2^-18 of
           A = scale sum_c |q_c| (|k_c| + |z_c|).
  softmax  2^x is good to 2^-21; a probability is held as p 2^k in hi + lo parts:
           2^-22, or half of the last bit: 2^-25 2^-k of the largest one, where 2^-k
           <= max(2^-15, 2^-13 S) for the largest value step S.
  values   p 2^k step as h + l again, h a multiple of 2^-15 of the largest p 2^k step
           allowed, top = max(4 S, 2^-13) of the largest p, or of its own last bit: l is off by 2^-11 of its
           size, so a product per unit of code by 2^-27 top or 2^-11 of itself, whichever
           is less, and 2^-22 of itself.  The MMAs cut 17 2^-27 top a tile off the l.
  sums     n tokens in n / 16 steps, shared by `warps` warps at least, and the merge:
           (32 + n / 16 / warps) 2^-23 of sum w (|v| + |z|).
  output   one rounding to fp16: 2^-11 of it, 2^-25 below 2^-14.

An error d of a token's logit moves the output by w (exp(d) - 1) (v - o).
"""
from __future__ import annotations

import numpy as np

from blocks_harness import block_tokens


class Slot:
    """What a decode of one oracle slot reads, in fp64."""

    def __init__(self, oc, bits):
        G, n = oc.G, oc.n_quant
        self.G, self.n_quant, self.bits = G, n, bits
        self.K, self.V = oc.keys_hat()[0, 0], oc.values_hat()[0, 0]
        D = self.K.shape[1]
        rows = lambda x, times, axis: np.repeat(x.astype(np.float64), times, axis=axis).reshape(-1, D)  # noqa: E731
        # (fp16 rows have neither; with the value queue values are quantized later than keys)
        fill = lambda x: np.concatenate([x, np.zeros((self.K.shape[0] - len(x), D))])  # noqa: E731
        self.zk, self.sk = (fill(rows(x[0, 0], G, 0)) for x in (oc.k_z, oc.k_s))
        self.zv, self.sv = (fill(rows(x[0, 0], G, 1)) for x in (oc.v_z, oc.v_s))

    def tokens(self, blocks=None):
        """Token indices of the listed blocks (None: all) and the residual."""
        if blocks is None:
            return np.arange(self.K.shape[0])
        return np.concatenate([block_tokens(blocks, self.G), np.arange(self.n_quant, self.K.shape[0])])

    def decode(self, q, at, scale, warps=1):
        """(out, bound), both [nq][D], of attention of q [nq][D] over tokens at (of self.tokens)."""
        q, bits = np.asarray(q, np.float64), self.bits
        K, V, zk, sk, zv, sv = (t[at] for t in (self.K, self.V, self.zk, self.sk, self.zv, self.sv))
        (n, D), nq = K.shape, len(q)
        listed = int((at < self.n_quant).sum())
        L = 2.0 ** bits - 1
        s = scale * (q @ K.T)                                                    # [nq][n]
        e = np.exp(s - s.max(1, keepdims=True))
        w = e / e.sum(1, keepdims=True)
        o = w @ V
        x = scale * np.abs(q)
        xmax = x.max(1)[:, None]
        # logits
        one = xmax * 2.0 ** -8 * max(sk.max(initial=0.0) / 16, 2.0 ** -15)
        d = 2.0 ** -18 * (x @ (np.abs(K) + np.abs(zk)).T) + 2.0 ** -20
        d[:, :listed] += xmax * 2.0 ** -27 * L * sk[:listed].sum(1) + one * (D * L * 2.0 ** -11 + D / 16 * 17 * 2.0 ** -12)
        rows = np.maximum(np.abs(K[listed:]), 2.0 ** -14)
        d[:, listed:] += D / 16 * 17 * 2.0 ** -24 * (x[:, None] * rows).max(-1)
        moved = np.einsum("hn,hnd->hd", w * np.expm1(d), np.abs(V[None] - o[:, None]))
        # values; those of the listed tokens that are still fp16 (a value queue) have step 0
        wmax, S = w.max(1)[:, None], sv.max(initial=0.0)
        top = wmax * max(4 * S, 2.0 ** -13)
        ws = w[:, :, None] * sv                                                  # [nq][n][D]
        lost = L * (np.minimum(2.0 ** -27 * top[..., None], 2.0 ** -11 * ws) + 2.0 ** -22 * ws).sum(1)
        lost += n * (2.0 ** -25 * wmax * max(2.0 ** -15, 2.0 ** -13 * S) * L * S + 17 / 16 * 2.0 ** -27 * top)
        tail = np.maximum(np.abs(V), 2.0 ** -14) * (sv == 0)
        lost += 17 * 2.0 ** -24 * (w @ tail) + n * 2.0 ** -25 * wmax * max(2.0 ** -15, 2.0 ** -13 * S) * tail.max(0)
        sums = (32 + n / 16 / warps) * 2.0 ** -23 * (w @ (np.abs(V) + np.abs(zv)))
        return o, 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + 1.01 * moved + lost + sums


def close(got, ref, bound, what=""):
    got = np.asarray(got, np.float64)
    assert not np.isnan(got).any(), f"{what}: NaN"
    over = np.abs(got - ref) / bound
    i = np.unravel_index(over.argmax(), over.shape)
    assert over[i] <= 1, f"{what}: off by {abs(got[i] - ref[i]):.3e} at {i}, bound {bound[i]:.3e}, value {ref[i]:.3e}"
    return over[i]
