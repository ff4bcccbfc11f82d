"""Drives the chunk calls of the paged cache beside the CPU oracle, with an fp64
reference of the attention and an error bound per output that follows the inputs.

The bound, from the kernel's arithmetic:

  keys     dequantized ones are rounded to fp16, half a step of 2^-10: each channel is off by
           2^-11 of itself (2^-25 below 2^-14); fp16 rows are exact.  A number beyond fp16's
           range is taken as 65504: it is at most z + 2 * 65504 (1 + 2^-11) with z >= -65504, so
           65568, off by 64: 2^-10 of itself (deq_step).
  logits   products of fp16 numbers are exact, the sum over D channels in D / 16 tensor-core
           steps of fp32 sums, which may be cut (2^-23 of the largest partial sum each) after
           alignment of 17 terms: below 2^-18 of A = scale sum |q_c k_c|.  The softmax works on
           x log2(e) - ref in fp32: 2^-22 (|x| + |ref|).  Capped: cap tanh(x / cap) as
           cap (1 - 2 / (e + 1)) is off by 2^-20 cap (the exponential and the division to 2^-21
           each, of numbers up to 1); its slope is at most 1.  A bias: 2^-22 of itself.
  weights  2^y to 2^-21; rounded to fp16 for the product with the values (2^-11) but not in the
           sum that they are divided by; a weight below fp16's range is off by 2^-25 where the
           largest one is held as 2^4 at least: 2^-29 of it.  A reference raised within a tile
           scales its first half's weights, by f = 2^-1 at most and rounded again: 2^-25 (1 + f +
           f / 2^-15) where f < 2^-15 is made of two factors, else 2^-25 (1 + f): below 2^-28 in all.
  values   dequantized ones rounded to fp16 (2^-11, 2^-25 below 2^-14).
  sums     n tokens in n / 16 steps cut to 2^-23, over two halves of a tile, parts and tiles:
           (64 + n / 16) 2^-23 of sum w |v|.
  output   one rounding to fp16: 2^-11 of it, 2^-25 below 2^-14.

An error d of a token's logit moves the output by w (exp(d) - 1) (v - o).
"""
from __future__ import annotations

import math

import numpy as np
import torch

from bit_kivi_kv_gb300 import kivi as K
from bit_kivi_kv_gb300.synth import RANGE_2_6_X10_50, SynthKV
from guards import Banded, GuardedPagedCache
from oracle import layout
from oracle.cache import OracleCache


def chunk_quant(oc, n):
    """Quantized tokens of an oracle cache when n more are appended as a chunk."""
    total = oc.n_quant + oc.n_resid + n
    return max(oc.n_quant, oc.G * ((max(total - oc.R, 0) + oc.G - 1) // oc.G))


def oracle_chunk(oc, k, v):
    """Append k, v [H][n][D] (numpy fp16) to an oracle cache as kivi_paged_append_chunk does."""
    kr = np.concatenate([oc.k_res, k[None]], axis=2)
    vr = np.concatenate([oc.v_res, v[None]], axis=2)
    fresh = chunk_quant(oc, k.shape[1]) - oc.n_quant
    if fresh:
        oc._quantize_into(kr[:, :, :fresh], vr[:, :, :fresh])
    oc.k_res, oc.v_res = kr[:, :, fresh:].copy(), vr[:, :, fresh:].copy()


def oracle_copy(oc):
    new = OracleCache(oc.B, oc.H, oc.d, oc.bits, oc.G, oc.R)
    for name in ("k_codes", "k_s", "k_z", "v_codes", "v_s", "v_z", "k_res", "v_res"):
        setattr(new, name, getattr(oc, name).copy())
    return new


def oracle_truncate(oc, n):
    """Keep the first n tokens."""
    if n < oc.n_quant:
        assert n % oc.G == 0
        for name in ("k_codes", "v_codes", "v_s", "v_z"):
            setattr(oc, name, getattr(oc, name)[:, :, :n])
        oc.k_s, oc.k_z = oc.k_s[:, :, :n // oc.G], oc.k_z[:, :, :n // oc.G]
    oc.k_res, oc.v_res = (x[:, :, :max(0, n - oc.n_quant)] for x in (oc.k_res, oc.v_res))


def ref_attend(keys, vals, n_quant, q, past, scale=None, cap=0.0, window=0, slope=0.0, deq_step=2.0 ** -11):
    """(out, bound) [n][D] of one query head: q [n][D] (fp64) at positions past .. past + n - 1 over keys and
    vals [past + n][D] (fp64, exact), the first n_quant of them dequantized."""
    n, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    at = torch.arange(past, past + n, device=q.device)[:, None]
    t = torch.arange(past + n, device=q.device)
    raw = scale * (q @ keys.T)
    x = cap * torch.tanh(raw / cap) if cap else raw
    bias = slope * (t - at)
    x = x + bias
    hidden = t > at
    if window:
        hidden = hidden | (t <= at - window)
    x = x.masked_fill(hidden, -math.inf)
    top = x.amax(1, keepdim=True)
    w = torch.softmax(x, dim=1)
    o = w @ vals
    deq = (t < n_quant).double()
    a = scale * (q.abs() @ keys.abs().T)
    d = a * (deq_step * deq + 2.0 ** -18) + scale * q.abs().sum(1, keepdim=True) * 2.0 ** -25 * deq
    size = x.masked_fill(hidden, 0.0).abs()
    d = d + 2.0 ** -22 * (size + top.abs() + bias.abs()) + 2.0 ** -20 * cap + 2.0 ** -21
    move = w * (torch.expm1(d) + 2.0 ** -11) + 2.0 ** -28 * (~hidden) / torch.exp(x - top).sum(1, keepdim=True)
    av = vals.abs()
    verr = (deq_step * av + 2.0 ** -25) * deq[:, None]
    bound = (move @ av + o.abs() * (w * torch.expm1(d)).sum(1, keepdim=True) + w @ verr
             + (64 + (past + n) / 16) * 2.0 ** -23 * (w @ av) + 2.0 ** -11 * o.abs() + 2.0 ** -25)
    return o, bound


def head_strided(x):
    """The same [T][H][D] values in head-major memory, as norm and rotation leave them."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def in_wider(x):
    """The same values as a part of a wider row (a packed projection)."""
    T, H, D = x.shape
    wide = torch.full((T, H + 3, D + 8), 1e4, dtype=x.dtype, device=x.device)
    wide[:, 1:H + 1, 8:] = x
    return wide[:, 1:H + 1, 8:]


class ChunkRun:
    def __init__(self, Hq, Hkv, D, bits, G, R, max_seqs=8, max_blocks=64, n_pages=256, seed=1, sink=True):
        self.Hq, self.Hkv, self.D, self.bits, self.G, self.R = Hq, Hkv, D, bits, G, R
        self.max_blocks, self.seed, self.sink = max_blocks, seed, sink
        self.cache = GuardedPagedCache(max_seqs, Hq, Hkv, D, bits, G, R, max_blocks, n_pages)
        self.live, self.made = {}, 0
        self.worst = 0.0

    # -- tokens ---------------------------------------------------------------------
    def draw(self, n, syn=None):
        """(K, V [Hkv][n][D], q [n][Hq][D]) on the GPU."""
        syn = syn or self._syn()
        Kp, Vp = syn.prompt(n)
        g = torch.Generator(device="cuda").manual_seed(self.seed * 31 + self.made)
        self.made += 1
        q = torch.randn(n, self.Hq, self.D, generator=g, device="cuda")
        return Kp[0].contiguous(), Vp[0].contiguous(), (1.5 * q).half()

    def _syn(self):
        self.made += 1
        return SynthKV(1, self.Hq, self.Hkv, self.D, self.seed * 7919 + self.made, outliers=RANGE_2_6_X10_50,
                       sink=self.sink, device="cuda")

    def add(self, L, kv=None):
        Kp, Vp = kv or self.draw(L)[:2]
        s = self.cache.add(Kp, Vp)
        oc = OracleCache(1, self.Hkv, self.D, self.bits, self.G, self.R)
        oc.prefill(Kp.cpu().numpy()[None], Vp.cpu().numpy()[None])
        assert s not in self.live
        self.live[s] = oc
        return s

    def chunk(self, lens):
        """Packed new tokens: q [T][Hq][D], k, v [T][Hkv][D]."""
        parts = [self.draw(n) for n in lens]
        if not parts:
            parts = [self.draw(0)]
        k = torch.cat([p[0].transpose(0, 1) for p in parts]).contiguous()
        v = torch.cat([p[1].transpose(0, 1) for p in parts]).contiguous()
        return torch.cat([p[2] for p in parts]).contiguous(), k, v

    # -- calls ----------------------------------------------------------------------
    def attend(self, seqs, lens, data=None, scale=0.0, cap=0.0, window=0, slopes=None, check=True, fit=lambda x: x, **bound):
        q, k, v = data or self.chunk(lens)
        qs, ks, vs = fit(q), fit(k), fit(v)
        bands = Banded()
        out = bands.like(q)
        out.fill_(float("nan"))
        ws = bands.bytes(K.kivi_paged_chunk_workspace_bytes(self.cache.cfg, lens), "cuda")
        a = K.kivi_chunk()
        for name, t in (("q", qs), ("k", ks), ("v", vs), ("out", out)):
            setattr(a, name, t.data_ptr())
            getattr(a, name + "_stride")[:] = (t.stride(0), t.stride(1))
        a.softmax_scale, a.cap, a.window = scale, cap, window
        a.slopes = slopes.data_ptr() if slopes is not None else None
        before = self.cache.buffer.clone()
        K.kivi_paged_chunk_attn(self.cache.handle, seqs, lens, a, ws.data_ptr(), ws.numel(),
                                torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        bands.check(f"after attention of {list(lens)} over {list(seqs)}")
        self.cache.bands.check("after attention")
        assert torch.equal(before, self.cache.buffer), "attention changed the cache"
        if check:
            self.check_out(seqs, lens, q, k, v, out, scale, cap, window, slopes, **bound)
        return out

    def check_out(self, seqs, lens, q, k, v, out, scale=0.0, cap=0.0, window=0, slopes=None, **bound):
        first, rep = 0, self.Hq // self.Hkv
        for s, n in zip(seqs, lens):
            oc = self.live[s]
            past = oc.n_quant + oc.n_resid
            part = slice(first, first + n)
            kc = torch.from_numpy(oc.keys_hat()[0]).cuda()
            vc = torch.from_numpy(oc.values_hat()[0]).cuda()
            for h in range(self.Hq if n else 0):
                keys = torch.cat([kc[h // rep], k[part, h // rep].double()])
                vals = torch.cat([vc[h // rep], v[part, h // rep].double()])
                ref, most = ref_attend(keys, vals, oc.n_quant, q[part, h].double(), past, scale or None, cap, window,
                                        float(slopes[h]) if slopes is not None else 0.0, **bound)
                got = out[part, h].double()
                what = f"sequence {s} ({past} + {n} tokens) head {h}"
                assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values not finite"
                over = ((got - ref).abs() / most).max().item()
                self.worst = max(self.worst, over)
                assert over <= 1.0, f"{what}: {over:.2f} of the bound, off by {(got - ref).abs().max().item():.3e}"
            first += n

    def append(self, seqs, lens, data=None, fit=lambda x: x):
        q, k, v = data or self.chunk(lens)
        ks, vs = fit(k), fit(v)
        K.kivi_paged_append_chunk(self.cache.handle, seqs, lens, ks.data_ptr(), ks.stride()[:2], vs.data_ptr(),
                                  vs.stride()[:2], torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        self.cache.bands.check(f"after appending {list(lens)} to {list(seqs)}")
        first = 0
        for s, n in zip(seqs, lens):
            oracle_chunk(self.live[s], k[first:first + n].transpose(0, 1).cpu().numpy(),
                         v[first:first + n].transpose(0, 1).cpu().numpy())
            first += n

    def fork(self, seqs):
        new = self.cache.fork(seqs)
        for s, t in zip(seqs, new):
            assert t not in self.live
            self.live[t] = oracle_copy(self.live[s])
        return new

    def truncate(self, s, n):
        self.cache.truncate(s, n)
        oracle_truncate(self.live[s], n)

    def release(self, s):
        self.cache.release(s)
        del self.live[s]

    # -- the cache's bytes against the oracle's --------------------------------------------
    def check(self, only=None):
        torch.cuda.synchronize()
        lay, buf = self.cache.layout, self.cache.buffer.cpu().numpy()
        D, G, R, bits = self.D, self.G, self.R, self.bits
        for s in self.live if only is None else only:
            oc = self.live[s]
            assert self.cache.counts(s) == (oc.n_quant, oc.n_resid), (s, self.cache.counts(s), oc.n_quant, oc.n_resid)
            pages = self.cache.pages(s)
            assert len(pages) * G == oc.n_quant
            table = buf[lay.table_offset + s * self.max_blocks * 4:][: len(pages) * 4].view(np.int32)
            assert table.tolist() == pages, f"block table row of sequence {s}"
            for h in range(self.Hkv):
                if pages:
                    part = lambda j: np.stack([buf[((p * self.Hkv + h) * 2 + j) * lay.part_bytes:][: lay.part_bytes]  # noqa: E731
                                               for p in pages])
                    ek = layout.pack_key_parts(oc.k_codes[0, h], oc.k_s[0, h], oc.k_z[0, h], bits, G)
                    ev = layout.pack_value_parts(oc.v_codes[0, h], oc.v_s[0, h], oc.v_z[0, h], bits, G)
                    assert np.array_equal(part(0), ek), f"key blocks of sequence {s} head {h}"
                    assert np.array_equal(part(1), ev), f"value blocks of sequence {s} head {h}"
                rows, n = (s * self.Hkv + h) * R * D * 2, oc.n_resid * D * 2
                assert buf[lay.k_resid_offset + rows:][:n].tobytes() == oc.k_res[0, h].tobytes(), f"keys of {s}, head {h}"
                assert buf[lay.v_resid_offset + rows:][:n].tobytes() == oc.v_res[0, h].tobytes(), f"values of {s}, head {h}"
