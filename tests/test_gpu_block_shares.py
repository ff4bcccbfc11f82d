"""Which blocks a decode over lists reads: inputs where every pair of tiles moves the output by more
than the error bound, so that one that is lost, read twice or taken for another one shows.

Keys are constant in a block (exact when quantized) and give it a weight of its own between 1 and e;
values are +-1 at random for every 32 tokens and channel (exact too, the ends of their groups).  Each test
checks, for every listed pair, that without it the reference moves by more than twice the bound."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from decode_bounds import Slot, close  # noqa: E402
from guards import GuardedCache, GuardedPagedCache  # noqa: E402
from oracle.cache import OracleCache  # noqa: E402


def prompt(rows, D, G, R, L, seed):
    """k, v [rows][L][D] fp16 and the queries' direction u [rows][D] (one channel each)."""
    g = np.random.default_rng(seed)
    at = g.integers(0, D, rows)
    u = np.zeros((rows, D))
    u[np.arange(rows), at] = np.sqrt(D)
    k = np.zeros((rows, L, D))
    for r in range(rows):
        k[r, :, at[r]] = np.repeat(g.uniform(0, 1, L // G + 1), G)[:L]
    v = np.repeat(g.choice([-1.0, 1.0], (rows, L // 32 + 1, D)), 32, axis=1)[:, :L]
    return k.astype(np.float16), v.astype(np.float16), u


def check_row(got, oc, bits, q, blocks, what, warps):
    slot = Slot(oc, bits)
    at, scale = slot.tokens([int(b) for b in blocks]), q.shape[-1] ** -0.5
    ref, bound = slot.decode(q, at, scale, warps)
    s = scale * (q.astype(np.float64) @ slot.K[at].T)
    w = np.exp(s)
    listed = int((at < oc.n_quant).sum())
    w = w[:, :listed].reshape(len(q), -1, 32).sum(-1), w.sum(1)[:, None]          # of a pair; in all
    o = slot.V[at][:listed:32]                                                   # a pair's values [pairs][D]
    moved = np.abs(ref[:, None] - o[None]) * (w[0] / (w[1] - w[0]))[..., None]       # [nq][pairs][D]
    assert (moved > 2 * bound[:, None]).any(-1).all(), f"{what}: a pair that could be lost unseen"
    close(got, ref, bound, what)


def queries(u, B, Hkv, nq, seed):
    """Multiples of u: a query head's logits are the keys times a factor between 1/2 and 1."""
    g = np.random.default_rng(seed + 7)
    q = np.repeat(u.reshape(B, Hkv, 1, -1), nq, axis=2) * g.uniform(0.5, 1, (B, Hkv, nq, 1))
    return q.astype(np.float16).reshape(B, Hkv * nq, -1)


def some_rows(B, Hkv, seed):
    rng = random.Random(seed)
    return sorted({(0, 0), (B - 1, Hkv - 1)} | {(rng.randrange(B), rng.randrange(Hkv)) for _ in range(4)})


@pytest.mark.parametrize("B,Hkv,nq,D,bits,G,L,keep", [
    (1, 1, 1, 64, 2, 32, 33000, None), (1, 1, 4, 128, 4, 128, 40000, None), (5, 3, 1, 128, 8, 64, 3500, None),
    (1, 1, 1, 128, 2, 32, 9000, 270), (1, 3, 2, 64, 4, 64, 1200, 9), (1, 8, 1, 128, 2, 32, 4000, 100),
    (2, 32, 1, 128, 2, 32, 1500, 40), (8, 19, 1, 128, 2, 32, 700, 12), (9, 17, 4, 128, 4, 64, 700, 5),
    (16, 19, 1, 128, 8, 32, 600, 12), (38, 16, 2, 64, 2, 32, 400, 6), (61, 25, 1, 64, 2, 32, 300, 4),
    (2, 2, 1, 128, 4, 128, 1300, 7)])
def test_no_pair_is_lost(B, Hkv, nq, D, bits, G, L, keep):
    R = max(G, 64)
    k, v, u = prompt(B * Hkv, D, G, R, L, B + Hkv + L)
    q = queries(u, B, Hkv, nq, L)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cache = GuardedCache(B, Hkv * nq, Hkv, D, bits, G, R, L + 1)
    cache.prefill(dev(k.reshape(B, Hkv, L, D)), dev(v.reshape(B, Hkv, L, D)))
    nb = cache.counts()[0] // G
    rng = random.Random(L)
    n = nb if keep is None else keep
    for holes in (False, True):
        blocks = np.stack([rng.sample(range(nb), n) for _ in range(B * Hkv)]).astype(np.int32).reshape(B, Hkv, n)
        if holes:
            blocks[np.random.default_rng(n).random(blocks.shape) < 0.2] = -1
        qt = dev(q)
        got = cache.decode_blocks(qt, dev(blocks), out=cache.bands.like(qt))
        cache.bands.check("after a decode over blocks")
        got = got.cpu().numpy()
        for b, h in some_rows(B, Hkv, L):
            oc = OracleCache(1, 1, D, bits, G, R)
            oc.prefill(k[b * Hkv + h][None, None], v[b * Hkv + h][None, None])
            check_row(got[b, h * nq:(h + 1) * nq], oc, bits, q[b, h * nq:(h + 1) * nq], blocks[b, h], f"row {(b, h)}",
                      8 if B * Hkv <= 16 else 1)


@pytest.mark.parametrize("Hkv,nq,D,bits,G,n", [(4, 1, 128, 2, 32, 40), (2, 4, 128, 4, 128, 6), (32, 1, 64, 8, 64, 200)])
def test_no_pair_is_lost_in_pages(Hkv, nq, D, bits, G, n):
    """Ragged sequences, lists longer than the shorter ones' blocks, blocks anywhere in them."""
    R = max(G, 64)
    lengths = [23 * G + 5, 3 * G + R, R + 1, 41 * G, 9 * G + 17]
    most = max(lengths) // G + 2
    cache = GuardedPagedCache(len(lengths), Hkv * nq, Hkv, D, bits, G, R, most, len(lengths) * most)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    data = [prompt(Hkv, D, G, R, L, 100 + L) for L in lengths]
    seqs = [cache.add(dev(k), dev(v)) for k, v, _ in data]
    q = np.concatenate([queries(u, 1, Hkv, nq, 5 + i) for i, (_, _, u) in enumerate(data)])
    rng = random.Random(n)
    blocks = np.full((len(lengths), Hkv, n), -1, np.int32)
    for i, s in enumerate(seqs):
        nb = cache.counts(s)[0] // G
        for h in range(Hkv):
            m = min(nb, n)
            blocks[i, h, sorted(rng.sample(range(n), m))] = rng.sample(range(nb), m)
    qt = dev(q)
    got = cache.decode_blocks(seqs, qt, dev(blocks), out=cache.bands.like(qt))
    cache.bands.check("after a paged decode over blocks")
    got = got.cpu().numpy()
    for i in range(len(lengths)):
        for h in sorted({0, Hkv // 2, Hkv - 1}):
            oc = OracleCache(1, 1, D, bits, G, R)
            oc.prefill(data[i][0][h][None, None], data[i][1][h][None, None])
            check_row(got[i, h * nq:(h + 1) * nq], oc, bits, q[i, h * nq:(h + 1) * nq], blocks[i, h], f"sequence {i}, head {h}", 1)
