"""Decode over chosen blocks on the GPU against the CPU oracle in fp64: block
scores, selection, attention over block lists, on dense and paged caches, alone
and as the steps of a decode."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300 import kivi as K  # noqa: E402
from bit_kivi_kv_gb300.kivi import KiviCache, KiviPagedCache, select_blocks  # noqa: E402
from bit_kivi_kv_gb300.synth import SynthKV  # noqa: E402
from blocks_harness import assert_within, ref_decode, ref_scores, ref_select  # noqa: E402
from guards import Banded, GuardedCache, GuardedPagedCache  # noqa: E402
from oracle.attention import decode_attention  # noqa: E402
from oracle.cache import OracleCache  # noqa: E402


class Lazy(dict):
    """Oracles of the slots asked for."""

    def __init__(self, make):
        self.make = make

    def __missing__(self, key):
        self[key] = self.make(*key)
        return self[key]


def dense(B, Hq, Hkv, D, bits, G, R, L, seed, n_app=0, sink=True):
    """A dense cache of prompt L and n_app appends, the oracle of each slot, and a next query."""
    syn = SynthKV(B, Hq, Hkv, D, seed, sink=sink, device="cuda")
    Kp, Vp = syn.prompt(L)
    cache = GuardedCache(B, Hq, Hkv, D, bits, G, R, max(L + n_app, 1) + 8)
    cache.prefill(Kp, Vp)
    new = [syn.step(s)[1:] for s in range(n_app)]
    for k, v in new:
        cache.append(k, v)

    def oracle(b, h):
        o = OracleCache(1, 1, D, bits, G, R)
        o.prefill(Kp[b, h][None, None].cpu().numpy(), Vp[b, h][None, None].cpu().numpy())
        for k, v in new:
            o.append(k[b, h][None, None].cpu().numpy(), v[b, h][None, None].cpu().numpy())
        return o

    oc = Lazy(oracle)
    if B * Hkv <= 64:
        for b in range(B):
            for h in range(Hkv):
                oc[b, h]
    return cache, oc, syn.step(1000)[0]


def paged(lengths, Hq, Hkv, D, bits, G, R, seed, extra=2):
    """A paged cache of these prompts (pages handed out after a churn, so not in
    order), the oracle of each (sequence, kv head), and one query per sequence."""
    most = max(lengths) // G + extra
    cache = GuardedPagedCache(len(lengths) + 1, Hq, Hkv, D, bits, G, R, most, (len(lengths) + 2) * most)
    syn0 = SynthKV(1, Hq, Hkv, D, seed + 99, device="cuda")
    Kp, Vp = syn0.prompt(max(lengths))
    first = cache.add(Kp[0].contiguous(), Vp[0].contiguous())
    seqs, oc, qs = [], {}, []
    for i, L in enumerate(lengths):
        syn = SynthKV(1, Hq, Hkv, D, seed + i, device="cuda")
        Kp, Vp = syn.prompt(L)
        if i == len(lengths) // 2:
            cache.release(first)
        seqs.append(cache.add(Kp[0].contiguous(), Vp[0].contiguous()))
        for h in range(Hkv):
            oc[i, h] = OracleCache(1, 1, D, bits, G, R)
            oc[i, h].prefill(Kp[:, h:h + 1].cpu().numpy(), Vp[:, h:h + 1].cpu().numpy())
        qs.append(syn.step(1000)[0][0])
    return cache, seqs, oc, torch.stack(qs).contiguous()


def lists(rng, rows, blocks_of, n, holes=True):
    """Random lists of distinct blocks in random order, with -1 among and behind them."""
    out = np.full((rows, n), -1, np.int32)
    for r in range(rows):
        nb = blocks_of(r)
        m = min(n, nb)
        pick = rng.sample(range(nb), m)
        for j in range(m):
            if not (holes and rng.random() < 0.15):
                out[r, j] = pick[j]
    return out


def check_scores(scores, oc, q, bits, Hkv, nq, tight=True):
    scores, q = scores.cpu().numpy(), q.cpu().numpy()
    for (i, h), o in oc.items():
        row = scores[i, h]
        nb = o.n_quant // o.G
        assert np.all(np.isneginf(row[nb:])), (i, h)
        if not nb:
            continue
        ref, bound = ref_scores(o, q[i, h * nq:(h + 1) * nq], bits)
        assert_within(row[:nb], ref, bound, f"scores of row {(i, h)}")
        # a bound on every logit of the block's tokens
        k = o.keys_hat()[0, 0][:o.n_quant]
        x = (q[i, h * nq:(h + 1) * nq].astype(np.float64) @ k.T / np.sqrt(k.shape[1])).max(0).reshape(nb, -1).max(1)
        assert (x <= row[:nb] + bound).all(), (i, h)


def check_decode(out, oc, q, blocks, G, nq, what=""):
    out, q = out.cpu().numpy(), q.cpu().numpy()
    for (i, h), o in oc.items():
        sl = slice(h * nq, (h + 1) * nq)
        ref, bound = ref_decode(o, q[i, sl], [int(x) for x in blocks[i, h]], G)
        assert_within(out[i, sl], ref, bound, f"{what} row {(i, h)}")


COMBOS = [(D, bits, nq, G) for D in (64, 128) for bits in (2, 4, 8) for nq in (1, 2, 4)
          for G in (32, 64, 128) if G <= D]
IDS = [f"D{c[0]}b{c[1]}nq{c[2]}G{c[3]}" for c in COMBOS]


# ---- selection -------------------------------------------------------------------------


@pytest.mark.parametrize("rows,cols,keep,first", [
    (1, 1, 1, 0), (1, 1, 1, 1), (3, 5, 5, 0), (3, 5, 8, 2), (7, 31, 4, 1), (5, 32, 31, 0), (4, 33, 16, 4),
    (256, 124, 32, 1), (64, 257, 100, 3), (9, 1000, 1, 0), (9, 1023, 1023, 0), (3, 4092, 128, 1), (2, 8192, 512, 2),
    (2, 8193, 77, 0), (2, 20011, 3000, 5), (1, 70000, 64, 1), (600, 40, 8, 8), (5, 2000, 300, 300), (3, 9500, 128, 1),
    (2, 12000, 200, 2), (2, 16384, 16384, 0), (3, 32768, 512, 1), (2, 49152, 40, 0), (2, 49153, 40, 1), (40, 700, 130, 129)])
def test_select_against_sort(rows, cols, keep, first):
    """Spread values, many equal values, masked tails, special values, in every row layout."""
    g = np.random.default_rng(rows * 1000003 + cols)
    s = g.normal(5, 3, (rows, cols)).astype(np.float32)
    s[1::3] = np.round(s[1::3])                            # ties
    s[2::5] = 1.25                                         # all equal
    tails = g.integers(0, cols + 1, rows)
    for r in range(0, rows, 2):
        s[r, tails[r]:] = -np.inf
    for r in range(rows):
        at = g.integers(0, cols, 6)
        s[r, at] = np.array([np.nan, np.inf, -np.inf, -0.0, 0.0, np.finfo(np.float32).min], np.float32)
    s[rows // 2:rows // 2 + 1] = -np.inf if rows > 1 else s[:1]     # a row that keeps nothing
    bands = Banded()
    out = bands.bytes(rows * keep * 4, "cuda").view(torch.int32).view(rows, keep)
    got = select_blocks(torch.from_numpy(s).cuda(), keep, first, out=out)
    bands.check("after a selection")
    want = ref_select(s, keep, first)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("rows,cols,keep,first", [
    (384, 257, 30, 1), (383, 300, 30, 1), (401, 511, 511, 0), (390, 512, 64, 64), (385, 513, 1, 1), (402, 800, 799, 2),
    (400, 1023, 128, 1), (387, 1024, 900, 0), (386, 1025, 100, 3)])
def test_select_many_rows(rows, cols, keep, first):
    """Rows of a warp's 16 and 32 keys a lane, and the sizes beside them."""
    test_select_against_sort(rows, cols, keep, first)


def test_select_strided_rows_and_odd_offsets():
    g = torch.Generator(device="cuda").manual_seed(3)
    big = torch.randn(11, 301, generator=g, device="cuda")
    part = big[:, 3:204]                                   # rows of 201 columns, 301 apart, 4-byte aligned
    got = select_blocks(part, 17, 2)
    assert np.array_equal(got.cpu().numpy(), ref_select(part.cpu().numpy(), 17, 2))
    three = torch.randn(4, 3, 50, generator=g, device="cuda")
    got = select_blocks(three, 9)
    assert got.shape == (4, 3, 9)
    assert np.array_equal(got.view(12, 9).cpu().numpy(), ref_select(three.view(12, 50).cpu().numpy(), 9, 0))
    assert select_blocks(three, 0).shape == (4, 3, 0)
    empty = select_blocks(torch.empty(5, 0, device="cuda"), 3)
    assert (empty == -1).all()


def test_select_crowded_bins():
    """Rows whose wanted score sits among many near ones: bins that hold more keys than
    are ranked, ranges that shrink by rounds, outliers that stretch the first range."""
    g = np.random.default_rng(9)
    rows = [np.concatenate([np.full(2, 3e38), 5 + 1e-4 * g.random(4000), np.full(98, -3e38)]),
            np.concatenate([np.full(50, 7.0), 5 + 1e-6 * g.integers(0, 3, 4050)]),
            5 + 1e-6 * g.random(4100), np.concatenate([-g.random(2000) * 1e-30, g.random(2100) * 1e-30]),
            np.concatenate([np.full(4000, 1.0), np.full(100, np.inf)])]
    s = np.stack([g.permutation(r) for r in rows]).astype(np.float32)
    for cols in (4100, 600, 200):
        for keep in (1, 60, 150):
            got = select_blocks(torch.from_numpy(s[:, :cols].copy()).cuda(), keep, 1)
            assert np.array_equal(got.cpu().numpy(), ref_select(s[:, :cols], keep, 1)), (cols, keep)


def test_select_bits_that_differ_low_down():
    """Scores that agree in all but their last bits, of both signs."""
    base = np.array([1.0, -1.0, 1e-38, -1e-38, 3e38], np.float32)
    rows = []
    for x in base:
        u = np.full(3000, x, np.float32).view(np.uint32) + np.random.default_rng(5).integers(0, 7, 3000).astype(np.uint32)
        rows.append(u.view(np.float32))
    s = np.stack(rows)
    for keep in (1, 2, 499, 1500, 2999):
        got = select_blocks(torch.from_numpy(s).cuda(), keep)
        assert np.array_equal(got.cpu().numpy(), ref_select(s, keep, 0)), keep


# ---- scores and decode over lists, every instance ------------------------------------------


@pytest.mark.parametrize("combo", COMBOS, ids=IDS)
def test_every_dense_instance(combo):
    D, bits, nq, G = combo
    R = max(G, 64)
    rng = random.Random(sum(combo))
    Hkv = 2
    cache, oc, q = dense(3, Hkv * nq, Hkv, D, bits, G, R, 7 * G + R + 5, sum(combo), n_app=R // 2)
    nb = cache.counts()[0] // G
    out = cache.bands.bytes(3 * Hkv * (nb + 3) * 4, "cuda").view(torch.float32).view(3, Hkv, nb + 3)
    check_scores(cache.block_scores(q, out=out), oc, q, bits, Hkv, nq)
    for n in (nb, 3):
        blocks = lists(rng, 3 * Hkv, lambda r: nb, n).reshape(3, Hkv, n)
        got = cache.decode_blocks(q, torch.from_numpy(blocks).cuda(), out=cache.bands.like(q))
        cache.bands.check("after a decode over blocks")
        check_decode(got, oc, q, blocks, G, nq)


@pytest.mark.parametrize("combo", COMBOS, ids=IDS)
def test_every_paged_instance(combo):
    D, bits, nq, G = combo
    R = max(G, 64)
    rng = random.Random(sum(combo) + 1)
    Hkv = 2
    lengths = [9 * G + R + 3, 1, R, 2 * G + R + 1, 5 * G]
    cache, seqs, oc, q = paged(lengths, Hkv * nq, Hkv, D, bits, G, R, sum(combo))
    check_scores(cache.block_scores(seqs, q), oc, q, bits, Hkv, nq)
    for n in (12, 2):
        blocks = lists(rng, 5 * Hkv, lambda r: oc[r // Hkv, r % Hkv].n_quant // G, n).reshape(5, Hkv, n)
        got = cache.decode_blocks(seqs, q, torch.from_numpy(blocks).cuda(), out=cache.bands.like(q))
        cache.bands.check("after a paged decode over blocks")
        check_decode(got, oc, q, blocks, G, nq)


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 97, 130, 161])
def test_short_contexts(L):
    """From one token on: no block at all, one block, residuals of every size class."""
    G, R = 32, 64
    cache, oc, q = dense(2, 4, 2, 128, 2, G, R, L, 50 + L)
    nb = cache.counts()[0] // G
    scores = cache.block_scores(q)
    assert scores.shape == (2, 2, nb)
    check_scores(scores, oc, q, 2, 2, 2)
    blocks = np.tile(np.arange(nb, dtype=np.int32), (2, 2, 1))
    check_decode(cache.decode_blocks(q, torch.from_numpy(blocks).cuda()), oc, q, blocks, G, 2)
    none = np.full((2, 2, 3), -1, np.int32)
    check_decode(cache.decode_blocks(q, torch.from_numpy(none).cuda()), oc, q, none, G, 2)
    empty = torch.empty(2, 2, 0, dtype=torch.int32, device="cuda")
    check_decode(cache.decode_blocks(q, empty), oc, q, empty.cpu().numpy(), G, 2)   # (another split: not bit for bit)
    assert torch.equal(cache.sparse_decode(q, 64), cache.decode_blocks(q, torch.from_numpy(blocks).cuda()))


@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 2, 32, 70000), (1, 4, 1, 128, 4, 128, 40000), (5, 3, 3, 128, 8, 64, 3500)],
                         ids=["D64G32", "D128G128nq4", "b8"])
def test_lists_longer_than_a_warp_keeps(shape):
    """Every block listed: a warp's share passes the entries it keeps at a time;
    the result is the whole cache's decode."""
    B, Hq, Hkv, D, bits, G, L = shape
    cache, oc, q = dense(B, Hq, Hkv, D, bits, G, 2 * G, L, 5)
    nb = cache.counts()[0] // G
    rng = random.Random(4)
    blocks = np.stack([rng.sample(range(nb), nb) for _ in range(B * Hkv)]).astype(np.int32).reshape(B, Hkv, nb)
    got = cache.decode_blocks(q, torch.from_numpy(blocks).cuda())
    check_decode(got, oc, q, blocks, G, Hq // Hkv)
    whole = cache.decode_attn(q)
    full = {k: ref_decode(o, q.cpu().numpy()[k[0], k[1] * (Hq // Hkv):(k[1] + 1) * (Hq // Hkv)], range(nb), G)[1]
            for k, o in oc.items()}
    worst = max(float(b.max()) for b in full.values())
    assert (got.float() - whole.float()).abs().max().item() <= 2 * worst


def test_many_rows():
    """More rows than the GPU holds at once, one CTA each."""
    cache, oc, q = dense(80, 8, 8, 64, 4, 32, 32, 200, 21, sink=False)
    nb = cache.counts()[0] // 32
    blocks = lists(random.Random(1), 640, lambda r: nb, 3).reshape(80, 8, 3)
    some = {k: oc[k] for k in [(0, 0), (17, 3), (41, 7), (79, 7)]}
    check_scores(cache.block_scores(q), some, q, 4, 8, 1)
    check_decode(cache.decode_blocks(q, torch.from_numpy(blocks).cuda()), some, q, blocks, 32, 1)


@pytest.mark.parametrize("B,Hkv,nq,bits,G,L,keep", [
    (1, 1, 1, 2, 32, 900, 20), (1, 3, 2, 4, 64, 1200, 9), (1, 8, 1, 2, 32, 4000, 100), (2, 32, 1, 2, 32, 1500, 40),
    (8, 19, 1, 2, 32, 700, 12), (9, 17, 4, 4, 64, 700, 5), (16, 19, 1, 8, 32, 600, 12), (38, 16, 2, 2, 32, 400, 6),
    (61, 25, 1, 2, 32, 300, 4)])
def test_row_counts(B, Hkv, nq, bits, G, L, keep):
    """From one row to ten times what the GPU's SMs hold: clusters of 8 CTAs down to
    several waves of small ones, one or more than one row an SM."""
    cache, oc, q = dense(B, Hkv * nq, Hkv, 128 if B < 30 else 64, bits, G, G, L, B + Hkv)
    nb = cache.counts()[0] // G
    rng = random.Random(B)
    blocks = lists(rng, B * Hkv, lambda r: nb, keep).reshape(B, Hkv, keep)
    got = cache.decode_blocks(q, torch.from_numpy(blocks).cuda(), out=cache.bands.like(q))
    cache.bands.check("after a decode over blocks")
    rows = {(0, 0), (B - 1, Hkv - 1)} | {(rng.randrange(B), rng.randrange(Hkv)) for _ in range(6)}
    some = {r: oc[r] for r in rows}
    check_decode(got, some, q, blocks, G, nq)
    check_scores(cache.block_scores(q), some, q, bits, Hkv, nq)


@pytest.mark.parametrize("B,Hkv,nq,D,L", [(330, 8, 1, 64, 5), (90, 32, 2, 128, 40), (1040, 63, 1, 64, 16)])
def test_many_rows_with_one_tile_each(B, Hkv, nq, D, L):
    """Thousands of rows that have at most one residual tile to read: more rows
    than the SMs hold warps, none with work for two of them."""
    cache, oc, q = dense(B, Hkv * nq, Hkv, D, 2, 32, 32, L, B)
    some = {r: oc[r] for r in [(0, 0), (B // 2, Hkv // 3), (B - 1, Hkv - 1)]}
    nothing = torch.empty(B, Hkv, 0, dtype=torch.int32, device="cuda")
    got = cache.decode_blocks(q, nothing, out=cache.bands.like(q))
    cache.bands.check("after a decode of one tile a row")
    check_decode(got, some, q, nothing.cpu().numpy(), 32, nq)


def test_many_paged_rows_with_one_tile_each():
    lengths = [1 + i % 16 for i in range(46)]
    cache, seqs, oc, q = paged(lengths, 64, 64, 64, 2, 32, 32, 31)
    none = np.full((46, 64, 2), -1, np.int32)
    got = cache.decode_blocks(seqs, q, torch.from_numpy(none).cuda())
    cache.bands.check("after a paged decode of one tile a row")
    some = {r: oc[r] for r in [(0, 0), (15, 63), (30, 7), (45, 40)]}
    check_decode(got, some, q, none, 32, 1)


def test_offsets_past_4_gib():
    """A dense cache and a page pool of more than 4 GiB: the last rows' blocks, scores and tables."""
    B, H, D, bits, G, R, L = 8, 32, 128, 8, 32, 32, 60000
    syn = SynthKV(B, H, H, D, 3, device="cuda")
    Kp, Vp = syn.prompt(L)
    q = syn.step(0)[0]
    some = {}
    for r in [(0, 0), (7, 31), (7, 0)]:
        some[r] = OracleCache(1, 1, D, bits, G, R)
        some[r].prefill(Kp[r][None, None].cpu().numpy(), Vp[r][None, None].cpu().numpy())
    nb = some[0, 0].n_quant // G
    blocks = np.sort(np.random.default_rng(1).integers(0, nb, (B, H, 9)).astype(np.int32), axis=-1)
    blocks[..., -1] = nb - 1
    bt = torch.from_numpy(blocks).cuda()
    cache = KiviCache(B, H, H, D, bits, G, R, L + 1)
    assert cache.buffer.numel() > 1 << 32
    cache.prefill(Kp, Vp)
    check_scores(cache.block_scores(q), some, q, bits, H, 1)
    check_decode(cache.decode_blocks(q, bt), some, q, blocks, G, 1, "dense")
    del cache
    pool = KiviPagedCache(B, H, H, D, bits, G, R, nb + 1, B * nb + 3)
    assert pool.buffer.numel() > 1 << 32
    seqs = [pool.add(Kp[b], Vp[b]) for b in range(B)]
    check_scores(pool.block_scores(seqs, q), some, q, bits, H, 1)
    check_decode(pool.decode_blocks(seqs, q, bt), some, q, blocks, G, 1, "paged")


def test_block_listed_twice_counts_twice():
    cache, oc, q = dense(1, 2, 2, 64, 2, 32, 32, 300, 9)
    blocks = np.array([[[2, 2, 5, 2], [0, 1, 1, 7]]], np.int32)
    check_decode(cache.decode_blocks(q, torch.from_numpy(blocks).cuda()), oc, q, blocks, 32, 1)


def test_entries_outside_the_cache_make_their_row_nan():
    """An entry past the last block is not read; only its row's heads become NaN."""
    for make in ("dense", "paged"):
        if make == "dense":
            cache, oc, q = dense(3, 4, 2, 128, 2, 32, 64, 400, 31)
            call = lambda b: cache.decode_blocks(q, b)  # noqa: E731
        else:
            cache, seqs, oc, q = paged([400, 300, 420], 4, 2, 128, 2, 32, 64, 31)
            call = lambda b: cache.decode_blocks(seqs, q, b)  # noqa: E731
        blocks = torch.zeros(3, 2, 4, dtype=torch.int32, device="cuda")
        blocks[..., 1:] = torch.tensor([3, 5, 1], device="cuda")
        good = call(blocks)
        for bad in (oc[1, 1].n_quant // 32, 2 ** 31 - 1):
            b2 = blocks.clone()
            b2[1, 1, 2] = bad
            out = call(b2)
            assert out[1, 2:].isnan().all()
            out[1, 2:] = good[1, 2:]
            assert torch.equal(out, good)
        check_decode(call(blocks), oc, q, blocks.cpu().numpy(), 32, 2)


def test_entries_past_the_rows_blocks_are_not_read():
    """A ragged row reads as many entries as its sequence has blocks."""
    cache, seqs, oc, q = paged([64, 400], 2, 2, 64, 2, 32, 64, 3)
    blocks = torch.full((2, 2, 12), -1, dtype=torch.int32, device="cuda")
    blocks[1] = torch.arange(12, device="cuda") % 10
    want = cache.decode_blocks(seqs, q, blocks)
    blocks[0] = 2 ** 30                                     # sequence 0 has no block
    assert torch.equal(cache.decode_blocks(seqs, q, blocks), want)


def test_masked_and_extreme_queries():
    """Scales that flatten or sharpen the softmax, a zero query, and NaN kept to its rows."""
    cache, oc, q = dense(2, 2, 2, 128, 4, 64, 64, 500, 13)
    nb = cache.counts()[0] // 64
    blocks = np.tile(np.arange(0, nb, 2, dtype=np.int32), (2, 2, 1))
    bt = torch.from_numpy(blocks).cuda()
    for scale in (1e-6, 0.02, 3.0):
        out = cache.decode_blocks(q, bt, softmax_scale=scale).cpu().numpy()
        for (i, h), o in oc.items():
            ref, bound = ref_decode(o, q[i, h:h + 1].cpu().numpy(), blocks[i, h], 64, scale)
            assert_within(out[i, h:h + 1], ref, bound, f"scale {scale}")
    zero = torch.zeros_like(q)
    check_decode(cache.decode_blocks(zero, bt), oc, zero, blocks, 64, 1)
    good = cache.decode_blocks(q, bt)
    bad = q.clone()
    bad[1, 0, 5] = float("nan")
    out, sc = cache.decode_blocks(bad, bt), cache.block_scores(bad)
    assert out[1, 0].isnan().all() and sc[1, 0].isnan().all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[1, 1], good[1, 1])
    assert (select_blocks(sc, 4)[1, 0] == -1).all()


# ---- the steps together -----------------------------------------------------------------


def test_what_a_selection_leaves_out():
    """The softmax mass mu of the blocks left out is at most what their scores allow,
    sum over them of G exp(score) over the total, and leaving it out moves the output
    by at most 2 mu max|v| (whole = (1 - mu) sparse + mu rest)."""
    B, Hq, Hkv, D, bits, G, nq = 2, 4, 2, 128, 4, 32, 2
    cache, oc, q = dense(B, Hq, Hkv, D, bits, G, 64, 2000, 6)
    scores = cache.block_scores(q)
    blocks = select_blocks(scores, 12, 1).cpu().numpy()
    sparse, whole = (t.cpu().numpy().astype(np.float64) for t in (cache.sparse_decode(q, 12), cache.decode_attn(q)))
    for (b, h), o in oc.items():
        sl = slice(h * nq, (h + 1) * nq)
        qn, sc = q[b, sl].cpu().numpy(), scores[b, h].cpu().numpy().astype(np.float64)
        x = qn.astype(np.float64) @ o.keys_hat()[0, 0].T / np.sqrt(D)
        out = np.setdiff1d(np.arange(sc.size), blocks[b, h])
        total = np.exp(x).sum(1)
        mu = np.exp(x.reshape(nq, -1)[:, np.concatenate([np.arange(n * G, (n + 1) * G) for n in out])]).sum(1) / total
        assert (mu <= G * np.exp(sc[out] * (1 + 1e-5)).sum() / total).all()
        vmax = np.abs(o.values_hat()).max()
        _, b1 = ref_decode(o, qn, blocks[b, h], G)
        _, b2 = ref_decode(o, qn, range(sc.size), G)
        assert (np.abs(sparse[b, sl] - whole[b, sl]) <= 2 * mu[:, None] * vmax + b1 + b2).all()


@pytest.mark.parametrize("bits,G,R,Hq,Hkv", [(2, 32, 64, 4, 2), (4, 64, 64, 8, 2), (8, 128, 128, 2, 2)])
def test_dense_decode_steps(bits, G, R, Hq, Hkv):
    """A decode loop through append + scores + selection + attention, over flushes."""
    B, D, nq, L = 2, 128, Hq // Hkv, 5 * G + 3
    syn = SynthKV(B, Hq, Hkv, D, 8, device="cuda")
    Kp, Vp = syn.prompt(L)
    cache = GuardedCache(B, Hq, Hkv, D, bits, G, R, L + 200)
    cache.prefill(Kp, Vp)
    oc = {(b, h): OracleCache(1, 1, D, bits, G, R) for b in range(B) for h in range(Hkv)}
    for (b, h), o in oc.items():
        o.prefill(Kp[b, h][None, None].cpu().numpy(), Vp[b, h][None, None].cpu().numpy())
    for s in range(R + 10):
        q, k, v = syn.step(s)
        cache.append(k, v)
        for (b, h), o in oc.items():
            o.append(k[b, h][None, None].cpu().numpy(), v[b, h][None, None].cpu().numpy())
        if s % 7 and s < R - 3:
            cache.sparse_decode(q, 3)
            continue
        scores = cache.block_scores(q)
        check_scores(scores, oc, q, bits, Hkv, nq)
        n = min(3, scores.shape[-1])
        blocks = select_blocks(scores, n, 1)
        want = ref_select(scores.reshape(B * Hkv, -1).cpu().numpy(), n, 1).reshape(B, Hkv, -1)
        assert np.array_equal(blocks.cpu().numpy(), want)
        out = cache.sparse_decode(q, 3, out=cache.bands.like(q))
        cache.bands.check(f"after step {s}")
        assert torch.equal(out, cache.decode_blocks(q, blocks))
        check_decode(out, oc, q, want, G, nq, f"step {s}")


def test_paged_append_and_decode_steps():
    """kivi_paged_append leaves the cache as kivi_paged_append_decode does, and the
    sparse steps over changing subsets agree with the oracle."""
    G, R, Hq, Hkv, D, bits = 32, 64, 4, 2, 64, 4
    rng = random.Random(2)
    lengths = [0, 1, 64, 200, 333]
    caches = [GuardedPagedCache(5, Hq, Hkv, D, bits, G, R, 24, 100) for _ in range(2)]
    syns = [SynthKV(1, Hq, Hkv, D, 40 + i, device="cuda") for i in range(5)]
    oc = {}
    for i, L in enumerate(lengths):
        Kp, Vp = syns[i].prompt(L)
        for c in caches:
            assert c.add(Kp[0].contiguous(), Vp[0].contiguous()) == i
        for h in range(Hkv):
            oc[i, h] = OracleCache(1, 1, D, bits, G, R)
            oc[i, h].prefill(Kp[:, h:h + 1].cpu().numpy(), Vp[:, h:h + 1].cpu().numpy())
    for s in range(90):
        seqs = rng.sample(range(5), rng.randint(1, 5))
        q, k, v = (torch.stack(t).contiguous() for t in zip(*[[x[0] for x in syns[i].step(s)] for i in seqs]))
        caches[0].append(seqs, k, v)
        whole = caches[1].append_decode(seqs, k, v, q)
        for j, i in enumerate(seqs):
            for h in range(Hkv):
                oc[i, h].append(k[j, h][None, None].cpu().numpy(), v[j, h][None, None].cpu().numpy())
        assert [caches[0].counts(i) for i in range(5)] == [caches[1].counts(i) for i in range(5)]
        assert torch.equal(caches[0].append_decode(seqs, None, None, q), whole)
        if s % 9 == 0:
            rows = {(j, h): oc[i, h] for j, i in enumerate(seqs) for h in range(Hkv)}
            scores = caches[0].block_scores(seqs, q)
            check_scores(scores, rows, q, bits, Hkv, 2)
            n = min(4, scores.shape[-1])
            want = ref_select(scores.reshape(len(seqs) * Hkv, -1).cpu().numpy(), n, min(1, n)).reshape(len(seqs), Hkv, n)
            out = caches[0].sparse_decode(seqs, q, 4)
            caches[0].bands.check(f"after step {s}")
            check_decode(out, rows, q, want, G, 2, f"step {s}")
    for i in range(5):
        assert caches[0].pages(i) == caches[1].pages(i)
    assert caches[0].free() == caches[1].free()


# ---- streams, graphs -------------------------------------------------------------------


def test_captured_steps_replay_with_new_queries():
    """Two captures of the same cache's steps, replayed in turn and beside each other."""
    cache, oc, q0 = dense(2, 4, 2, 128, 2, 32, 64, 900, 17)
    qs = [q0, SynthKV(2, 4, 2, 128, 17, device="cuda").step(5)[0]]
    want = [cache.sparse_decode(q, 6) for q in qs]
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        q = qs[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = cache.sparse_decode(q, 6)
        runs.append((g, q, out))
    for order in ((0, 1), (1, 0)):
        for (g, q, _), j in zip(runs, order):
            q.copy_(qs[j])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in runs]
        for (g, _, _), st in zip(runs, streams):
            with torch.cuda.stream(st):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for (_, _, out), j in zip(runs, order):
            assert torch.equal(out, want[j])


def test_two_streams_at_once():
    cache, oc, q = dense(4, 8, 8, 128, 2, 32, 128, 3000, 3)
    q2 = torch.flip(q, [0]).contiguous()
    want = [cache.sparse_decode(x, 8) for x in (q, q2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for j, x in enumerate((q, q2)):
            outs[j].append(cache.sparse_decode(x, 8, stream=st[j]))
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j]) for o in outs[j])


def test_outputs_allocated_on_a_side_stream():
    """Calls on a side stream take their outputs from that stream's memory: work of the
    current stream that is still running cannot meet them."""
    cache, oc, q = dense(2, 4, 4, 128, 2, 32, 64, 2000, 12)
    want_s, want_o = cache.block_scores(q), cache.sparse_decode(q, 6)
    want_b = select_blocks(want_s, 6, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        big = torch.full((want_s.numel() * 4,), 7.0, device="cuda")
        for _ in range(20):
            big = big * 1.0001
        del big                                             # its memory is free again while it is still written
        s = cache.block_scores(q, stream=side)
        b = select_blocks(s, 6, 1, stream=side)
        o = cache.decode_blocks(q, b, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(s, want_s) and torch.equal(b, want_b) and torch.equal(o, want_o)


def test_copy_wait_runs_out_marks_its_row():
    """The failure-detection hook: the wait of one warp runs out (about 2 s), the heads
    of its row are NaN, the others and the next call are right."""
    cache, oc, q = dense(2, 4, 2, 64, 2, 32, 64, 600, 8)
    blocks = torch.arange(6, dtype=torch.int32, device="cuda").expand(2, 2, 6).contiguous()
    want = cache.decode_blocks(q, blocks)
    K.kivi_cache_set_fault(cache.handle, K.KIVI_FAULT_COPY_STALL)
    out = cache.decode_blocks(q, blocks)
    torch.cuda.synchronize()
    assert out[0, :2].isnan().all()
    out[0, :2] = want[0, :2]
    assert torch.equal(out, want)
    assert torch.equal(cache.decode_blocks(q, blocks), want)


def test_refusals_with_tensors():
    cache, oc, q = dense(1, 2, 2, 64, 2, 32, 32, 200, 1)
    nb = cache.counts()[0] // 32
    ok = torch.zeros(1, 2, 2, dtype=torch.int32, device="cuda")
    bad = [lambda: cache.decode_blocks(q.float(), ok), lambda: cache.decode_blocks(q, ok.long()),
           lambda: cache.decode_blocks(q, ok[:, :1]), lambda: cache.decode_blocks(q, ok.cpu()),
           lambda: cache.decode_blocks(q.cpu(), ok), lambda: cache.block_scores(q[:, :1]),
           lambda: cache.block_scores(q, out=torch.empty(1, 2, nb - 1, device="cuda")),
           lambda: cache.decode_blocks(q, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")[..., ::2]),
           lambda: cache.block_scores(q, softmax_scale=float("nan")),
           lambda: select_blocks(torch.zeros(2, 3, device="cuda"), 2, 3),
           lambda: select_blocks(torch.zeros(2, 3, device="cuda"), -1),
           lambda: select_blocks(torch.zeros(2, 3), 1), lambda: select_blocks(torch.zeros(2, 3, device="cuda").half(), 1),
           lambda: select_blocks(torch.zeros(3, 2, device="cuda").T, 1)]
    for f in bad:
        with pytest.raises((K.KiviError, RuntimeError)):
            f()
    torch.cuda.synchronize()
    queue = KiviCache(1, 2, 2, 64, 2, 32, 32, 300)
    queue.set_value_residual(K.KIVI_VALUE_QUEUE)
    Kp, Vp = SynthKV(1, 2, 2, 64, 1, device="cuda").prompt(200)
    queue.prefill(Kp, Vp)
    with pytest.raises(K.KiviError) as e:
        queue.decode_blocks(q, ok)
    assert e.value.status == K.KIVI_ERR_UNSUPPORTED
    check_scores(queue.block_scores(q), oc, q, 2, 2, 1)     # keys as with the default residual
