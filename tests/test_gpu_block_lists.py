"""Lists of blocks in every form that a caller may give: -1 in front, among and behind, more
entries than the row has blocks, entries out of range anywhere."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from decode_bounds import Slot, close  # noqa: E402
from test_gpu_blocks import dense, paged  # noqa: E402


def check(out, oc, q, blocks, bits, nq, what=""):
    out, q = out.cpu().numpy(), q.cpu().numpy()
    for (i, h), o in oc.items():
        sl, slot = slice(h * nq, (h + 1) * nq), Slot(o, bits)
        ref, bound = slot.decode(q[i, sl], slot.tokens([int(x) for x in blocks[i, h]]), q.shape[-1] ** -0.5)
        close(out[i, sl], ref, bound, f"{what} row {(i, h)}")


def layouts(rng, rows, blocks_of, n):
    """Every row's blocks at places of its own in a list of n: in front, behind, spread, with repeats."""
    out = np.full((rows, n), -1, np.int32)
    for r in range(rows):
        nb = blocks_of(r)
        if not nb:
            continue
        m = rng.randint(1, min(n, nb + 3))
        pick = [rng.randrange(nb) for _ in range(m)] if r % 3 == 2 else rng.sample(range(nb), min(m, nb))
        at = {0: range(len(pick)), 1: range(n - len(pick), n), 2: sorted(rng.sample(range(n), len(pick))),
              3: sorted(rng.sample(range(n), len(pick)))}[r % 4]
        for a, b in zip(at, pick):
            out[r, a] = b
    return out


@pytest.mark.parametrize("D,bits,nq,G,n", [(128, 2, 1, 32, 3), (128, 2, 1, 32, 9), (64, 4, 2, 64, 40), (128, 4, 4, 128, 70),
                                           (128, 8, 1, 64, 200), (64, 2, 4, 32, 1100)])
def test_entries_anywhere(D, bits, nq, G, n):
    rng = random.Random(n)
    Hkv = 4
    cache, oc, q = dense(3, Hkv * nq, Hkv, D, bits, G, 2 * G, 8 * G + 5, n)
    nb = cache.counts()[0] // G
    for _ in range(2):
        blocks = layouts(rng, 3 * Hkv, lambda r: nb, n).reshape(3, Hkv, n)
        got = cache.decode_blocks(q, torch.from_numpy(blocks).cuda(), out=cache.bands.like(q))
        cache.bands.check("after a decode over blocks")
        check(got, oc, q, blocks, bits, nq, "dense")
    lengths = [7 * G + 1, 2 * G, 3 * G + 7, 20 * G, 2 * G + 1]
    pool, seqs, oc, q = paged(lengths, Hkv * nq, Hkv, D, bits, G, 2 * G, n)
    blocks = layouts(rng, 5 * Hkv, lambda r: oc[r // Hkv, r % Hkv].n_quant // G, n).reshape(5, Hkv, n)
    got = pool.decode_blocks(seqs, q, torch.from_numpy(blocks).cuda(), out=pool.bands.like(q))
    pool.bands.check("after a paged decode over blocks")
    check(got, oc, q, blocks, bits, nq, "paged")


def test_two_blocks_behind_an_empty_entry():
    """[-1, 0, 1] is [0, 1] of a cache of two blocks."""
    cache, oc, q = dense(2, 2, 2, 64, 2, 32, 32, 96, 4)
    assert cache.counts()[0] // 32 == 2
    for row in ([-1, 0, 1], [-1, -1, 1, -1, 0], [-1] * 50 + [1], [1, 1, 1, 0, 1]):
        blocks = np.tile(np.array(row, np.int32), (2, 2, 1))
        check(cache.decode_blocks(q, torch.from_numpy(blocks).cuda()), oc, q, blocks, 2, 1, str(row))


def test_entries_out_of_range_are_marked_wherever_they_stand():
    cache, oc, q = dense(2, 4, 2, 128, 2, 32, 64, 300, 5)
    nb = cache.counts()[0] // 32
    blocks = torch.full((2, 2, 3 * nb), -1, dtype=torch.int32, device="cuda")
    blocks[..., :3] = torch.arange(3, device="cuda")
    good = cache.decode_blocks(q, blocks)
    for place in (0, nb - 1, nb, 2 * nb + 1, 3 * nb - 1):
        b2 = blocks.clone()
        b2[1, 0, place] = nb
        out = cache.decode_blocks(q, b2)
        assert out[1, :2].isnan().all(), place
        out[1, :2] = good[1, :2]
        assert torch.equal(out, good), place


@pytest.mark.parametrize("n", [30, 31, 517, 4000])
def test_more_places_than_blocks(n):
    """A ragged row's blocks, then -1, in lists of any width."""
    cache, seqs, oc, q = paged([64, 400, 999, 120], 4, 2, 128, 2, 32, 64, 3)
    blocks = np.full((4, 2, n), -1, np.int32)
    for i, s in enumerate(seqs):
        nb = cache.counts(s)[0] // 32
        blocks[i, :, :nb] = np.arange(nb)
    got = cache.decode_blocks(seqs, q, torch.from_numpy(blocks).cuda(), out=cache.bands.like(q))
    cache.bands.check("after a paged decode over blocks")
    check(got, oc, q, blocks, 2, 2, str(n))
