"""Chunk calls on pages that lie past 4 GiB in the pool, with a residual and a block table behind them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from chunk_harness import ChunkRun  # noqa: E402


@pytest.mark.parametrize("D,bits,G,Hkv", [(128, 8, 32, 32), (64, 8, 64, 40)])
def test_pages_past_4_gib(D, bits, G, Hkv):
    page = Hkv * 2 * (G * D * bits // 8 + 4 * D)
    held = 2 ** 32 // page + 1
    run = ChunkRun(Hkv, Hkv, D, bits, G, 64, max_seqs=4, max_blocks=held + 1, n_pages=held + 200, seed=14)
    c = run.cache
    assert c.layout.page_bytes == page
    zeros = torch.zeros(Hkv, held * G + 64, D, dtype=torch.half, device="cuda")
    holder = c.add(zeros, zeros)                                  # every page below 4 GiB, and not given back
    del zeros
    assert c.counts(holder) == (held * G, 64)
    s = run.add(700)
    run.attend([s], [3])                                          # few rows
    run.attend([s], [40])                                         # the wide kernel
    run.attend([s], [1], window=300)
    run.append([s], [150])
    f = run.fork([s])[0]
    run.append([f, s], [1, 200])
    run.attend([f, s], [2, 130])
    run.check()
    for x in (s, f):
        assert min(c.pages(x)) * page >= 2 ** 32
        n = sum(c.counts(x))
        for first, count in ((0, n), (333, 200), (n - 90, 90)):
            for got, hat in zip(c.read([x], first, count), (run.live[x].keys_hat(), run.live[x].values_hat())):
                assert torch.equal(got[0], torch.from_numpy(hat[0][:, first:first + count]).half().cuda())
