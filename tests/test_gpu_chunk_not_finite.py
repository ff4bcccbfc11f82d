"""Values that are not finite make the outputs that see them NaN, whole rows of them, and change no other output: in long
prompts, between the ends of a window, among few rows and in the cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300.kivi import KiviPagedCache  # noqa: E402
from chunk_harness import ChunkRun  # noqa: E402


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("tokens", [(150,), (10, 290), (10, 290, 150), (0, 299), (40, 41, 128, 260)])
@pytest.mark.parametrize("window", [0, 1, 20, 100, 250])
@pytest.mark.parametrize("D,nq,cached", [(128, 1, 0), (64, 4, 300), (128, 2, 70)])
def test_a_window_between_two_of_them(tokens, window, D, nq, cached):
    run = ChunkRun(nq, 1, D, 4, 32, 64, max_seqs=1, seed=D)
    s = run.add(cached)
    q, k, v = run.chunk([300])
    clean = run.attend([s], [300], (q, k, v), window=window, check=False)
    bad = v.clone()
    for j, t in enumerate(tokens):
        bad[t, 0, 7 * j % D] = (float("inf"), float("nan"), float("-inf"))[j % 3]
    out = run.attend([s], [300], (q, k, bad), window=window, check=False)
    at = torch.arange(300, device="cuda")[:, None]
    t = torch.tensor(tokens, device="cuda")[None]
    sees = ((t <= at) & ((t > at - window) if window else True)).any(1)
    assert torch.isnan(out[sees]).all() and same(out[~sees], clean[~sees])


@pytest.mark.parametrize("window", [0, 1000])
def test_a_long_prompt_with_a_late_one(window):
    n, t = 300_000, 299_001
    c = KiviPagedCache(1, 1, 1, 128, 2, 32, 32, 4, 4)
    s = c.add(*(torch.zeros(1, 0, 128, dtype=torch.half, device="cuda") for _ in range(2)))
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(n, 1, 128, generator=g, device="cuda").half() for _ in range(3))
    clean = c.chunk_attn([s], [n], q, k, v, window=window)
    assert torch.isfinite(clean).all()
    v[t, 0, 100] = float("inf")
    if window:
        v[5, 0, 0] = float("nan")
    out = c.chunk_attn([s], [n], q, k, v, window=window)
    first = 5 + window if window else 0
    assert same(out[first:t], clean[first:t])
    assert torch.isnan(out[t:t + (window or n)]).all() and torch.isnan(out[5:first]).all()
    if window:
        assert same(out[t + window:], clean[t + window:]) and same(out[:5], clean[:5])


@pytest.mark.parametrize("D,bits,G,nq", [(128, 2, 32, 1), (64, 4, 64, 2), (128, 8, 128, 4), (64, 2, 32, 4)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("weight", ["some", "none"])
def test_few_rows_that_see_one(D, bits, G, nq, value, weight):
    """A new token's: NaN for every channel from that token on.  A residual one's: for every row.  Whatever weight the
    token has: with keys far from every query its exponential is 0."""
    run = ChunkRun(2 * nq, 2, D, bits, G, 2 * G, max_seqs=2, seed=D + bits)
    n = 16 // nq
    L = 700
    K, V, _ = run.draw(L)
    q, k, v = run.chunk([n])
    if weight == "none":
        q = q.abs() + 1
        k[n // 2] = -3000.0
        K[:, L - 3] = -3000.0
    s = run.cache.add(K, V)
    clean = run.attend([s], [n], (q, k, v), check=False)
    assert torch.isfinite(clean).all()
    bad = v.clone()
    bad[n // 2, 0, 5] = value                                     # kv head 0 alone
    out = run.attend([s], [n], (q, k, bad), check=False)
    assert torch.isnan(out[n // 2:, :nq]).all()
    assert same(out[:n // 2], clean[:n // 2]) and same(out[:, nq:], clean[:, nq:])
    run.cache.release(s)
    V[1, L - 3, D - 1] = value                                    # kv head 1, a residual row
    s = run.cache.add(K, V)
    out = run.attend([s], [n], (q, k, v), check=False)
    assert torch.isnan(out[:, nq:]).all() and same(out[:, :nq], clean[:, :nq])


@pytest.mark.parametrize("D,bits,G,nq", [(128, 2, 32, 1), (64, 4, 64, 2), (128, 8, 128, 4)])
def test_few_rows_over_a_quantized_one(D, bits, G, nq):
    """An infinity in a quantized token's group: its values read back as such, and no row of that head is a number."""
    run = ChunkRun(2 * nq, 2, D, bits, G, G, max_seqs=2, seed=D + bits)
    L = 900
    K, V, _ = run.draw(L)
    data = run.chunk([16 // nq])
    s = run.cache.add(K, V)
    clean = run.attend([s], [16 // nq], data, check=False)
    run.cache.release(s)
    V[0, 333, 1] = float("inf")
    s = run.cache.add(K, V)
    assert not torch.isfinite(run.cache.read([s], 333, 1)[1][0, 0]).all()
    out = run.attend([s], [16 // nq], data, check=False)
    assert torch.isnan(out[:, :nq]).all() and same(out[:, nq:], clean[:, nq:])
