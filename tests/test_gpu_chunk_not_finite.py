"""Values that are not finite make the outputs that see them NaN, whole rows of them, and change no other output: in long
prompts and between the ends of a window."""
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
