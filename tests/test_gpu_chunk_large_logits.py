"""Chunk attention where scores reach 2^18 to 2^40, whose neighbours in fp32 are up to 2^17 apart: a row's largest
score takes all, equal ones share, and scores of a common size behind hugely negative ones keep their weights.

Each score is one product of two fp16 numbers times a power of two, exact in fp32, so their order is exact; times log2(e)
they are not.  The
weights that count are off by 2^-21 and rounded to fp16 (2^-11), the output by 2^-11: 2^-10 + 2^-19 of sum w |v| in all."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from chunk_harness import ChunkRun  # noqa: E402

MOST = 2.0 ** -10 + 2.0 ** -19


def attend(run, seqs, n, q, k, v, e, slopes=None):
    """Scores k[:, :, 0] * 2^(e - 11): q's first channel is 2^14."""
    return run.attend(seqs, [n], (q, k, v), scale=2.0 ** (e - 25), slopes=slopes, check=False)


def inputs(run, n, values):
    q, k, v = run.chunk([n])
    q.zero_()
    k.zero_()
    q[:, :, 0] = 2.0 ** 14
    k[:, 0, 0] = values
    return q, k, v


@pytest.mark.parametrize("e", [18, 20, 24, 27, 29, 33, 40])
@pytest.mark.parametrize("mod", [False, True])
@pytest.mark.parametrize("kind", ["both signs", "negative", "rising", "falling", "ties"])
def test_the_largest_logit_takes_all(e, mod, kind):
    n = 400
    run = ChunkRun(1, 1, 64, 2, 32, 32, max_seqs=1, seed=e)
    s = run.add(0)
    g = torch.Generator(device="cuda").manual_seed(e)
    r = torch.randperm(2000, generator=g, device="cuda")[:n].float()
    if kind == "both signs":
        r -= 1000
    elif kind == "negative":
        r -= 2001
    elif kind == "ties":
        r = torch.randint(1, 40, (n,), generator=g, device="cuda").float() * 50
    else:
        r = r.sort(descending=kind == "falling").values
    q, k, v = inputs(run, n, r)
    out = attend(run, [s], n, q, k, v, e, torch.zeros(1, device="cuda") if mod else None)[:, 0].double()
    hidden = torch.ones(n, n, device="cuda").triu(1).bool()
    x = r.double()[None].masked_fill(hidden, -math.inf)
    w = (x == x.amax(1, keepdim=True)).double()                  # (r is whole, a step of it 2^7 at least)
    w /= w.sum(1, keepdim=True)
    ref, most = w @ v[:, 0].double(), MOST * (w @ v[:, 0].double().abs()) + 2.0 ** -24
    assert ((out - ref).abs() <= most).all()


@pytest.mark.parametrize("at", [1, 60, 64, 100, 128, 150, 200, 256, 300])
@pytest.mark.parametrize("mod", [False, True])
@pytest.mark.parametrize("e", [26, 33])
def test_common_logits_behind_hugely_negative_ones(at, mod, e):
    n = 400
    run = ChunkRun(1, 1, 64, 2, 32, 32, max_seqs=1, seed=at)
    s = run.add(0)
    g = torch.Generator(device="cuda").manual_seed(at)
    x = torch.randint(-12, 13, (n,), generator=g, device="cuda").float() / 2       # scores
    r = x * 2.0 ** (11 - e)                                       # (2^-23 steps at e = 33: fp16 holds them)
    r[:at] = -2.0 ** 9 - torch.arange(at, device="cuda")          # -2^(e - 2) and below
    q, k, v = inputs(run, n, r)
    assert torch.equal(k[at:, 0, 0].double() * 2.0 ** (e - 11), x[at:].double())
    out = attend(run, [s], n, q, k, v, e, torch.zeros(1, device="cuda") if mod else None)[at:, 0].double()
    hidden = torch.ones(n, n, device="cuda").triu(1).bool()[at:, at:]
    w = torch.softmax(x[at:].double()[None].masked_fill(hidden, -math.inf), 1)
    # (log2(e) in fp32, products and differences with the reference: 12 log2(e) is off by 2^-19, and so are the weights)
    ref, most = w @ v[at:, 0].double(), (MOST + 2.0 ** -18) * (w @ v[at:, 0].double().abs()) + 2.0 ** -24
    assert ((out - ref).abs() <= most).all()


def test_equal_logits_of_different_parts_share():
    """One row of queries over 33000 cached tokens on all CTAs: the parts' references are the same numbers."""
    for e in (20, 29, 36):
        run = ChunkRun(1, 1, 128, 2, 32, 128, max_seqs=1, max_blocks=1100, n_pages=1100, seed=e)
        K, V, _ = run.draw(33000)
        K.zero_()
        K[:, ::32, 0] = 48.0                                      # (codes 0 and 3 of a step of 16)
        s = run.add(33000, (K, V))
        q, k, v = inputs(run, 20, -64.0)
        out = attend(run, [s], 20, q, k, v, e)[:, 0].double()
        oc = run.live[s]
        hat = torch.from_numpy(oc.keys_hat()[0]).cuda()[0, :, 0]
        vals = torch.from_numpy(oc.values_hat()[0]).cuda()[0].double()
        assert set(hat.tolist()) == {0.0, 48.0}
        w = (hat == 48.0).double()
        w /= w.sum()
        ref = w @ vals
        # values rounded to fp16, sums of 33000 tokens
        most = (MOST + 2.0 ** -11 + (64 + 33000 / 16) * 2.0 ** -23) * (w @ vals.abs()) + 2.0 ** -24
        assert ((out - ref).abs() <= most).all(), e
