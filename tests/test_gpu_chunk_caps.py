"""Capped scores of chunk attention at caps of every size: the bound follows the scores, not the cap.

As chunk_harness.ref_attend's, but for the cap's own error.  With y = score / cap, 1 - 2 / (exp(2 y) + 1) is off by under
2^-21.5 of 1 at |y| = 1/4 (the exponential and the division to 2^-22 each, of numbers up to 1, and y to 2^-23 of itself),
2^-19.5 of tanh(1/4), and 2^-20 of 1 at most.  Caps up to 64 are computed so throughout: 2^-20 of the cap.  With larger ones
tanh(y) is y times its series up to y^6 below 1/4 (the next term is 62/2835 y^8, 2^-21.5; five roundings of 2^-24): the
capped score is off by 2^-19 of itself.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from chunk_harness import ChunkRun  # noqa: E402


def reference(keys, vals, n_quant, q, past, scale, cap, window=0, slope=0.0):
    """(out, bound) [n][D] of one query head, in 64 bits."""
    n = q.shape[0]
    at = torch.arange(past, past + n, device=q.device)[:, None]
    t = torch.arange(past + n, device=q.device)
    raw = scale * (q @ keys.T)
    x = cap * torch.tanh(raw / cap)
    bias = slope * (t - at)
    hidden = t > at
    if window:
        hidden = hidden | (t <= at - window)
    size = (x.abs() + bias.abs()).masked_fill(hidden, 0.0)
    d = 2.0 ** -19 * x.abs() + (2.0 ** -20 * cap if cap <= 64 else 0.0)
    x = (x + bias).masked_fill(hidden, -math.inf)
    top = x.amax(1, keepdim=True)
    w = torch.softmax(x, dim=1)
    o = w @ vals
    deq = (t < n_quant).double()
    d = d + scale * (q.abs() @ keys.abs().T) * (2.0 ** -11 * deq + 2.0 ** -18)
    d = d + scale * q.abs().sum(1, keepdim=True) * 2.0 ** -25 * deq + 2.0 ** -22 * (size + top.abs()) + 2.0 ** -21
    move = w * (torch.expm1(d) + 2.0 ** -11) + 2.0 ** -28 * (~hidden) / torch.exp(x - top).sum(1, keepdim=True)
    av = vals.abs()
    bound = (move @ av + o.abs() * (w * torch.expm1(d)).sum(1, keepdim=True) + w @ ((2.0 ** -11 * av + 2.0 ** -25) * deq[:, None])
             + (64 + (past + n) / 16) * 2.0 ** -23 * (w @ av) + 2.0 ** -11 * o.abs() + 2.0 ** -25)
    return o, bound


def check(run, seqs, lens, data, cap, scale=0.0, window=0, slopes=None):
    q, k, v = data
    out = run.attend(seqs, lens, data, scale=scale, cap=cap, window=window, slopes=slopes, check=False)
    assert torch.isfinite(out).all()
    first, rep = 0, run.Hq // run.Hkv
    for s, n in zip(seqs, lens):
        oc, part = run.live[s], slice(first, first + n)
        kc, vc = torch.from_numpy(oc.keys_hat()[0]).cuda(), torch.from_numpy(oc.values_hat()[0]).cuda()
        for h in range(run.Hq):
            keys = torch.cat([kc[h // rep], k[part, h // rep].double()])
            vals = torch.cat([vc[h // rep], v[part, h // rep].double()])
            ref, most = reference(keys, vals, oc.n_quant, q[part, h].double(), oc.n_quant + oc.n_resid,
                                  scale or run.D ** -0.5, cap, window, float(slopes[h]) if slopes is not None else 0.0)
            over = ((out[part, h].double() - ref).abs() / most).max().item()
            assert over <= 1.0, f"cap {cap}, sequence {s}, head {h}: {over:.2f} of the bound"
        first += n
    return out


# (as the kernel's argument, a float)
CAPS = [1e-44, 1e-38, 1e-3, 0.25, 4.0, 30.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e8, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("cap", [torch.tensor(c).item() for c in CAPS])
@pytest.mark.parametrize("D,bits,G", [(128, 2, 32), (64, 8, 64)])
def test_caps_of_every_size(cap, D, bits, G):
    run = ChunkRun(4, 2, D, bits, G, 64, max_seqs=3, seed=D)
    seqs = [run.add(L) for L in (0, 300, 5)]
    slopes = torch.tensor([0.5, 0.25, 0.0, -0.01], device="cuda")
    for lens in ([200, 70, 1], [3, 1, 260]):
        data = run.chunk(lens)
        check(run, seqs, lens, data, cap)
        check(run, seqs, lens, data, cap, window=100, slopes=slopes)
        check(run, seqs, lens, data, cap, scale=1.0)


def test_scores_of_zero_under_the_smallest_cap():
    run = ChunkRun(1, 1, 64, 2, 32, 32, max_seqs=1, seed=5)
    s = run.add(40)
    q, k, v = run.chunk([150])
    q.zero_()
    for cap in (1e-44, 1e-38, 1.0, 3e38):
        for scale in (0.0, 1e30):
            check(run, [s], [150], (q, k, v), torch.tensor(cap).item(), scale=scale)
