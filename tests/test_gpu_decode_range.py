"""Decode calls over the whole range that fp16 inputs have: small and large values, small
queries against large keys and the other way round, scales that change along the context.
Every decode path of the tensor-core kernels, against fp64 with bounds that follow the scales."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300 import kivi as K  # noqa: E402
from bit_kivi_kv_gb300.kivi import KiviCache, KiviPagedCache  # noqa: E402
from decode_bounds import Slot, close  # noqa: E402
from oracle.cache import OracleCache, OracleCacheFifo  # noqa: E402

PATHS = ("blocks", "dense", "fused", "queue", "paged blocks", "paged")


def inputs(Hkv, nq, D, L, seed, qs=1.0, ks=1.0, vs=1.0, sink=8.0):
    """q [Hkv nq][D], k, v [Hkv][L][D] (fp16) and a softmax scale: logits around N(0, 1), token 0's around `sink`."""
    g = np.random.default_rng(seed)
    k = g.standard_normal((Hkv, L, D))
    u = g.standard_normal((Hkv, 1, D))
    u /= np.linalg.norm(u, axis=-1, keepdims=True)
    k[:, 0] = np.sqrt(D) * u[:, 0]
    q = g.standard_normal((Hkv, nq, D)) + sink * u
    v = g.standard_normal((Hkv, L, D))
    half = lambda x: np.clip(x, -6e4, 6e4).astype(np.float16)  # noqa: E731
    return (half(q * qs).reshape(Hkv * nq, D), half(k * ks), half(v * np.asarray(vs).reshape(-1, 1)),
            1.0 / (qs * ks * np.sqrt(D)))


def run(path, q, k, v, scale, bits, G, R):
    """The path's output [Hq][D] for the prompt k, v (its last token appended where the path appends)."""
    (Hkv, L, D), Hq = k.shape, q.shape[0]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    qt, kt, vt = dev(q)[None], dev(k)[None], dev(v)[None]
    last = path in ("fused", "paged", "queue")
    n = L - 1 if last else L
    kp, vp = kt[:, :, :n].contiguous(), vt[:, :, :n].contiguous()
    k1, v1 = (t[:, :, n].contiguous() for t in (kt, vt)) if last else (None, None)
    if path.startswith("paged"):
        cache = KiviPagedCache(1, Hq, Hkv, D, bits, G, R, L // G + 2, L // G + 2)
        s = cache.add(kp[0], vp[0])
        if path == "paged":
            return cache.append_decode([s], k1, v1, qt, softmax_scale=scale)[0].cpu().numpy()
        nb = cache.counts(s)[0] // G
        blocks = torch.arange(nb, dtype=torch.int32, device="cuda").expand(1, Hkv, nb).contiguous()
        return cache.decode_blocks([s], qt, blocks, softmax_scale=scale)[0].cpu().numpy()
    cache = KiviCache(1, Hq, Hkv, D, bits, G, R, L + 1)
    if path == "queue":
        cache.set_value_residual(K.KIVI_VALUE_QUEUE)
    cache.prefill(kp, vp)
    if last:
        return cache.append_decode(k1, v1, qt, softmax_scale=scale)[0].cpu().numpy()
    if path == "dense":
        return cache.decode_attn(qt, softmax_scale=scale)[0].cpu().numpy()
    nb = cache.counts()[0] // G
    blocks = torch.arange(nb, dtype=torch.int32, device="cuda").expand(1, Hkv, nb).contiguous()
    return cache.decode_blocks(qt, blocks, softmax_scale=scale)[0].cpu().numpy()


def check(path, q, k, v, scale, bits, G, R):
    got = run(path, q, k, v, scale, bits, G, R)
    (Hkv, L, D), nq = k.shape, q.shape[0] // k.shape[0]
    last = path in ("fused", "paged", "queue")
    worst = 0.0
    for h in range(Hkv):
        oc = (OracleCacheFifo if path == "queue" else OracleCache)(1, 1, D, bits, G, R)
        n = L - 1 if last else L
        oc.prefill(k[None, h:h + 1, :n], v[None, h:h + 1, :n])
        if last:
            oc.append(k[None, h:h + 1, n], v[None, h:h + 1, n])
        slot = Slot(oc, bits)
        ref, bound = slot.decode(q[h * nq:(h + 1) * nq], slot.tokens(), scale)
        worst = max(worst, close(got[h * nq:(h + 1) * nq], ref, bound, f"{path}, kv head {h}"))
    return worst


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("D,bits,nq,G", [(64, 2, 1, 32), (128, 2, 1, 32), (128, 2, 4, 128), (128, 4, 1, 64),
                                         (128, 4, 4, 32), (64, 8, 2, 64), (128, 8, 1, 32), (128, 8, 4, 128)])
def test_value_scales(path, D, bits, nq, G):
    """Values from fp16's subnormal numbers up to its largest, a sink in front of the others."""
    for vs in (1e-5, 1e-4, 1e-3, 1e-2, 0.1, 1.0, 30.0, 1e3, 1e4):
        q, k, v, scale = inputs(2, nq, D, 900, int(D + bits + nq), vs=vs)
        check(path, q, k, v, scale, bits, G, 128)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bits,G", [(2, 32), (4, 64), (8, 128)])
def test_value_scales_that_change_along_the_context(path, bits, G):
    """The range that the probabilities are held in goes down when larger steps come."""
    L, D = 1100, 128
    t = np.arange(L) / L
    for vs in (10 ** (-3 + 7 * t), 10 ** (4 - 7 * t), np.where(t < 0.5, 1e-3, 1e3), np.where(np.arange(L) % 97 == 5, 2e4, 1e-2)):
        q, k, v, scale = inputs(1, 2, D, L, bits, vs=vs, sink=2.0)
        check(path, q, k, v, scale, bits, G, 128)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("D,bits,nq,G", [(64, 2, 2, 32), (128, 2, 1, 32), (128, 4, 4, 64), (64, 4, 1, 32), (128, 8, 1, 128),
                                         (128, 2, 4, 64)])
def test_query_and_key_scales(path, D, bits, nq, G):
    """Small queries against large keys, large ones against small keys, and a softmax scale
    that makes up for both being small or large."""
    for qs, ks in ((0.1, 100), (1e-2, 1e3), (1e-3, 5e3), (100, 1e-2), (3e3, 1e-3), (1e-3, 1e-3), (1e3, 1e3)):
        q, k, v, scale = inputs(2, nq, D, 700, int(D + bits + nq), qs=qs, ks=ks)
        check(path, q, k, v, scale, bits, G, 128)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bits,G", [(2, 32), (4, 64), (8, 128)])
def test_key_scales_that_change_along_the_context(path, bits, G):
    """Blocks whose key steps pass the limit among blocks of small ones, heads of very different
    queries, and a few channels that are larger by far."""
    L, D, nq = 1100, 128, 4
    g = np.random.default_rng(bits)
    q, k, v, _ = inputs(1, nq, D, L, bits, sink=2.0)
    t = np.arange(L)
    qh = (q.astype(np.float64) * np.array([1e-3, 0.03, 1.0, 20.0])[:, None]).astype(np.float16)
    wide = k.astype(np.float64)
    wide[:, :, g.permutation(D)[:3]] *= np.array([1e4, 500.0, 60.0])
    for kk, scale in ((k.astype(np.float64) * 10.0 ** (-2 + 5 * t / L)[:, None], 1e-3),
                      (k.astype(np.float64) * np.where(t % 260 < 40, 5e3, 0.1)[:, None], 3e-4),
                      (np.clip(wide, -6e4, 6e4), 1e-3)):
        check(path, qh, kk.astype(np.float16), v, scale, bits, G, 128)


@pytest.mark.parametrize("path", PATHS)
def test_queries_at_the_ends_of_the_range(path):
    """A zero head, one of fp16's smallest numbers, one of its largest, beside an ordinary one."""
    q, k, v, scale = inputs(1, 4, 128, 500, 3)
    q = q.astype(np.float64)
    q[0] = 0.0
    q[1] = np.sign(q[1]) * 2.0 ** -24
    q[2] *= 1e4 / np.abs(q[2]).max()
    for s in (scale, 1e-30, 1e-38):
        check(path, q.astype(np.float16), k, v, s, 4, 32, 64)
