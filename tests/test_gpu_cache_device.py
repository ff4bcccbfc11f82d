"""Calls of a cache whose buffer is on another device than the current one are refused before any
launch (one GPU: the cache is told that its buffer is elsewhere)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300 import kivi as K  # noqa: E402
from bit_kivi_kv_gb300.kivi import KiviCache, KiviPagedCache, QKNormRope  # noqa: E402


def test_cache_on_another_device():
    B, H, D = 2, 2, 64
    rnd = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    k, v, q, q1 = rnd(B, H, 100, D), rnd(B, H, 100, D), rnd(B, H, D), rnd(1, H, D)
    lists, list1 = (torch.zeros(n, H, 1, dtype=torch.int32, device="cuda") for n in (B, 1))
    cache = KiviCache(B, H, H, D, 2, 32, 32, 200)
    cache.prefill(k, v)
    pool = KiviPagedCache(2, H, H, D, 2, 32, 32, 8, 16)
    seq = pool.add(k[0], v[0])
    op = QKNormRope(H, H, D)
    calls = [lambda: cache.append_qkv(op, q, q, q), lambda: cache.block_scores(q), lambda: cache.decode_blocks(q, lists),
             lambda: cache.sparse_decode(q, 1), lambda: pool.append([seq], q1, q1), lambda: pool.block_scores([seq], q1),
             lambda: pool.decode_blocks([seq], q1, list1), lambda: pool.sparse_decode([seq], q1, 1)]
    for c in (cache, pool):
        assert c._device == torch.cuda.current_device()
        c._device += 1
    before = K.kivi_launch_count(), cache.counts(), pool.counts(seq)
    for f in calls:
        with pytest.raises(K.KiviError) as e:
            f()
        assert e.value.status == K.KIVI_ERR_INVALID_ARG
    assert before == (K.kivi_launch_count(), cache.counts(), pool.counts(seq))
    for c in (cache, pool):
        c._device -= 1
    for f in calls:
        f()
