"""A list that is longer than the block decode's counters hold is refused on the host (no GPU
needed; the fake device pointers are never dereferenced)."""
from test_blocks_abi import FAKE, K, refuses  # noqa: F401  (K: the fixture)


def test_list_length_limit(K):
    cfg = K.make_config(1, 2, 2, 64, 2, 32, 32, 64)
    h = K.kivi_cache_create(cfg, FAKE, K.kivi_cache_bytes(cfg))
    try:
        refuses(K, K.KIVI_ERR_UNSUPPORTED, K.kivi_decode_blocks, h, FAKE, FAKE, (1 << 28) + 1, FAKE, 0.0, 0)
        refuses(K, K.KIVI_ERR_STATE, K.kivi_decode_blocks, h, FAKE, FAKE, 1 << 28, FAKE, 0.0, 0)   # (an empty cache)
    finally:
        K.kivi_cache_destroy(h)
