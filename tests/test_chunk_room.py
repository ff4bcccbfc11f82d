"""Room for a chunk, asked for ahead of its attention (no GPU)."""
from test_chunk_abi import K, h, status  # noqa: F401 - fixtures


def test_append_room(K, h):  # noqa: F811
    a, b, c = (K.kivi_paged_add(h, 0, 0, 0, 0) for _ in range(3))
    bad = K.KIVI_ERR_INVALID_ARG
    ask = lambda seqs, lens: K.kivi_paged_append_room(h, seqs, lens)  # noqa: E731
    before = K.kivi_launch_count()
    # 16 blocks of 32 tokens and 64 of residual are the most of a sequence; 32 pages the pool's
    ask([a, b], [16 * 32 + 64, 16 * 32 + 64])
    ask([a, b, c], [0, 5, 64])
    assert status(K, ask, [a], [16 * 32 + 65]) == K.KIVI_ERR_CAPACITY
    assert status(K, ask, [a, b, c], [400 + 64] * 3) == K.KIVI_ERR_CAPACITY
    assert status(K, ask, [a, a], [1, 1]) == bad
    assert status(K, ask, [a, 5], [1, 1]) == bad
    assert status(K, ask, [a], [-1]) == bad
    assert status(K, ask, [], []) == bad
    assert K.kivi_paged_seq_counts(h, a) == (0, 0) and K.kivi_paged_free(h) == (32, 3)
    assert K.kivi_launch_count() == before


def test_extend_asks_first(K, h, monkeypatch):  # noqa: F811
    """The attention of an extend without room is not begun."""
    import torch
    cache = object.__new__(K.KiviPagedCache)
    monkeypatch.setattr(cache, "handle", h, raising=False)        # (the fixture's to destroy)
    a = K.kivi_paged_add(h, 0, 0, 0, 0)
    monkeypatch.setattr(cache, "chunk_attn", lambda *x, **y: (_ for _ in ()).throw(AssertionError("begun")))
    x = torch.zeros(16 * 32 + 65, 4, 64, dtype=torch.half)
    assert status(K, cache.extend, [a], [16 * 32 + 65], x, x, x) == K.KIVI_ERR_CAPACITY
    assert status(K, cache.extend, [a], [1, 2], x, x, x) == K.KIVI_ERR_INVALID_ARG
