"""Argument checks of the calls over chosen blocks and of the norm and rotation:
every refusal happens on the host, before anything is launched (no GPU needed;
the fake device pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest

from blocks_harness import ref_select

FAKE = 1 << 20


@pytest.fixture(scope="module")
def K():
    from bit_kivi_kv_gb300 import build
    build.build()
    from bit_kivi_kv_gb300 import kivi
    return kivi


def refuses(K, status, f, *args):
    before = K.kivi_launch_count()
    with pytest.raises(K.KiviError) as e:
        f(*args)
    assert e.value.status == status, (args, e.value)
    assert K.kivi_last_error_string()
    assert K.kivi_launch_count() == before


def test_dense_block_calls(K):
    cfg = K.make_config(1, 2, 2, 64, 2, 32, 32, 64)
    h = K.kivi_cache_create(cfg, FAKE, K.kivi_cache_bytes(cfg))
    nan, inf = float("nan"), float("inf")
    try:
        K.kivi_block_scores(h, FAKE, 0.0, 0, 0, 0)                                 # no columns: nothing to do
        for args, status in [((0, 0.0, FAKE, 4, 0), K.KIVI_ERR_INVALID_ARG), ((FAKE, 0.0, 0, 4, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE + 8, 0.0, FAKE, 4, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, 0.0, FAKE + 2, 4, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, 0.0, FAKE, -1, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, nan, FAKE, 4, 0), K.KIVI_ERR_INVALID_ARG), ((FAKE, inf, FAKE, 4, 0), K.KIVI_ERR_INVALID_ARG)]:
            refuses(K, status, K.kivi_block_scores, h, *args)
        for args, status in [((FAKE, FAKE, 1, FAKE, 0.0, 0), K.KIVI_ERR_STATE),   # empty cache
                             ((0, FAKE, 1, FAKE, 0.0, 0), K.KIVI_ERR_INVALID_ARG), ((FAKE, 0, 1, FAKE, 0.0, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, FAKE, 1, 0, 0.0, 0), K.KIVI_ERR_INVALID_ARG), ((FAKE, FAKE, -1, FAKE, 0.0, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE + 4, FAKE, 1, FAKE, 0.0, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, FAKE + 1, 1, FAKE, 0.0, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, FAKE, 1, FAKE + 8, 0.0, 0), K.KIVI_ERR_INVALID_ARG),
                             ((FAKE, FAKE, 1, FAKE, nan, 0), K.KIVI_ERR_INVALID_ARG)]:
            refuses(K, status, K.kivi_decode_blocks, h, *args)
        K.kivi_cache_set_value_residual(h, K.KIVI_VALUE_QUEUE)
        refuses(K, K.KIVI_ERR_UNSUPPORTED, K.kivi_decode_blocks, h, FAKE, FAKE, 1, FAKE, 0.0, 0)
        for f, n in ((K.kivi_block_scores, 5), (K.kivi_decode_blocks, 6)):
            refuses(K, K.KIVI_ERR_INVALID_ARG, f, None, *((FAKE, 0.0, FAKE, 4, 0) if n == 5 else (FAKE, FAKE, 1, FAKE, 0.0, 0)))
    finally:
        K.kivi_cache_destroy(h)


def test_select(K):
    f = K.kivi_select_blocks
    for args in [(FAKE, -1, 4, 4, 2, 0, FAKE, 0), (FAKE, 1, -4, 4, 2, 0, FAKE, 0), (FAKE, 1, 4, 3, 2, 0, FAKE, 0),
                 (FAKE, 1, 4, 4, -2, 0, FAKE, 0), (FAKE, 1, 4, 4, 2, 3, FAKE, 0), (FAKE, 1, 4, 4, 2, -1, FAKE, 0),
                 (0, 1, 4, 4, 2, 0, FAKE, 0), (FAKE, 1, 4, 4, 2, 0, 0, 0), (FAKE + 2, 1, 4, 4, 2, 0, FAKE, 0),
                 (FAKE, 1, 4, 4, 2, 0, FAKE + 1, 0)]:
        refuses(K, K.KIVI_ERR_INVALID_ARG, f, *args)
    refuses(K, K.KIVI_ERR_UNSUPPORTED, f, FAKE, 1 << 31, 4, 4, 2, 0, FAKE, 0)
    refuses(K, K.KIVI_ERR_UNSUPPORTED, f, FAKE, 1, (1 << 30) + 1, 1 << 31, 2, 0, FAKE, 0)
    refuses(K, K.KIVI_ERR_UNSUPPORTED, f, FAKE, 1, 4, 4, (1 << 30) + 1, 0, FAKE, 0)
    f(0, 0, 4, 4, 2, 0, 0, 0)            # no rows, nothing kept: nothing to do
    f(0, 5, 4, 4, 0, 0, 0, 0)


def test_paged_block_calls(K):
    cfg = K.make_paged_config(3, 2, 2, 64, 2, 32, 32, 4, 6)
    h = K.kivi_paged_create(cfg, FAKE, K.kivi_paged_bytes(cfg))
    many = [0] * (K.KIVI_PAGED_MAX_CALL_SEQS + 1)
    try:
        assert [K.kivi_paged_add(h, 0, 0, 0, 0) for _ in range(2)] == [0, 1]
        for seqs, status in [([], K.KIVI_ERR_INVALID_ARG), (many, K.KIVI_ERR_INVALID_ARG), ([0, 0], K.KIVI_ERR_INVALID_ARG),
                             ([2], K.KIVI_ERR_INVALID_ARG), ([-1], K.KIVI_ERR_INVALID_ARG), ([0], K.KIVI_ERR_STATE)]:
            refuses(K, status, K.kivi_paged_block_scores, h, seqs, FAKE, 0.0, FAKE, 4, 0)
            refuses(K, status, K.kivi_paged_decode_blocks, h, seqs, FAKE, FAKE, 1, FAKE, 0.0, 0)
            if status != K.KIVI_ERR_STATE:
                refuses(K, status, K.kivi_paged_append, h, seqs, FAKE, FAKE, 0)
        for args in [(0, FAKE), (FAKE, 0), (FAKE + 8, FAKE), (FAKE, FAKE + 8)]:
            refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_paged_append, h, [0, 1], *args, 0)
        refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_paged_block_scores, h, [0], 0, 0.0, FAKE, 4, 0)
        refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_paged_decode_blocks, h, [0], FAKE, 0, 1, FAKE, 0.0, 0)
        assert [K.kivi_paged_seq_counts(h, s) for s in (0, 1)] == [(0, 0)] * 2 and K.kivi_paged_free(h) == (6, 1)
    finally:
        K.kivi_paged_destroy(h)


def qkv(K, **over):
    a = K.kivi_qkv()
    a.batch, a.n_q_heads, a.n_kv_heads, a.head_dim, a.n_tokens, a.dtype = 1, 2, 2, 64, 1, K.KIVI_BF16
    a.q = a.k = a.v = a.q_out = a.k_out = a.v_out = FAKE
    for s in (a.q_stride, a.k_stride, a.v_stride):
        s[0], s[1], s[2] = 128, 128, 64
    a.cos_sin, a.n_positions, a.rot_dim, a.eps = FAKE, 8, 64, 1e-6
    for name, x in over.items():
        if name.endswith("stride"):
            getattr(a, name)[2] = x
        else:
            setattr(a, name, x)
    return a


BAD_QKV = [dict(batch=-1), dict(n_tokens=-1), dict(n_q_heads=0), dict(n_kv_heads=0), dict(dtype=7), dict(q=None, k=None, v=None),
           dict(q=FAKE + 8), dict(v=FAKE + 2), dict(q_stride=66), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(q_weight=FAKE + 4), dict(rot_dim=0), dict(rot_dim=12), dict(rot_dim=72), dict(n_positions=0), dict(cos_sin=FAKE + 4),
           dict(positions=FAKE + 4, positions_64bit=1), dict(positions=FAKE + 2)]
UNSUPPORTED_QKV = [dict(head_dim=96), dict(head_dim=256), dict(n_q_heads=8193), dict(batch=1 << 20, n_tokens=1 << 14)]


def test_norm_rope_arguments(K):
    for over in BAD_QKV + [dict(q_out=None), dict(k_out=None), dict(v_out=None), dict(q_out=FAKE + 8)]:
        refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_qk_norm_rope, qkv(K, **over), 0)
    for over in UNSUPPORTED_QKV:
        refuses(K, K.KIVI_ERR_UNSUPPORTED, K.kivi_qk_norm_rope, qkv(K, **over), 0)
    K.kivi_qk_norm_rope(qkv(K, batch=0), 0)
    K.kivi_qk_norm_rope(qkv(K, n_tokens=0, q=None, k=None, v=None), 0)
    assert K.lib.kivi_qk_norm_rope(ctypes.POINTER(K.kivi_qkv)(), None) == K.KIVI_ERR_INVALID_ARG


def test_append_qkv_arguments(K):
    cfg = K.make_config(1, 2, 2, 64, 2, 32, 32, 64)
    h = K.kivi_cache_create(cfg, FAKE, K.kivi_cache_bytes(cfg))
    try:
        for over in BAD_QKV + [dict(n_tokens=2), dict(batch=2), dict(n_q_heads=1), dict(n_kv_heads=1), dict(head_dim=128),
                               dict(k=None), dict(v=None), dict(q_out=None), dict(q_out=FAKE + 8), dict(batch=0)]:
            refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_append_qkv, h, qkv(K, **over), 0)
        refuses(K, K.KIVI_ERR_INVALID_ARG, K.kivi_append_qkv, None, qkv(K), 0)
        assert K.kivi_cache_counts(h) == (0, 0)
    finally:
        K.kivi_cache_destroy(h)


def test_reference_selection():
    """The tests' own selection: ties to the lowest index, -inf and NaN never, the first columns always."""
    inf, nan = np.inf, np.nan
    s = np.array([[1, 3, 3, 2, 3], [nan, -inf, 0, -0.0, -1], [-inf, nan, -inf, nan, -inf], [-inf, 1, 2, 3, 4]], np.float32)
    assert ref_select(s, 2, 0).tolist() == [[1, 2], [2, 3], [-1, -1], [3, 4]]
    assert ref_select(s, 3, 1).tolist() == [[0, 1, 2], [2, 3, 4], [-1, -1, -1], [2, 3, 4]]
    assert ref_select(s, 3, 2).tolist() == [[0, 1, 2], [2, 3, 4], [-1, -1, -1], [1, 3, 4]]
    assert ref_select(s, 6, 0)[0].tolist() == [0, 1, 2, 3, 4, -1]
