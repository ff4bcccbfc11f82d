"""Refusals and host-side rules of the chunk calls (no GPU: every check here comes before a launch)."""
import pytest


@pytest.fixture(scope="module")
def K():
    from bit_kivi_kv_gb300 import build
    build.build()
    from bit_kivi_kv_gb300 import kivi
    return kivi


@pytest.fixture
def h(K):
    """Empty sequences need no device: a handle over a buffer that is never touched."""
    cfg = K.make_paged_config(6, 8, 4, 64, 2, 32, 64, 16, 32)
    handle = K.kivi_paged_create(cfg, 1 << 20, K.kivi_paged_bytes(cfg))
    yield handle
    K.kivi_paged_destroy(handle)


def status(K, f, *a):
    with pytest.raises(K.KiviError) as e:
        f(*a)
    assert str(e.value)
    return e.value.status


def chunk(K, **kw):
    a = K.kivi_chunk()
    for name in "q", "k", "v", "out":
        setattr(a, name, 4096)
        getattr(a, name + "_stride")[:] = (512, 64)
    for name, x in kw.items():
        if name.endswith("_stride"):
            getattr(a, name)[:] = x
        else:
            setattr(a, name, x)
    return a


def test_workspace_size(K):
    cfg = K.make_paged_config(6, 8, 4, 64, 2, 32, 64, 16, 32)
    wide, group = 192 * (2 * 256 * 68 * 4 + 16), 4 * 4 * 64 * 2 + 4 * 4 * 65 * 68 * 4
    # (2 query heads per kv head: 16 rows are 8 tokens, 4 rows a group)
    for lens, groups in (([9], 0), ([1], 1), ([2], 1), ([3, 8], 6), ([0, 100, 5], 3), ([8] * 200, 512), ([1] + [8] * 128, 512)):
        assert K.kivi_paged_chunk_workspace_bytes(cfg, lens) == wide + groups * group
    assert K.kivi_paged_chunk_workspace_bytes(cfg, []) == 0 and K.kivi_paged_chunk_workspace_bytes(cfg, [1] * 513) == 0
    assert K.kivi_paged_chunk_workspace_bytes(K.make_paged_config(6, 8, 4, 96, 2, 32, 64, 16, 32), [1]) == 0


def test_attention_refusals(K, h):
    a, b = (K.kivi_paged_add(h, 0, 0, 0, 0) for _ in range(2))
    cfg = K.make_paged_config(6, 8, 4, 64, 2, 32, 64, 16, 32)
    ws, n = 1 << 20, K.kivi_paged_chunk_workspace_bytes(cfg, [1])
    call = lambda seqs, lens, x, w=ws, m=n: K.kivi_paged_chunk_attn(h, seqs, lens, x, w, m, 0)  # noqa: E731
    bad = K.KIVI_ERR_INVALID_ARG
    assert status(K, call, [], [], chunk(K)) == bad
    assert status(K, call, [a] * 513, [1] * 513, chunk(K)) == bad
    assert status(K, call, [a, a], [1, 1], chunk(K)) == bad                    # listed twice
    assert status(K, call, [a, 5], [1, 1], chunk(K)) == bad                    # not live
    assert status(K, call, [a, -1], [1, 1], chunk(K)) == bad
    assert status(K, call, [a, b], [1, -1], chunk(K)) == bad
    assert status(K, call, [a, b], [1 << 30, 1 << 30], chunk(K)) == K.KIVI_ERR_UNSUPPORTED
    assert status(K, call, [a, b], [1, 1], chunk(K, softmax_scale=float("nan"))) == bad
    for cap in (-1.0, float("inf"), float("nan")):
        assert status(K, call, [a], [1], chunk(K, cap=cap)) == bad
    assert status(K, call, [a], [1], chunk(K, window=-1)) == bad
    assert status(K, call, [a], [1], chunk(K, slopes=4098)) == bad
    for name in "q", "k", "v", "out":
        assert status(K, call, [a], [1], chunk(K, **{name: None})) == bad
        assert status(K, call, [a], [1], chunk(K, **{name: 4104})) == bad
        assert status(K, call, [a], [1], chunk(K, **{name + "_stride": (512, 68)})) == bad
    assert status(K, call, [a], [1], chunk(K), ws + 8) == bad
    assert status(K, call, [a], [1], chunk(K), 0) == bad
    assert status(K, call, [a], [1], chunk(K), ws, n - 1) == K.KIVI_ERR_CAPACITY
    before = K.kivi_launch_count()
    call([a, b], [0, 0], chunk(K, q=None))                                     # nothing to do
    assert K.kivi_launch_count() == before


def test_append_refusals(K, h):
    a, b = (K.kivi_paged_add(h, 0, 0, 0, 0) for _ in range(2))
    call = lambda seqs, lens, k=4096, v=4096, ks=(256, 64), vs=(256, 64): K.kivi_paged_append_chunk(  # noqa: E731
        h, seqs, lens, k, ks, v, vs, 0)
    bad = K.KIVI_ERR_INVALID_ARG
    assert status(K, call, [a, a], [1, 1]) == bad
    assert status(K, call, [a], [-1]) == bad
    assert status(K, call, [a], [1], 0) == bad
    assert status(K, call, [a], [1], 4096, 4100) == bad
    assert status(K, call, [a], [1], 4096, 4096, (256, 60)) == bad
    # 16 blocks of 32 tokens and 64 of residual are the most of a sequence; 32 pages the pool's
    assert status(K, call, [a], [16 * 32 + 65]) == K.KIVI_ERR_CAPACITY
    c = K.kivi_paged_add(h, 0, 0, 0, 0)
    assert status(K, call, [a, b, c], [400 + 64] * 3) == K.KIVI_ERR_CAPACITY
    call([a, b], [0, 0])
    assert K.kivi_paged_seq_counts(h, a) == (0, 0) and K.kivi_paged_free(h) == (32, 3)


def test_branches_of_empty_sequences_and_truncation(K, h):
    a = K.kivi_paged_add(h, 0, 0, 0, 0)
    f = K.kivi_paged_fork(h, [a, a], 0)
    assert len(set(f) | {a}) == 3 and K.kivi_paged_free(h) == (32, 3)
    bad = K.KIVI_ERR_INVALID_ARG
    assert status(K, K.kivi_paged_fork, h, [a] * 4, 0) == K.KIVI_ERR_CAPACITY
    assert status(K, K.kivi_paged_fork, h, [], 0) == bad
    assert status(K, K.kivi_paged_fork, h, [a, 5], 0) == bad
    assert K.kivi_paged_free(h) == (32, 3)
    K.kivi_paged_truncate(h, a, 0)
    assert status(K, K.kivi_paged_truncate, h, a, 1) == bad
    assert status(K, K.kivi_paged_truncate, h, a, -1) == bad
    assert status(K, K.kivi_paged_truncate, h, 5, 0) == bad
    for s in f:
        K.kivi_paged_release(h, s)
    assert K.kivi_paged_free(h) == (32, 5)


def test_read_refusals(K, h):
    a = K.kivi_paged_add(h, 0, 0, 0, 0)
    bad = K.KIVI_ERR_INVALID_ARG
    call = lambda seqs, first, count, k=4096, v=4096: K.kivi_paged_read(h, seqs, first, count, k, v, 0)  # noqa: E731
    assert status(K, call, [a], 0, 1) == bad
    assert status(K, call, [a], -1, 0) == bad
    assert status(K, call, [a], 0, -1) == bad
    assert status(K, call, [], 0, 0) == bad
    assert status(K, call, [5], 0, 0) == bad
    call([a, a], 0, 0, 0, 0)
