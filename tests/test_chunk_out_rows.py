"""Outputs of chunk attention whose rows overlap are refused (no GPU: the check comes before a launch)."""
import itertools
import random

import pytest

from test_chunk_abi import K, chunk, h, status  # noqa: F401 - fixtures


def overlap(st, sh, tokens, heads, D):
    """By listing the elements."""
    seen = set()
    for t, g in itertools.product(range(tokens), range(heads)):
        row = range(t * st + g * sh, t * st + g * sh + D)
        if not seen.isdisjoint(row):
            return True
        seen.update(row)
    return False


def cases():
    """(token stride, head stride, tokens) of eight heads of 64."""
    fixed = [(512, 64, 3), (64, 192, 3), (0, 64, 2), (0, 64, 1), (512, 0, 2), (448, 64, 2), (504, 64, 2), (-512, 64, 3),
             (512, -64, 3), (64, 64, 2), (56, 512, 2), (64, 128, 2), (64, 128, 3), (64, 120, 2), (128, 64, 2), (192, 128, 4),
             (1024, 128, 5), (960, 128, 5), (968, 128, 2), (320, 128, 2), (320, 128, 9)]
    rng = random.Random(3)
    return fixed + [(8 * rng.randint(-80, 80), 8 * rng.randint(-80, 80), rng.randint(1, 12)) for _ in range(300)]


def test_overlapping_rows_of_out(K, h):  # noqa: F811
    a = K.kivi_paged_add(h, 0, 0, 0, 0)
    cfg = K.make_paged_config(6, 8, 4, 64, 2, 32, 64, 16, 32)
    found = set()
    for st, sh, tokens in cases():
        x = chunk(K, out_stride=(st, sh))
        need = K.kivi_paged_chunk_workspace_bytes(cfg, [tokens])
        # (one byte of workspace short: a call that passes the check of its rows fails there, before any launch)
        got = status(K, K.kivi_paged_chunk_attn, h, [a], [tokens], x, 1 << 20, need - 1, 0)
        want = overlap(st, sh, tokens, 8, 64)
        assert got == (K.KIVI_ERR_INVALID_ARG if want else K.KIVI_ERR_CAPACITY), (st, sh, tokens)
        found.add(want)
    assert found == {False, True}


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_inputs_may_repeat(K, h, name):  # noqa: F811
    """The same row for all tokens or heads is an input like any other."""
    a = K.kivi_paged_add(h, 0, 0, 0, 0)
    cfg = K.make_paged_config(6, 8, 4, 64, 2, 32, 64, 16, 32)
    for strides in ((0, 64), (512, 0), (0, 0)):
        x = chunk(K, **{name + "_stride": strides})
        need = K.kivi_paged_chunk_workspace_bytes(cfg, [3])
        assert status(K, K.kivi_paged_chunk_attn, h, [a], [3], x, 1 << 20, need - 1, 0) == K.KIVI_ERR_CAPACITY
