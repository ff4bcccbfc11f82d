"""Calls that follow each other on a stream with nothing between them: what one writes, the next one reads."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300.kivi import KiviPagedCache, kivi_launch_count  # noqa: E402


def rows(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").half()


@pytest.mark.parametrize("Hq,Hkv,D,L", [(4, 4, 128, 500), (8, 2, 64, 3000), (32, 32, 128, 4000)])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_right_after_fork(Hq, Hkv, D, L, captured):
    """The branch's slot still holds the block table of a released sequence, whose pages are valid and hold other tokens:
    the first call on the branch reads the new table."""
    G, R = 32, 64
    g = torch.Generator(device="cuda").manual_seed(L)
    blocks = (L + G - 1) // G
    c = KiviPagedCache(2, Hq, Hkv, D, 2, G, R, blocks + 4, 2 * blocks + 8)
    s = c.add(rows(g, Hkv, L, D), rows(g, Hkv, L, D))
    other = rows(g, Hkv, L + 2 * G, D), rows(g, Hkv, L + 2 * G, D)
    q, k, v = rows(g, 1, Hq, D), rows(g, 1, Hkv, D), rows(g, 1, Hkv, D)

    def decode(x):
        return c.append_decode([x], None, None, q)

    def chunk(x):
        return c.chunk_attn([x], [1], q, k, v)

    for call in (decode, chunk):
        ref = call(s).clone()
        for _ in range(10):
            t = c.add(*other)
            assert not torch.equal(call(t), ref)
            c.release(t)
            if captured:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    b = c.fork([s])
                    out = call(b[0])
                graph.replay()
            else:
                b = c.fork([s])
                out = call(b[0])
            assert b == [t]
            assert torch.equal(out, ref)
            c.release(t)


def test_the_last_kernel_of_a_fork_writes_no_table():
    """Table entries and residual rows are two launches; branches without a block need the second one alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    c = KiviPagedCache(4, 2, 2, 64, 4, 32, 32, 8, 16)
    for L, launches in ((100, 2), (20, 1)):
        s = c.add(rows(g, 2, L, 64), rows(g, 2, L, 64))
        before = kivi_launch_count()
        b = c.fork([s])
        assert kivi_launch_count() - before == launches
        for x, y in zip(c.read(b, 0, L), c.read([s], 0, L)):
            assert torch.equal(x, y)
        c.release(b[0])
        c.release(s)
