"""Appends and branches captured into a graph: the host's counts move when they are captured, the bytes when the graph runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from chunk_harness import ChunkRun, head_strided, in_wider, oracle_chunk, oracle_copy  # noqa: E402


def told(run, seqs, lens, k, v):
    first = 0
    for s, n in zip(seqs, lens):
        oracle_chunk(run.live[s], k[first:first + n].transpose(0, 1).cpu().numpy(), v[first:first + n].transpose(0, 1).cpu().numpy())
        first += n


@pytest.mark.parametrize("fit", [head_strided, in_wider])
@pytest.mark.parametrize("D,bits,G,R", [(128, 2, 32, 64), (64, 8, 64, 64), (128, 4, 128, 128)])
def test_append_of_views(fit, D, bits, G, R):
    """Chunks that complete several blocks, one and none, through views; a second graph goes on where the first ends."""
    run = ChunkRun(4, 2, D, bits, G, R, max_seqs=3, seed=D + bits)
    c = run.cache
    seqs = [run.add(L) for L in (500, R, 3)]
    graphs = []
    for lens in ([2 * G + 5, 1, 7], [3, G, 2]):
        q, k, v = run.chunk(lens)
        kv = fit(k), fit(v)                                       # (held by the list: the graph reads them)
        before = c.buffer.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.append_chunk(seqs, lens, *kv)
        torch.cuda.synchronize()
        assert torch.equal(before, c.buffer)
        told(run, seqs, lens, k, v)
        assert [c.counts(s) for s in seqs] == [(run.live[s].n_quant, run.live[s].n_resid) for s in seqs]
        graphs.append((graph, kv))
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    run.check()
    run.attend(seqs, [5, 40, 1])


def test_a_step_of_branches():
    """fork, attention, append and reading back in one graph, and the same calls outside it on another branch."""
    run = ChunkRun(4, 2, 128, 2, 32, 64, max_seqs=6, seed=8)
    c = run.cache
    s = run.add(700)
    q, k, v = run.chunk([100])
    run.fork([s])                                                 # (its slot's table is written before)
    first = list(run.live)[-1]
    run.append([first], [300])
    run.release(first)

    def step():
        b = c.fork([s])[0]
        out = c.extend([b], [100], q, k, v)
        return b, out, c.read([b], 0, 800), c.chunk_attn([b], [3], q[:3], k[:3], v[:3])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b, *captured = step()
    graph.replay()
    torch.cuda.synchronize()
    other, *eager = step()
    torch.cuda.synchronize()
    assert other != b

    def flat(x):
        return (x[0], *x[1], x[2])

    for x, y in zip(flat(captured), flat(eager)):
        assert torch.equal(x, y)
    for t in (b, other):
        run.live[t] = oracle_copy(run.live[s])
        told(run, [t], [100], k, v)
    run.check()
