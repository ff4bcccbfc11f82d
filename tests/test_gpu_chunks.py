"""Chunks of new tokens over the paged cache on the GPU: attention against an fp64
reference over the oracle's exact values (bounds derived in chunk_harness.py), the
cache's bytes after appends, branches and truncations against the oracle's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300.kivi import (KiviError, KiviPagedCache, QKNormRope, kivi_paged_set_max_ctas,  # noqa: E402
                                    rope_table)
from chunk_harness import ChunkRun, head_strided, in_wider, oracle_chunk  # noqa: E402
from oracle.cache import OracleCache  # noqa: E402


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


INSTANCES = [(D, bits, G, nq) for D in (128, 64) for bits in (2, 4, 8) for G, nq in ((32, 1), (64, 2), (D, 4))]


@pytest.mark.parametrize("D,bits,G,nq", INSTANCES)
def test_every_instance(D, bits, G, nq):
    run = ChunkRun(2 * nq, 2, D, bits, G, G * (2 if G < 128 else 1), seed=D + bits + G + nq)
    seqs = [run.add(L) for L in (700, 0, 3 * G + 5)]
    run.attend(seqs, [5, 70, 33])
    run.attend(seqs, [300, 1, 130], cap=20.0, slopes=slopes_of(2 * nq), window=200)


@pytest.mark.parametrize("past", [0, 1, 31, 127, 128, 129, 255, 512, 1000])
@pytest.mark.parametrize("n", [1, 2, 16, 64, 127, 128, 129, 255, 256, 257, 400])
def test_lengths(past, n):
    run = ChunkRun(2, 1, 128, 2, 32, 64, max_seqs=2, seed=past * 1000 + n)
    run.attend([run.add(past)], [n])


@pytest.mark.parametrize("nq,lens", [(1, [1, 2, 3, 4, 5, 16, 17]), (2, [1, 2, 3, 8, 9, 0, 4]), (4, [1, 2, 4, 5, 1, 3, 1])])
@pytest.mark.parametrize("D,bits", [(128, 2), (64, 8), (128, 4)])
def test_few_rows(nq, lens, D, bits):
    """Sequences of 16 rows at most go to the single-token decode kernel in groups, others beside them do not."""
    run = ChunkRun(2 * nq, 2, D, bits, 64, 128, max_seqs=7, n_pages=400, seed=nq + D)
    seqs = [run.add(L) for L in (1, 130, 700, 64, 3000, 400, 0)]
    data = run.chunk(lens)
    a = run.attend(seqs, lens, data)
    run.attend(seqs, lens, data, fit=in_wider)
    assert torch.equal(a, run.attend(seqs, lens, data, window=5000))      # (cuts nothing)
    run.attend(seqs, lens, data, window=300)
    run.attend(seqs, lens, data, cap=20.0, scale=0.2)
    ones = [1] * 7
    data = run.chunk(ones)
    run.attend(seqs[:6], ones[:6], tuple(x[:6].contiguous() for x in data))      # single tokens: read where they lie
    run.attend(seqs[:6], ones[:6], tuple(x[:6].contiguous() for x in data), fit=head_strided)


@pytest.mark.parametrize("window", [1, 2, 31, 128, 129, 300, 5000])
@pytest.mark.parametrize("nq", [1, 4])
def test_windows(window, nq):
    run = ChunkRun(nq, 1, 64, 4, 64, 64, max_seqs=3, seed=window)
    seqs = [run.add(L) for L in (0, 500, 1500)]
    run.attend(seqs, [300, 7, 513], window=window)


@pytest.mark.parametrize("cap,bias,scale", [(0.5, False, 0.0), (50.0, False, 0.3), (0.0, True, 0.0), (8.0, True, 0.02)])
def test_caps_and_biases(cap, bias, scale):
    run = ChunkRun(8, 4, 128, 2, 32, 128, max_seqs=3, seed=17)
    seqs = [run.add(L) for L in (333, 900)]
    run.attend(seqs, [40, 260], cap=cap, slopes=slopes_of(8) if bias else None, scale=scale)


@pytest.mark.parametrize("fit", [head_strided, in_wider])
def test_strides(fit):
    run = ChunkRun(8, 2, 128, 4, 128, 128, seed=5)
    seqs = [run.add(L) for L in (300, 10)]
    data = run.chunk([150, 3])
    a = run.attend(seqs, [150, 3], data)
    assert torch.equal(a, run.attend(seqs, [150, 3], data, fit=fit))
    run.append(seqs, [150, 3], data, fit=fit)
    run.check()


def test_many_sequences_of_mixed_lengths():
    """More items than CTAs and fewer rows than a tile, sequences without a cached token, lengths of zero."""
    run = ChunkRun(16, 16, 64, 2, 32, 32, max_seqs=40, n_pages=400, seed=9)
    lens = [(0, 1, 3, 200, 1, 17)[i % 6] for i in range(40)]
    seqs = [run.add((0, 90, 33, 250, 400, 64)[(i * 7) % 6]) for i in range(40)]
    order = [seqs[(i * 11) % 40] for i in range(40)]
    run.attend(order, lens)
    run.append(order, lens)
    run.attend(order, lens)
    run.check()


def test_one_long_sequence_over_all_ctas():
    run = ChunkRun(1, 1, 128, 2, 32, 128, max_seqs=1, max_blocks=1100, n_pages=1100, seed=3)
    s = run.add(33000)
    run.attend([s], [1])
    run.attend([s], [130])
    run.attend([s], [300])


@pytest.mark.parametrize("D,bits,G,R", [(128, 2, 32, 128), (64, 8, 64, 64), (128, 4, 128, 256), (64, 4, 32, 96)])
def test_a_prompt_in_pieces(D, bits, G, R):
    """Pieces of every size give the bytes of the whole prompt, and attention as it goes."""
    run = ChunkRun(4, 2, D, bits, G, R, max_seqs=4, seed=D + bits)
    a, b = run.add(0), run.add(0)
    whole = OracleCache(1, 2, D, bits, G, R)
    parts = []
    for n in (1, 30, G, 2, R, R + G + 7, 3, 500, 1, 1):
        data = run.chunk([n, 2])
        run.attend([a, b], [n, 2], data)
        run.append([a, b], [n, 2], data)
        run.check()
        parts.append([x[:n].transpose(0, 1).cpu().numpy() for x in data[1:]])
    import numpy as np
    whole.prefill(*(np.concatenate([p[j] for p in parts], axis=1)[None] for j in (0, 1)))
    oc = run.live[a]
    assert np.array_equal(oc.k_codes, whole.k_codes) and np.array_equal(oc.v_codes, whole.v_codes)
    assert np.array_equal(oc.k_res, whole.k_res)


def test_branches_share_pages_and_part():
    run = ChunkRun(4, 2, 128, 2, 32, 64, max_seqs=8, max_blocks=64, n_pages=40, seed=4)
    a = run.add(500)
    pages, _ = run.cache.free()
    f = run.fork([a, a, a])
    assert run.cache.free()[0] == pages and all(run.cache.pages(x) == run.cache.pages(a) for x in f)
    run.check()
    run.append([f[0], a], [100, 3])                 # each goes on by itself
    run.append([f[1]], [1])
    run.check()
    run.attend([f[0], f[1], a, f[2]], [3, 4, 200, 5])
    run.release(a)                                  # the pages stay with the branches
    run.check()
    g = run.fork([f[0]])[0]
    run.truncate(f[0], 480)
    run.truncate(g, 64)
    run.append([f[0], g], [50, 60])
    run.check()
    run.attend([f[0], g], [7, 129])
    for s in list(run.live):
        run.release(s)
    assert run.cache.free() == (40, 8)


def test_truncate_then_go_on():
    run = ChunkRun(2, 1, 64, 4, 32, 64, seed=6)
    s = run.add(300)
    n_quant, n_resid = run.cache.counts(s)
    run.truncate(s, n_quant + n_resid - 5)
    run.check()
    with pytest.raises(KiviError):
        run.cache.truncate(s, n_quant - 1)
    with pytest.raises(KiviError):
        run.cache.truncate(s, 1000)
    run.truncate(s, n_quant - 32)
    run.append([s], [130])
    run.check()
    run.truncate(s, 0)
    run.append([s], [7])
    run.check()
    run.attend([s], [9])


def test_single_token_calls_and_chunks_mix():
    """append_decode and append of the paged cache between chunk calls: its flushes of R tokens and theirs of G."""
    run = ChunkRun(4, 2, 128, 2, 32, 64, max_seqs=3, max_blocks=64, n_pages=100, seed=8)
    seqs = [run.add(L) for L in (63, 200)]
    for step in range(5):
        for _ in range(70 if step == 1 else 3):
            _, k, v = run.chunk([1, 1])
            run.cache.append(seqs, k, v)
            for i, s in enumerate(seqs):
                run.live[s].append(k[i].cpu().numpy()[None], v[i].cpu().numpy()[None])
        run.check()
        run.attend(seqs, [2 + step, 40])
        run.append(seqs, [33, 1 + step])
        run.check()
        q, k, v = run.chunk([1, 1])
        one = run.attend(seqs, [1, 1], (q, k, v))
        run.cache.append(seqs, k, v)
        for i, s in enumerate(seqs):
            run.live[s].append(k[i].cpu().numpy()[None], v[i].cpu().numpy()[None])
        torch.cuda.synchronize()
        if all(run.cache.counts(s)[1] > 1 for s in seqs):      # (no flush between: the same tokens)
            dec = run.cache.append_decode(seqs, None, None, q)
            assert (one.double() - dec.double()).abs().max() < 2e-2


@pytest.mark.parametrize("D,bits,G", [(128, 2, 32), (128, 4, 64), (128, 8, 128), (64, 2, 64), (64, 4, 32), (64, 8, 32)])
def test_read(D, bits, G):
    run = ChunkRun(3, 3, D, bits, G, 2 * G, max_seqs=4, seed=bits)
    seqs = [run.add(L) for L in (700, 777, 500)]
    for first, count in ((0, 500), (0, 1), (13, 400), (499, 1), (100, 0), (500 - 2 * G - 3, 2 * G), (17, 16)):
        Kr, Vr = run.cache.read(seqs, first, count)
        torch.cuda.synchronize()
        for i, s in enumerate(seqs):
            for got, hat in ((Kr[i], run.live[s].keys_hat()), (Vr[i], run.live[s].values_hat())):
                # fp16(code * step + zero), rounded once: equal bit for bit
                want = torch.from_numpy(hat[0][:, first:first + count]).half().cuda()
                assert torch.equal(got, want), (first, count, s)
    assert torch.equal(run.cache.read([seqs[1]] * 2, 600, 177)[0][1], run.cache.read([seqs[1]], 600, 177)[0][0])


def test_values_that_are_not_finite_reach_only_those_that_see_them():
    run = ChunkRun(2, 1, 128, 2, 32, 64, seed=2)
    s = run.add(250)
    q, k, v = run.chunk([300])
    clean = run.attend([s], [300], (q, k, v))
    for t, value in ((120, float("inf")), (299, float("nan")), (7, float("-inf"))):
        for x in (k, v):
            bad = x.clone()
            bad[t, 0, 5] = value
            out = run.attend([s], [300], (q, bad, v) if x is k else (q, k, bad), check=False)
            assert torch.equal(out[:t], clean[:t]), (t, value)
            assert torch.isnan(out[t:]).any(-1).all() or x is k
    for n in (3, 8):                                            # few rows: the other kernels
        few = [x[:n].contiguous() for x in (q, k, v)]
        clean_few = run.attend([s], [n], tuple(few))
        for x in (1, 2):
            bad = [y.clone() for y in few]
            bad[x][n - 2, 0, 7] = float("inf")
            out = run.attend([s], [n], tuple(bad), check=False)
            assert torch.equal(out[:n - 2], clean_few[:n - 2])
            assert x == 1 or not torch.isfinite(out[n - 2:]).all(-1).any()
    bad = q.clone()
    bad[9, 1] = float("nan")
    out = run.attend([s], [300], (bad, k, v), check=False)
    keep = torch.ones(300, 2, dtype=torch.bool, device="cuda")
    keep[9, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[9, 1]).all()


@pytest.mark.parametrize("cached", [0, 3])
@pytest.mark.parametrize("jump", [12, 17, 24, 25, 26, 29, 33, 40])
def test_logits_that_jump_within_a_tile(jump, cached):
    """Weights of up to 2^9 times the reference, then in the same tile one that raises it by 2^jump."""
    run = ChunkRun(1, 1, 64, 2, 32, 32, max_seqs=1, seed=jump)
    s = run.add(cached)
    q, k, v = run.chunk([300])
    q.zero_()
    k.zero_()
    q[:, :, 0] = 1.0
    k[150, 0, 0], k[200, 0, 0] = 9.0, float(jump)              # base-2 logits: scale ln 2
    v[150], v[200] = 60000.0, 0.0
    run.attend([s], [300], (q, k, v), scale=0.6931471805599453)


@pytest.mark.parametrize("D,bits,G", [(128, 2, 32), (64, 4, 64), (128, 8, 128), (128, 4, 32), (64, 2, 32)])
def test_numbers_up_to_the_largest_fp16(D, bits, G):
    """Blocks that reach from -65504 to 65504: a step's rounding takes some numbers beyond fp16's range."""
    run = ChunkRun(4, 2, D, bits, G, G, max_seqs=2, seed=D + bits + G)
    g = torch.Generator(device="cuda").manual_seed(7)

    def wide(*shape):
        x = (30000 * torch.randn(*shape, generator=g, device="cuda")).clamp(-65504, 65504)
        ends = torch.rand(*shape, generator=g, device="cuda")
        return torch.where(ends < 0.05, -65504.0, torch.where(ends > 0.95, 65504.0, x)).half()

    s = run.add(700, (wide(2, 700, D), wide(2, 700, D)))
    t = run.add(300, (wide(2, 300, D), torch.full((2, 300, D), 65504.0, device="cuda").half()))
    hat = run.live[s].keys_hat()
    assert hat.max() >= 65520 and torch.isinf(torch.from_numpy(hat).half()).any()
    for n in (1, 70, 300):
        q = torch.randn(n + 5, 4, D, generator=g, device="cuda").half()
        v = torch.cat([wide(n, 2, D), torch.full((5, 2, D), 65504.0, device="cuda").half()])
        run.attend([s, t], [n, 5], (q, wide(n + 5, 2, D), v), scale=2.0 ** -17, deq_step=2.0 ** -10)
        run.attend([t, s], [n, 5], (q, wide(n + 5, 2, D), v), scale=2.0 ** -17, window=250, deq_step=2.0 ** -10)


@pytest.mark.parametrize("bits,G,nq", [(2, 32, 1), (4, 64, 4), (8, 128, 2)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_quantized_values_that_are_not_finite_outside_the_window(bits, G, nq, value):
    run = ChunkRun(2 * nq, 2, 128, bits, G, G, max_seqs=3, seed=bits)
    K, V, _ = run.draw(1000)
    seqs = [run.cache.add(K, V)]
    for x in (K, V):
        bad = x.clone()
        bad[:, 500, 3] = value
        seqs.append(run.cache.add(bad if x is K else K, bad if x is V else V))
    data = run.chunk([300])
    # row i sees the tokens behind 1000 + i - 600
    clean, by_key, by_value = (run.attend([s], [300], data, window=600, check=False) for s in seqs)
    assert torch.isfinite(clean).all()
    # (a NaN leaves no trace in a quantized block: its extremes are taken over the numbers)
    lost_key = not torch.isfinite(run.cache.read([seqs[1]], 500, 1)[0]).all()
    lost_value = not torch.isfinite(run.cache.read([seqs[2]], 500, 1)[1]).all()
    assert lost_key == lost_value == (value == float("inf"))
    seen = by_value[:100]
    assert (torch.isnan(seen) if lost_value else torch.isfinite(seen)).all() and torch.equal(by_value[100:], clean[100:])
    block = 500 // G * G + G                                    # (a key's step is its block's)
    seen = torch.isfinite(by_key[:100])
    assert seen.all() if not lost_key else not seen.all(-1).any()
    assert torch.equal(by_key[block - 400:], clean[block - 400:])
    assert torch.isnan(run.attend([seqs[2]], [300], data, check=False)).all() == lost_value


def test_more_groups_of_few_rows_than_a_call_takes():
    """A sequence without tokens goes to the wide kernel: what it would have had of the groups is another's."""
    run = ChunkRun(2, 2, 64, 2, 32, 32, max_seqs=131, n_pages=300, seed=6)
    seqs = [run.add(0)] + [run.add(70) for _ in range(130)]
    run.attend(seqs, [1] + [16] * 128 + [3, 16])              # (four groups each: 512 in all)


def test_capped_grid():
    run = ChunkRun(8, 2, 128, 2, 32, 128, max_seqs=3, seed=12)
    seqs = [run.add(L) for L in (400, 1000, 90)]
    data = run.chunk([30, 400, 2])
    for most in (1, 3, 7, 0):
        kivi_paged_set_max_ctas(run.cache.handle, most)
        run.attend(seqs, [30, 400, 2], data)


def test_captured_few_rows_and_appends():
    """Single tokens and a few rows, captured and replayed twice on one workspace of each graph; between the replays the
    cache goes on as the calls outside the graphs leave it."""
    run = ChunkRun(8, 2, 128, 4, 64, 64, max_seqs=3, seed=13)
    c = run.cache
    seqs = [run.add(L) for L in (400, 1000, 1)]
    sets = [(lens, run.chunk(lens)) for lens in ([1, 1, 1], [2, 4, 3], [1, 40, 2])]
    refs = [run.attend(seqs, lens, data) for lens, data in sets]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in sets], []
    for graph, (lens, data) in zip(graphs, sets):
        with torch.cuda.graph(graph):
            outs.append(c.chunk_attn(seqs, lens, *data))
    side = [torch.cuda.Stream() for _ in sets]
    for _ in range(2):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for stream, graph in zip(side, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for o, ref in zip(outs, refs):
            assert torch.equal(o, ref)


def test_wrapper_streams_graphs_and_extend():
    run = ChunkRun(8, 2, 128, 2, 32, 128, max_seqs=4, seed=12)
    c = run.cache
    seqs = [run.add(L) for L in (400, 1000)]
    q, k, v = run.chunk([30, 200])
    ref = run.attend(seqs, [30, 200], (q, k, v))
    assert torch.equal(c.chunk_attn(seqs, [30, 200], q, k, v), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = c.chunk_attn(seqs, [30, 200], q, k, v, stream=side)
    b = c.chunk_attn(seqs, [30, 200], q, k, v)                  # at the same time, with scratch of its own
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    # two graphs, replayed at the same time on two streams
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(c.chunk_attn(seqs, [30, 200], q, k, v))
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    out = c.extend(seqs, [30, 200], q, k, v)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    for s, part in zip(seqs, (slice(0, 30), slice(30, 230))):
        oracle_chunk(run.live[s], k[part].transpose(0, 1).cpu().numpy(), v[part].transpose(0, 1).cpu().numpy())
    run.check()


def test_serving_run():
    """A prompt in pieces through norm + rotation, proposals on branches, the accepted ones appended, a single-token step."""
    Hq, Hkv, D = 8, 2, 64
    run = ChunkRun(Hq, Hkv, D, 4, 32, 64, max_seqs=6, seed=21)
    c = run.cache
    g = torch.Generator(device="cuda").manual_seed(3)
    prep = QKNormRope(Hq, Hkv, D, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"), rope_table(4096, D))
    s = run.add(0)

    def project(n, at):
        x = torch.randn(1, n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").half()
        q, k, v = (y.unflatten(-1, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
        q, k, v = prep(q, k, v, first_position=at)
        return tuple(y[0].transpose(0, 1) for y in (q, k, v))    # [n][heads][D] views of head-major memory

    at = 0
    for n in (300, 64, 1):
        q, k, v = project(n, at)
        out = c.extend([s], [n], q, k, v)
        torch.cuda.synchronize()
        run.check_out([s], [n], q, k, v, out)
        oracle_chunk(run.live[s], k.transpose(0, 1).cpu().numpy(), v.transpose(0, 1).cpu().numpy())
        at += n
    run.check()
    draft = run.fork([s, s])
    q, k, v = project(5, at)
    both = [torch.cat([x, x]) for x in (q, k, v)]
    out = c.chunk_attn(draft, [5, 5], *both)
    torch.cuda.synchronize()
    run.check_out(draft, [5, 5], *both, out)                    # (split over the CTAs as they come: not the same bits)
    c.append_chunk([s], [3], k[:3], v[:3])                      # three of the five are accepted
    oracle_chunk(run.live[s], k[:3].transpose(0, 1).cpu().numpy(), v[:3].transpose(0, 1).cpu().numpy())
    for d in draft:
        run.release(d)
    run.check()


def test_big_cache_offsets():
    """Pages beyond 4 GiB and a residual behind them."""
    run = ChunkRun(32, 32, 128, 8, 32, 32, max_seqs=2, max_blocks=64, n_pages=9000, seed=14)
    first = run.cache.free()[0]
    assert run.cache.layout.page_bytes * first > 2 ** 31
    held = [run.cache.add(torch.zeros(32, 32 * 64, 128, dtype=torch.half, device="cuda"),
                          torch.zeros(32, 32 * 64, 128, dtype=torch.half, device="cuda"))]
    run.cache.release(held[0])
    s = run.add(200)
    run.attend([s], [20])
    run.append([s], [70])
    run.check()


def test_wrong_device_or_shape():
    cache = KiviPagedCache(2, 4, 2, 64, 2, 32, 32, 8, 8)
    s = cache.add(*(torch.zeros(2, 10, 64, dtype=torch.half, device="cuda") for _ in range(2)))
    q, k = torch.zeros(3, 4, 64, dtype=torch.half, device="cuda"), torch.zeros(3, 2, 64, dtype=torch.half, device="cuda")
    cache.chunk_attn([s], [3], q, k, k)
    for args in (([s], [2], q, k, k), ([s], [3], q.cpu(), k, k), ([s], [3], q.float(), k, k), ([s], [3, 0], q, k, k),
                 ([s], [3], q, k, k.transpose(1, 2).contiguous().transpose(1, 2)), ([s, s], [1, 2], q, k, k),
                 ([s + 1], [3], q, k, k), ([s], [-3], q[:0], k[:0], k[:0])):
        with pytest.raises((KiviError, RuntimeError)):
            cache.chunk_attn(*args)
    with pytest.raises(KiviError):
        cache.chunk_attn([s], [3], q, k, k, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(KiviError):
        cache.append_chunk([s], [1000], torch.zeros(1000, 2, 64, dtype=torch.half, device="cuda"),
                           torch.zeros(1000, 2, 64, dtype=torch.half, device="cuda"))
    assert cache.counts(s) == (0, 10)
    cache.chunk_attn([s], [0], q[:0], k[:0], k[:0])
    cache.append_chunk([s], [0], k[:0], k[:0])
    assert cache.counts(s) == (0, 10)
