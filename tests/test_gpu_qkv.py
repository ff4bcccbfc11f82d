"""Norm and rotation of queries and keys on the GPU against the formula in fp64,
and the append that stores its result in the cache.

Bound: the row's mean square is a sum of 8 fused multiply-adds and 4 additions,
then a scaling, an addition, a root and a division: the norm factor is off by
fewer than 12 roundings of 2^-24 (half of the sum's, through the root), its
product with x and the weight by 2 more, a rotation by 3 more of the two
products: 20 * 2^-24 of |a| + |b| covers them.  Then one rounding to fp16: half a
step, 2^-11 of the value or 2^-25 below 2^-14."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300 import kivi as K  # noqa: E402
from bit_kivi_kv_gb300.kivi import KiviCache, QKNormRope, rope_table  # noqa: E402
from guards import Banded, GuardedCache  # noqa: E402


def reference(x, w, eps, table, pos, interleaved):
    """(y [B, H, L, D] fp64, bound) for x [B, L, H, D]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    size = x.abs()
    y = x.clone()
    if table is not None:
        rot = table.shape[1]
        cos, sin = (t[:, :, None] for t in table.double()[pos].chunk(2, -1))
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        both = x[..., a].abs() + x[..., b].abs()
        size[..., a] = both
        size[..., b] = both
    bound = 2.0 ** -11 * y.abs() + 2.0 ** -25 + 20 * 2.0 ** -24 * size
    return y.transpose(1, 2), bound.transpose(1, 2)


def check(out, x, w, eps, table, pos, interleaved, what):
    y, bound = reference(x, w, eps, table, pos, interleaved)
    d = (out.double() - y).abs()
    assert out.dtype == torch.float16 and not out.isnan().any(), what
    assert (d <= bound).all(), f"{what}: {d.max().item()} over {bound.max().item()}"


def inputs(B, L, Hq, Hkv, D, dtype, seed, packed=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if packed:
        x = (torch.randn(B, L, (Hq + 2 * Hkv) * D, generator=g, device="cuda") * 2).to(dtype)
        return tuple(t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))
    return tuple((torch.randn(B, h, L, D, generator=g, device="cuda") * 2).to(dtype).transpose(1, 2) for h in (Hq, Hkv, Hkv))


def op(Hq, Hkv, D, norm, rot, interleaved, far, seed, eps=1e-5):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    w = [torch.randn(D, generator=g, device="cuda") for _ in range(2)] if norm else [None, None]
    table = rope_table(far, rot) if rot else None
    return QKNormRope(Hq, Hkv, D, w[0], w[1], table, eps=eps, interleaved=interleaved), w, table


def run(B, L, Hq, Hkv, D, dtype, norm, rot, interleaved, seed, packed=True, far=5000, int32=False):
    q, k, v = inputs(B, L, Hq, Hkv, D, dtype, seed, packed)
    nr, w, table = op(Hq, Hkv, D, norm, rot, interleaved, far, seed)
    pos = torch.randint(0, far, (B, L), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    bands = Banded()
    out = tuple(bands.bytes(B * h * L * D * 2, "cuda").view(torch.float16).view(B, h, L, D) for h in (Hq, Hkv, Hkv))
    got = nr(q, k, v, pos.int() if int32 else pos, out=out)
    bands.check("after a norm and rotation")
    for o, x, ww, tt, what in ((got[0], q, w[0], table, "q"), (got[1], k, w[1], table, "k"), (got[2], v, None, None, "v")):
        check(o, x, ww, 1e-5, tt, pos, interleaved, what)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot", [0, 8, 24, 32, 64, "all"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_forms(dtype, D, rot, interleaved):
    rot = D if rot == "all" else rot
    run(2, 5, 6, 3, D, dtype, True, rot, interleaved, D + rot, int32=rot == 24)
    run(1, 1, 1, 1, D, dtype, False, rot, interleaved, D + rot + 1)


@pytest.mark.parametrize("B,L,Hq,Hkv,D", [(1, 1, 32, 8, 128), (1, 17, 5, 5, 64), (3, 333, 8, 2, 128), (64, 1, 40, 40, 128),
                                          (2, 2049, 32, 4, 64), (7, 129, 71, 1, 64), (1, 4099, 4, 1, 128), (4, 1000, 32, 32, 128)])
def test_sizes(B, L, Hq, Hkv, D):
    run(B, L, Hq, Hkv, D, torch.bfloat16, True, D, False, B + L)
    run(B, L, Hq, Hkv, D, torch.float16, True, D // 2, True, B + L, packed=False)


def test_strided_sources_and_wide_values():
    """Head-major sources, sources sliced out of a longer batch, and values past fp16's range."""
    B, L, H, D = 2, 9, 4, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.randn(B + 2, 2 * L, 3 * H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = big[1:1 + B, ::2, :H], big[1:1 + B, 1::2, H:2 * H], big[2:, ::2, 2 * H:]
    nr, w, table = op(H, H, D, True, D, False, 100, 3)
    got = nr(q, k, v, first_position=7)
    pos = (7 + torch.arange(L, device="cuda")).expand(B, L)
    for o, x, ww, tt in ((got[0], q, w[0], table), (got[1], k, w[1], table), (got[2], v, None, None)):
        check(o, x, ww, 1e-5, tt, pos, False, "strided")
    x = torch.full((1, 1, 2, D), 3e38, device="cuda")
    x[0, 0, 1] = 1e-30
    out = QKNormRope(2, 2, D)(x, x, x)
    assert out[2][0, 0].isinf().all() and (out[2][0, 1] == 0).all()
    zero = torch.zeros(1, 1, 2, D, device="cuda", dtype=torch.bfloat16)
    out = QKNormRope(2, 2, D, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"), eps=1e-6)(zero, zero, zero)
    assert all((o == 0).all() for o in out)


def test_more_than_2_31_values():
    """A query tensor of 2.2 billion values: 64-bit offsets on both sides."""
    B, L, Hq, Hkv, D = 17, 32768, 32, 1, 128
    nr, w, table = op(Hq, Hkv, D, True, D, False, L, 6)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty(B, L, Hq, D, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        q[b] = torch.randn(L, Hq, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(B, L, Hkv, D, generator=g, device="cuda").bfloat16()
    assert q.numel() > 1 << 31
    got = nr(q, k, k)
    at = torch.tensor([0, 1, L // 2, L - 1], device="cuda")
    for b in (0, B // 2, B - 1):
        check(got[0][b:b + 1, :, at], q[b:b + 1, at], w[0], 1e-5, table, at[None], False, f"row {b}")
        check(got[1][b:b + 1, :, at], k[b:b + 1, at], w[1], 1e-5, table, at[None], False, f"row {b}")


def test_positions_outside_the_table():
    """No table row is read for them; the rotated channels of the token's q and k become NaN."""
    B, L, H, D = 1, 6, 2, 128
    q, k, v = inputs(B, L, H, H, D, torch.float16, 5)
    table = rope_table(50, 64)
    pos = torch.tensor([[0, 49, 50, -1, 2 ** 40, 7]], device="cuda")
    nr = QKNormRope(H, H, D, cos_sin=table)
    got = nr(q, k, v, pos)
    good = [0, 1, 5]
    for o, x in ((got[0], q), (got[1], k)):
        assert o[:, :, 2:5, :64].isnan().all()
        assert torch.equal(o[:, :, 2:5, 64:], x.transpose(1, 2)[:, :, 2:5, 64:])
        check(o[:, :, good], x[:, good], None, 0, table, pos[:, good], False, "in the table")
    assert torch.equal(got[2], v.transpose(1, 2))


def test_far_positions():
    """The table's angles are exact to fp32 at any position, so far ones are as near as close ones."""
    run(2, 40, 4, 2, 64, torch.bfloat16, True, 64, False, 9, far=1 << 20)


@pytest.mark.parametrize("queue", [False, True], ids=["flush", "queue"])
@pytest.mark.parametrize("L", [0, 5, 64, 200])
def test_append_qkv_is_norm_rope_then_append(queue, L):
    """The same cache bytes, counts and queries, over flushes and queue pops."""
    B, Hq, Hkv, D, bits, G, R = 2, 4, 2, 64, 2, 32, 64
    nr, _, _ = op(Hq, Hkv, D, True, D, False, 1000, 2)
    a, b = (GuardedCache(B, Hq, Hkv, D, bits, G, R, 400) for _ in range(2))
    for c in (a, b):
        if queue:
            c.set_value_residual(K.KIVI_VALUE_QUEUE)
        c.buffer.zero_()
        q, k, v = inputs(B, L, Hq, Hkv, D, torch.bfloat16, 7)
        if L:
            pq, pk, pv = nr(q, k, v)
            c.prefill(pk, pv)
    for s in range(R + 20):
        q, k, v = (x[:, 0] for x in inputs(B, 1, Hq, Hkv, D, torch.bfloat16, 100 + s))
        pos = torch.full((B,), L + s, device="cuda", dtype=torch.int32)
        q1 = a.append_qkv(nr, q, k, v, pos, q_out=a.bands.like(torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")))
        a.bands.check(f"after step {s}")
        q2, k2, v2 = nr(q, k, v, pos)
        b.append(k2, v2)
        assert torch.equal(q1, q2)
        assert a.counts() == b.counts()
        if s % 13 == 0:
            assert torch.equal(a.decode_attn(q1), b.decode_attn(q2))
    assert torch.equal(a.buffer, b.buffer)


def test_prompt_to_sparse_decode():
    """The path of a step: projection output -> cache -> scores -> selection -> attention,
    and as a captured graph for the steps between two flushes."""
    B, Hq, Hkv, D, L = 2, 8, 4, 128, 700
    nr, _, _ = op(Hq, Hkv, D, True, D, False, 2000, 4)
    cache = KiviCache(B, Hq, Hkv, D, 4, 32, 64, 1000)
    q, k, v = inputs(B, L, Hq, Hkv, D, torch.bfloat16, 11)
    _, pk, pv = nr(q, k, v)
    cache.prefill(pk, pv)
    for s in range(5):
        q, k, v = (x[:, 0] for x in inputs(B, 1, Hq, Hkv, D, torch.bfloat16, 200 + s))
        qn = cache.append_qkv(nr, q, k, v, first_position=L + s)
        nb = cache.counts()[0] // 32
        everything = cache.sparse_decode(qn, nb)
        whole = cache.decode_attn(qn)
        assert (everything.float() - whole.float()).abs().max() <= 4e-3
    static = qn.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = cache.sparse_decode(static, 4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cache.sparse_decode(static, 4))


def test_refusals_with_tensors():
    D = 64
    q, k, v = inputs(2, 3, 4, 2, D, torch.float16, 1)
    nr = QKNormRope(4, 2, D)
    odd = torch.zeros(2, 3, 4 * D + 4, device="cuda", dtype=torch.float16)[..., 4:].unflatten(-1, (4, D))
    bad = [lambda: nr(q.double(), k.double(), v.double()), lambda: nr(q, k.bfloat16(), v), lambda: nr(q, k, v[:1]),
           lambda: nr(q[:, :, :3], k, v), lambda: nr(q.cpu(), k.cpu(), v.cpu()), lambda: nr(odd, k, v),
           lambda: nr(q, k, v, torch.zeros(2, 3, device="cuda")), lambda: nr(q, k, v, torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: nr(q, k, v, out=(torch.empty(2, 4, 3, D, device="cuda"),) * 3),
           lambda: QKNormRope(4, 2, D, q_weight=torch.ones(D, device="cuda").half()),
           lambda: QKNormRope(4, 2, D, cos_sin=rope_table(10, 20))(q, k, v),
           lambda: QKNormRope(4, 2, 96)(*inputs(2, 3, 4, 2, 96, torch.float16, 1)),
           lambda: nr(q.transpose(-1, -2), k, v)]
    for f in bad:
        with pytest.raises((K.KiviError, RuntimeError)):
            f()
    cache = KiviCache(2, 4, 2, D, 2, 32, 32, 33)
    with pytest.raises(K.KiviError):
        cache.append_qkv(nr, q, k, v)                       # three tokens
    for _ in range(33):
        cache.append_qkv(nr, q[:, 0], k[:, 0], v[:, 0])
    with pytest.raises(K.KiviError) as e:
        cache.append_qkv(nr, q[:, 0], k[:, 0], v[:, 0])
    assert e.value.status == K.KIVI_ERR_CAPACITY
    assert np.prod(nr(q[:, :0], k[:, :0], v[:, :0])[0].shape) == 0
