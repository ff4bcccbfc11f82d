"""Norm and rotation of rows whose squares leave fp32's range, beside ordinary rows, against fp64.

Bound: a square and its place in the sum meet 20 roundings of 2^-24 at most, the root, the quotient and
the products with row, weight, cosine and sine 8 more: under 2^-19 of |y_a| + |y_b| of a rotated pair
(twice the error of one), and one rounding to fp16 (2^-11 of the result, 2^-25 below 2^-14)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU hosts too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from bit_kivi_kv_gb300.kivi import QKNormRope, rope_table  # noqa: E402


def reference(x, w, table, pos, eps, interleaved):
    """(out, bound) in fp64 of x [B, L, H, D], both [B, H, L, D]."""
    x, w, t = (np.asarray(a.double().cpu()) for a in (x, w, table))
    top = np.abs(x).max(-1, keepdims=True)
    top = np.where((top > 0) & np.isfinite(top), top, 1.0)
    y = (x / top) / np.sqrt(np.mean((x / top) ** 2, -1, keepdims=True) + eps / top ** 2) * w
    rot = t.shape[1]
    c, s = t[pos, :rot // 2][..., None, :], t[pos, rot // 2:][..., None, :]       # [B, L, 1, rot / 2]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    out, size = y.copy(), np.abs(y)
    pa, pb, both = a * c - b * s, b * c + a * s, np.abs(a) + np.abs(b)
    for z, u, v in ((out, pa, pb), (size, both, both)):
        if interleaved:
            z[..., 0:rot:2], z[..., 1:rot:2] = u, v
        else:
            z[..., :rot // 2], z[..., rot // 2:rot] = u, v
    bound = 2.0 ** -11 * np.abs(out) + 2.0 ** -25 + 2.0 ** -19 * size
    return out.transpose(0, 2, 1, 3), bound.transpose(0, 2, 1, 3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_of_every_magnitude(D, interleaved, dtype):
    """One magnitude a token, from the smallest to the largest of the type, for eps from 0 up."""
    top = {torch.float32: 126, torch.bfloat16: 126, torch.float16: 14}[dtype]
    low = {torch.float32: -140, torch.bfloat16: -126, torch.float16: -20}[dtype]
    mags = np.concatenate([np.arange(low, top, 7), [top, 0, 62, 63, 64, -49, -50, -51, -64] if top > 64 else [top, 0]])
    B, L, Hq, Hkv = 2, len(mags), 5, 3
    g = np.random.default_rng(D)
    def rows(h):
        x = g.uniform(0.5, 1.9, (B, L, h, D)) * g.choice([-1.0, 1.0], (B, L, h, D)) * 2.0 ** mags[:, None, None]
        x[:, :, 0, :] = np.where(np.arange(D) == 7, x[:, :, 0, :], x[:, :, 0, :] * 2.0 ** -20)   # one large channel
        return torch.from_numpy(x).to(dtype).cuda()
    q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    wq, wk = (torch.from_numpy(g.uniform(0.5, 2, D)).float().cuda() for _ in range(2))
    table = rope_table(200, D)
    pos = g.integers(0, 200, (B, L))
    for eps in (0.0, 1e-38, 1e-30, 1e-6):
        op = QKNormRope(Hq, Hkv, D, wq, wk, table, eps=eps, interleaved=interleaved)
        outs = op(q, k, v, positions=torch.from_numpy(pos).cuda())
        for x, w, got in ((q, wq, outs[0]), (k, wk, outs[1])):
            ref, bound = reference(x, w, table, pos, float(np.float32(eps)), interleaved)
            some = np.asarray((x != 0).any(-1).cpu()).transpose(0, 2, 1)    # (a row of zeros without eps has no value)
            err = np.abs(got.double().cpu().numpy() - ref)
            assert (err <= bound)[some].all(), (eps, np.unique(mags[np.argwhere(~(err <= bound))[:, 2]]))


def test_infinite_and_empty_rows_stay_alone():
    """NaN, infinities and zero rows next to ordinary and huge ones change none of these."""
    D, H = 128, 6
    x = torch.randn(1, 1, H, D, device="cuda")
    x[0, 0, 1] *= 1e30
    w = torch.ones(D, device="cuda")
    op = QKNormRope(H, H, D, w, w, None, eps=1e-6)
    good = op(x, x, x)[0]
    assert good.isfinite().all() and good[0, 1].abs().max() > 1
    y = x.clone()
    y[0, 0, 2, 5] = float("nan")
    y[0, 0, 3, 9] = float("inf")
    y[0, 0, 4] = 0
    out = op(y, y, y)[0]
    for h in (0, 1, 5):
        assert torch.equal(out[0, h], good[0, h])
    assert out[0, 2].isnan().all() and out[0, 3, 0, 9].isnan() and (out[0, 4] == 0).all()
