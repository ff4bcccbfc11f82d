"""Block-sparse decode over the quantized KV cache and the norm + rotation in front of it, as measured cases.

Four operators, in the order in which a decode step calls them:

  norm_rope  norm of every query and key head, the position rotation and the change to the cache's fp16
             head-major layout, in one pass over a projection's output
  scores     an upper bound of each quantized key block's logits, from its per-channel steps and zeros
  select     the blocks of the largest scores of each (sequence, kv head) row
  decode     attention of one new query per sequence over the selected blocks and the fp16 residual

``prepare`` makes the inputs (keys with outlier channels and an attention sink, as everywhere in this
repository); ``run`` is one call, in its plain form or, with ``own``, through the package.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of each of 8 sequences, 7B layer: the step's first launch, pure latency
        dict(name="norm_rope_7b_token", op="norm_rope", B=8, L=1, Hq=32, Hkv=32, D=128, dtype="bf16", rot=128,
             interleaved=False, norm=True, far=131072),
        # one layer's whole prompt batch of the 7B shape
        dict(name="norm_rope_7b_prompt", op="norm_rope", B=8, L=4096, Hq=32, Hkv=32, D=128, dtype="bf16", rot=128,
             interleaved=False, norm=True, far=4096),
        # an odd chunk of a grouped-head prompt: fp32 input, interleaved pairs, half of the channels rotated
        dict(name="norm_rope_gqa_chunk", op="norm_rope", B=3, L=777, Hq=16, Hkv=8, D=64, dtype="f32", rot=32,
             interleaved=True, norm=True, far=32768),
        # the 7B layer at 4096 tokens: 124 blocks in each of 256 rows
        dict(name="scores_7b", op="scores", B=8, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=4096, ragged=False),
        # two sequences of 131072 tokens: 4092 blocks in each of 64 rows
        dict(name="scores_long", op="scores", B=2, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=131072, ragged=False),
        # the selections that follow those scores
        dict(name="select_7b", op="select", rows=256, cols=124, keep=32, first=1, ragged=False),
        dict(name="select_long", op="select", rows=64, cols=4092, keep=128, first=1, ragged=True),
        # one head, one sequence: pure latency
        dict(name="decode_tiny", op="decode", B=1, Hq=1, Hkv=1, D=64, bits=2, G=32, R=32, L=256, keep=4, ragged=False),
        # the 7B layer: 1024 of 4096 tokens
        dict(name="decode_7b", op="decode", B=8, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=4096, keep=32,
             ragged=False),
        # the same on the paged cache, prompts of 512 to 7680 tokens
        dict(name="decode_7b_ragged", op="decode", B=8, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=4096, keep=32,
             ragged=True),
        # grouped heads, 4 bits, groups of 128: 2048 of 8192 tokens of 64 sequences
        dict(name="decode_gqa", op="decode", B=64, Hq=32, Hkv=8, D=128, bits=4, G=128, R=128, L=8192, keep=16,
             ragged=False),
        # long context: 4096 of 131072 tokens
        dict(name="decode_long", op="decode", B=2, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=131072, keep=128,
             ragged=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_rope", "scores", "select", "decode", "decode"])
    if op == "select":
        cols = spread(3, 8192)
        rows = spread(1, max(2, min(2048, (1 << 21) // cols)))
        keep = min(cols, spread(1, 512))
        return dict(op=op, rows=rows, cols=cols, keep=keep, first=rng.randint(0, min(keep, 4)), ragged=rng.random() < 0.5)
    D = rng.choice([64, 128])
    nq = rng.choice([1, 2, 4])
    Hkv = rng.choice([1, 2, 5, 8, 16, 32])
    if op == "norm_rope":
        B = spread(1, 64)
        most = (1 << 25) // (B * Hkv * (nq + 2) * D)
        return dict(op=op, B=B, L=spread(1, max(2, min(32768, most))), Hq=nq * Hkv, Hkv=Hkv, D=D,
                    dtype=rng.choice(["f16", "bf16", "f32"]), rot=rng.choice([0, 16, 32, 48, 64, D]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, far=spread(40000, 200000))
    G = rng.choice([g for g in (32, 64, 128) if g <= D])
    R = G * rng.choice([1, 1, 2]) if G > 32 else rng.choice([32, 64, 96, 128])
    B = spread(1, 64)
    most = (1 << 22) // (B * Hkv)
    L = spread(R + G + 1, max(R + G + 2, min(131072, most)))
    blocks = (L - R + G - 1) // G
    case = dict(op=op, B=B, Hq=nq * Hkv, Hkv=Hkv, D=D, bits=rng.choice([2, 4, 8]), G=G, R=R, L=L,
                ragged=rng.random() < 0.4)
    if op == "decode":
        case["keep"] = min(blocks, spread(1, max(2, 8192 // G)))
    return case


# ---- the shapes of a case ---------------------------------------------------------------------------


def _lengths(c):
    """Tokens of each sequence: all L, or spread evenly around L."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [max(1, c["L"] * (2 * i + 1) // c["B"]) for i in range(c["B"])]


def _split(n, c):
    """(quantized blocks, residual rows) of a prompt of n tokens."""
    blocks = (max(n - c["R"], 0) + c["G"] - 1) // c["G"]
    return blocks, n - blocks * c["G"]


def _kept(c, blocks):
    return min(c["keep"], blocks)


def work(c):
    if c["op"] == "norm_rope":
        n = c["B"] * c["L"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (size + 2) + c["B"] * c["L"] * (8 + 4 * c["rot"]), "flops": 8 * n}
    if c["op"] == "select":
        return {"bytes": 4 * c["rows"] * (c["cols"] + c["keep"]), "flops": c["rows"] * c["cols"]}
    nb = [_split(n, c) for n in _lengths(c)]
    nq, D, G, Hkv = c["Hq"] // c["Hkv"], c["D"], c["G"], c["Hkv"]
    if c["op"] == "scores":
        blocks = sum(b for b, _ in nb) * Hkv
        return {"bytes": blocks * (4 * D + 4) + c["B"] * c["Hq"] * D * 2, "flops": blocks * nq * 4 * D}
    part = G * D * c["bits"] // 8 + 4 * D
    kept = sum(_kept(c, b) for b, _ in nb) * Hkv
    rows = sum(r for _, r in nb) * Hkv
    return {"bytes": kept * (2 * part + 4) + rows * 4 * D + 2 * c["B"] * c["Hq"] * D * 2,
            "flops": (kept * G + rows) * nq * 4 * D}


# ---- inputs -----------------------------------------------------------------------------------------


def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + tag)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _queries(c, seed):
    """q [B][Hq][D] fp16 and each kv head's sink direction."""
    g = _gen(seed, 1)
    u = _randn((c["B"], c["Hkv"], c["D"]), g)
    u = u / u.norm(dim=-1, keepdim=True)
    q = _randn((c["B"], c["Hq"], c["D"]), g)
    q = q + 0.5 * math.sqrt(c["D"]) * u.repeat_interleave(c["Hq"] // c["Hkv"], dim=1)
    return q.half(), u


def _keys_values(c, seed, i, n, u):
    """K, V [Hkv][n][D] fp16 of sequence i: four outlier channels per head, token 0 along the sink direction."""
    g = _gen(seed, 10 + i)
    scale = torch.ones(c["Hkv"], c["D"], device="cuda")
    at = torch.rand(c["Hkv"], c["D"], generator=g, device="cuda").argsort(dim=1)[:, :4]
    scale.scatter_(1, at, 10 + 40 * torch.rand(c["Hkv"], 4, generator=g, device="cuda"))
    k = _randn((c["Hkv"], n, c["D"]), g) * scale[:, None]
    k[:, 0] = 40.0 * u[i]
    k = k.half()
    return k, _randn((c["Hkv"], n, c["D"]), g).half()


def _block_lists(c, seed, cols):
    """The blocks that a selection kept: the first one, and others at random; ascending, -1 behind. [B][Hkv][keep]"""
    g = _gen(seed, 3)
    score = torch.rand(c["B"], c["Hkv"], cols, generator=g, device="cuda")
    score[..., 0] = 2
    nb = torch.tensor([_split(n, c)[0] for n in _lengths(c)], device="cuda")[:, None, None]
    at = torch.arange(cols, device="cuda")
    score = torch.where(at < nb, score, torch.full_like(score, -1))
    keep = min(c["keep"], cols)
    top = score.sort(dim=-1, descending=True, stable=True)
    pick = torch.where(top.values[..., :keep] >= 0, top.indices[..., :keep], torch.full_like(top.indices[..., :keep], cols))
    pick = pick.sort(dim=-1).values
    return torch.where(pick < cols, pick, torch.full_like(pick, -1)).int()


def _score_rows(c, seed):
    """Scores as a step gives them: spread around a common level, some of them equal, ragged rows padded with -inf."""
    g = _gen(seed, 4)
    s = 6 + 4 * _randn((c["rows"], c["cols"]), g)
    s[::3] = (s[::3] * 4).round() / 4
    if c["ragged"]:
        n = (torch.rand(c["rows"], generator=g, device="cuda") * (c["cols"] + 1)).long()
        s = s.masked_fill(torch.arange(c["cols"], device="cuda") >= n[:, None], -math.inf)
    return s


def _norm_rope_inputs(c, seed):
    g = _gen(seed, 5)
    B, L, Hq, Hkv, D = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"]
    dt = DTYPES[c["dtype"]]
    qkv = (_randn((B, L, (Hq + 2 * Hkv) * D), g) * 1.5).to(dt)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))
    w = [1 + 0.2 * _randn((D,), g) for _ in range(2)] if c["norm"] else [None, None]
    table = pos = None
    if c["rot"]:
        freq = 500000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        angle = torch.arange(c["far"], device="cuda", dtype=torch.float64)[:, None] * freq
        table = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
        start = (torch.rand(B, generator=g, device="cuda") * (c["far"] - L + 1)).long()
        pos = start[:, None] + torch.arange(L, device="cuda")
    return dict(q=q, k=k, v=v, wq=w[0], wk=w[1], table=table, pos=pos)


def prepare(c, seed):
    s = dict(c=c)
    if c["op"] == "norm_rope":
        s.update(_norm_rope_inputs(c, seed))
        shape = lambda h: (c["B"], h, c["L"], c["D"])  # noqa: E731
        s["out"] = tuple(torch.empty(shape(h), dtype=torch.float16, device="cuda") for h in (c["Hq"], c["Hkv"], c["Hkv"]))
        if own:
            from bit_kivi_kv_gb300.kivi import QKNormRope
            s["op"] = QKNormRope(c["Hq"], c["Hkv"], c["D"], s["wq"], s["wk"], s["table"], eps=1e-5,
                                 interleaved=c["interleaved"])
        return s
    if c["op"] == "select":
        s["scores"] = _score_rows(c, seed)
        s["out"] = torch.empty(c["rows"], c["keep"], dtype=torch.int32, device="cuda")
        if own:
            from bit_kivi_kv_gb300.kivi import select_blocks
            s["op"] = select_blocks
        return s
    lens = _lengths(c)
    nb = [_split(n, c)[0] for n in lens]
    q, u = _queries(c, seed)
    s["q"] = q
    s["cols"] = max(nb)
    if c["op"] == "scores":
        s["out"] = torch.empty(c["B"], c["Hkv"], max(nb), dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.empty_like(q)
        s["blocks"] = _block_lists(c, seed, max(nb))
    if own:
        _prepare_cache(s, c, seed, lens, u)
    else:
        _prepare_plain(s, c, seed, lens, nb, u)
    return s


def _prepare_cache(s, c, seed, lens, u):
    """The package's cache, holding the prompts."""
    from bit_kivi_kv_gb300.kivi import KiviCache, KiviPagedCache
    shape = (c["Hq"], c["Hkv"], c["D"], c["bits"], c["G"], c["R"])
    if c["ragged"]:
        most = max(_split(n, c)[0] for n in lens) + 1
        cache = KiviPagedCache(c["B"], *shape, most, sum(_split(n, c)[0] for n in lens) + c["B"])
        s["seqs"] = [cache.add(*_keys_values(c, seed, i, n, u)) for i, n in enumerate(lens)]
    else:
        cache = KiviCache(c["B"], *shape, c["L"] + 64)
        k = torch.empty(c["B"], c["Hkv"], c["L"], c["D"], dtype=torch.float16, device="cuda")
        v = torch.empty_like(k)
        for i in range(c["B"]):
            k[i], v[i] = _keys_values(c, seed, i, c["L"], u)
        cache.prefill(k, v)
        torch.cuda.synchronize()
    s["cache"] = cache


def _levels(x, dim, bits):
    """Step and zero (fp16) of groups along dim, and the code of every value."""
    x = x.float()
    lo, hi = x.amin(dim, keepdim=True) + 0.0, x.amax(dim, keepdim=True) + 0.0
    step, zero = ((hi - lo) / (2 ** bits - 1)).half(), lo.half()
    code = ((x - zero.float()) / step.float()).round().clamp(0, 2 ** bits - 1)
    return step, zero, torch.where(step == 0, torch.zeros_like(code), code).to(torch.uint8)


def _prepare_plain(s, c, seed, lens, nb, u):
    """The same cache as plain tensors: codes, steps and zeros per block, and the residual rows, padded to the longest."""
    B, H, D, G, most = c["B"], c["Hkv"], c["D"], c["G"], max(nb)
    half = dict(dtype=torch.float16, device="cuda")
    s["ks"], s["kz"] = torch.zeros(B, H, most, D, **half), torch.zeros(B, H, most, D, **half)
    if c["op"] == "decode":
        s["kc"] = torch.zeros(B, H, most, G, D, dtype=torch.uint8, device="cuda")
        s["vc"] = torch.zeros_like(s["kc"])
        s["vs"], s["vz"] = torch.zeros(B, H, most, G, D // G, **half), torch.zeros(B, H, most, G, D // G, **half)
        s["kr"], s["vr"] = torch.zeros(B, H, c["R"], D, **half), torch.zeros(B, H, c["R"], D, **half)
        s["rows"] = torch.tensor([n - b * G for n, b in zip(lens, nb)], device="cuda")
    for i, (n, b) in enumerate(zip(lens, nb)):
        k, v = _keys_values(c, seed, i, n, u)
        if b:
            step, zero, code = _levels(k[:, :b * G].reshape(H, b, G, D), 2, c["bits"])
            s["ks"][i, :, :b], s["kz"][i, :, :b] = step[:, :, 0], zero[:, :, 0]
            if c["op"] == "decode":
                s["kc"][i, :, :b] = code
                step, zero, code = _levels(v[:, :b * G].reshape(H, b, G, D // G, G), 4, c["bits"])
                s["vs"][i, :, :b], s["vz"][i, :, :b] = step[..., 0], zero[..., 0]
                s["vc"][i, :, :b] = code.reshape(H, b, G, D)
        if c["op"] == "decode":
            s["kr"][i, :, :n - b * G], s["vr"][i, :, :n - b * G] = k[:, b * G:], v[:, b * G:]
    s["nb"] = torch.tensor(nb, device="cuda")


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    c = s["c"]
    if own:
        return _own(s, c)
    return {"norm_rope": _plain_norm_rope, "scores": _plain_scores, "select": _plain_select,
            "decode": _plain_decode}[c["op"]](s, c)


def _own(s, c):
    if c["op"] == "norm_rope":
        return s["op"](s["q"], s["k"], s["v"], s["pos"], out=s["out"])
    if c["op"] == "select":
        return s["op"](s["scores"], c["keep"], keep_first=c["first"], out=s["out"])
    paged = (s["seqs"],) if c["ragged"] else ()
    if c["op"] == "scores":
        return s["cache"].block_scores(*paged, s["q"], out=s["out"])
    return s["cache"].decode_blocks(*paged, s["q"], s["blocks"], out=s["out"])


def _plain_norm_rope(s, c):
    def head(x, w):
        y = x.float()
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
        if c["rot"]:
            half = c["rot"] // 2
            cos, sin = s["table"][s["pos"]][:, :, None].split(half, dim=-1)
            if c["interleaved"]:
                a, b = y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]
                turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
            else:
                a, b = y[..., :half], y[..., half:c["rot"]]
                turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
            y = torch.cat([turned, y[..., c["rot"]:]], dim=-1)
        return y.half().transpose(1, 2).contiguous()

    return head(s["q"], s["wq"]), head(s["k"], s["wk"]), s["v"].half().transpose(1, 2).contiguous()


def _plain_scores(s, c):
    q = s["q"].float().unflatten(1, (c["Hkv"], -1))
    bound = q @ s["kz"].float().transpose(2, 3) + (2 ** c["bits"] - 1) * (q.clamp(min=0) @ s["ks"].float().transpose(2, 3))
    best = (bound / math.sqrt(c["D"])).amax(2)
    return best.masked_fill(torch.arange(s["cols"], device=best.device) >= s["nb"][:, None, None], -math.inf)


def _plain_select(s, c):
    x = s["scores"]
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    ok = x > -math.inf
    at = torch.arange(c["cols"], device=x.device)
    x = torch.where((at < c["first"]) & ok, torch.full_like(x, math.inf), x)
    top = x.sort(dim=1, descending=True, stable=True)
    pick = top.indices[:, :c["keep"]]
    pick = torch.where(ok.gather(1, pick), pick, torch.full_like(pick, c["cols"])).sort(dim=1).values
    return torch.where(pick < c["cols"], pick, torch.full_like(pick, -1)).int()


def _plain_decode(s, c):
    B, H, D, G = c["B"], c["Hkv"], c["D"], c["G"]
    q = s["q"].float().unflatten(1, (H, -1))
    at = s["blocks"].long().clamp(min=0)
    row = (torch.arange(B, device=q.device)[:, None, None], torch.arange(H, device=q.device)[None, :, None], at)
    k = s["kc"][row].float() * s["ks"][row].float()[..., None, :] + s["kz"][row].float()[..., None, :]
    v = s["vc"][row].unflatten(-1, (D // G, G)).float() * s["vs"][row].float()[..., None] + s["vz"][row].float()[..., None]
    k = torch.cat([k.flatten(2, 3), s["kr"].float()], dim=2)
    v = torch.cat([v.flatten(-2).flatten(2, 3), s["vr"].float()], dim=2)
    there = torch.cat([(s["blocks"] >= 0).repeat_interleave(G, dim=2),
                       (torch.arange(c["R"], device=q.device) < s["rows"][:, None])[:, None].expand(B, H, -1)], dim=2)
    x = (q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(~there[:, :, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    return (p @ v / p.sum(-1, keepdim=True)).flatten(1, 2).half()


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def exact(c, seed):
    return {"norm_rope": _exact_norm_rope, "scores": _exact_scores, "select": _exact_select,
            "decode": _exact_decode}[c["op"]](c, seed)


def _exact_norm_rope(c, seed):
    s = _norm_rope_inputs(c, seed)
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        z = x.double()
        if w is not None:
            z = z * torch.rsqrt((z * z).sum(-1, keepdim=True) / c["D"] + 1e-5) * w.double()
        if c["rot"]:
            t = s["table"].double()[s["pos"]].unsqueeze(2)
            turn = torch.complex(t[..., :c["rot"] // 2], t[..., c["rot"] // 2:])
            part = z[..., :c["rot"]]
            if c["interleaved"]:
                part = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
            else:
                both = torch.complex(part[..., :c["rot"] // 2].contiguous(), part[..., c["rot"] // 2:].contiguous()) * turn
                part = torch.cat([both.real, both.imag], dim=-1)
            z = torch.cat([part, z[..., c["rot"]:]], dim=-1)
        outs.append(z.permute(0, 2, 1, 3).contiguous())
    return tuple(outs) + (s["v"].double().permute(0, 2, 1, 3).contiguous(),)


def _f32(x):
    return x.float().double()


def _exact_groups(x, dim, bits):
    """Step and zero of each group along dim, in 64 bits with the format's single-precision roundings."""
    lo, hi = x.double().amin(dim), x.double().amax(dim)
    lo = torch.where(lo == 0, torch.zeros_like(lo), lo)
    return _f32(_f32(hi - lo) / (2 ** bits - 1)).half().double(), lo.half().double()


def _exact_hat(x, step, zero, bits):
    code = torch.round(_f32(_f32(x.double() - zero) / step)).clamp(0, 2 ** bits - 1)
    return torch.where(step == 0, torch.zeros_like(code), code) * step + zero


def _exact_scores(c, seed):
    q, u = _queries(c, seed)
    lens = _lengths(c)
    out = torch.full((c["B"], c["Hkv"], max(_split(n, c)[0] for n in lens)), -math.inf, dtype=torch.float64, device="cuda")
    nq = c["Hq"] // c["Hkv"]
    for i, n in enumerate(lens):
        b, _ = _split(n, c)
        k, _ = _keys_values(c, seed, i, n, u)
        for h in range(c["Hkv"] if b else 0):
            step, zero = _exact_groups(k[h, :b * c["G"]].reshape(b, c["G"], c["D"]), 1, c["bits"])
            top = zero + (2 ** c["bits"] - 1) * step
            x = q[i, h * nq:(h + 1) * nq].double()[:, None]
            out[i, h, :b] = (torch.where(x > 0, x * top, x * zero).sum(-1) / math.sqrt(c["D"])).max(0).values
    return out


def _exact_select(c, seed):
    scores = _score_rows(c, seed).double().cpu().numpy()
    out = torch.full((c["rows"], c["keep"]), -1, dtype=torch.int32)
    for r, row in enumerate(scores):
        fit = [n for n in range(c["cols"]) if row[n] > -math.inf]
        fit.sort(key=lambda n: (n >= c["first"], -row[n] if n >= c["first"] else 0.0, n))
        fit = sorted(fit[:c["keep"]])
        out[r, :len(fit)] = torch.tensor(fit, dtype=torch.int32)
    return out


def _exact_decode(c, seed):
    q, u = _queries(c, seed)
    lens = _lengths(c)
    blocks = _block_lists(c, seed, max(_split(n, c)[0] for n in lens)).cpu()
    D, G, nq = c["D"], c["G"], c["Hq"] // c["Hkv"]
    out = torch.empty(c["B"], c["Hq"], D, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        b, _ = _split(n, c)
        k, v = _keys_values(c, seed, i, n, u)
        for h in range(c["Hkv"]):
            at = [int(x) for x in blocks[i, h] if x >= 0]
            kb = k[h, :b * G].reshape(b, G, D)[at]
            vb = v[h, :b * G].reshape(b, G, D)[at].reshape(-1, D // G, G)
            step, zero = _exact_groups(kb, 1, c["bits"]) if at else (kb.double()[:, 0], kb.double()[:, 0])
            keys = torch.cat([_exact_hat(kb, step[:, None], zero[:, None], c["bits"]).reshape(-1, D), k[h, b * G:].double()])
            step, zero = _exact_groups(vb, 2, c["bits"]) if at else (vb.double()[..., 0], vb.double()[..., 0])
            vals = torch.cat([_exact_hat(vb, step[..., None], zero[..., None], c["bits"]).reshape(-1, D), v[h, b * G:].double()])
            x = q[i, h * nq:(h + 1) * nq].double() @ keys.T / math.sqrt(D)
            out[i, h * nq:(h + 1) * nq] = torch.softmax(x, dim=-1) @ vals
    return out
