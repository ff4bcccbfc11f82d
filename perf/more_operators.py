"""Chunks of new tokens over the paged cache, as measured cases.

Three operators of a serving step that brings more than one token of a sequence at a time (a piece of a prompt,
the proposals of a draft, several continuations of one prompt):

  attend  attention of the new tokens' queries over the sequences' cached tokens (quantized blocks and fp16
          residual, as they stand) and, causally, over the new tokens themselves; optionally with capped
          scores, a bias that grows with the distance, and a window
  branch  new sequences that share the pages of others, and a chunk appended to each: the blocks that the
          chunk completes quantized, the rest kept as residual rows
  read    cached tokens back as fp16, dequantized

``prepare`` makes the inputs (keys with outlier channels and an attention sink, as everywhere in this
repository); ``run`` is one call, in its plain form or, with ``own``, through the package.
"""
import math

import torch

own = False


def _attend(name, B, Hq, Hkv, D, bits, G, R, L, n, lens="equal", ragged=False, cap=0.0, window=0, slopes=False):
    return dict(name=name, op="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, bits=bits, G=G, R=R, L=L, n=n, lens=lens,
                ragged=ragged, cap=cap, window=window, slopes=slopes)


def listed():
    return [
        # one token of one short sequence of one head: pure latency
        _attend("attend_tiny", 1, 1, 1, 64, 2, 32, 32, 256, 1),
        # the 7B layer, 8 sequences of 512 to 7680 tokens: four proposals each checked in one call
        _attend("attend_7b_verify", 8, 32, 32, 128, 2, 32, 128, 4096, 4, ragged=True),
        # the same layer while one sequence's prompt comes in: 512 of its tokens beside one token of each other
        _attend("attend_7b_mixed", 8, 32, 32, 128, 2, 32, 128, 4096, 512, lens="first"),
        # a piece of every prompt, 512 tokens over 4096
        _attend("attend_7b_chunk", 8, 32, 32, 128, 2, 32, 128, 4096, 512),
        # grouped heads, 4 bits, groups of 128: chunks of different lengths over 8192 tokens
        _attend("attend_gqa_chunk", 16, 32, 8, 128, 4, 128, 128, 8192, 256, lens="ragged", ragged=True),
        # grouped heads, an odd piece over a long context: the last question after 131072 tokens
        _attend("attend_long", 1, 32, 8, 128, 2, 32, 128, 131072, 333),
        # a whole prompt into an empty cache
        _attend("attend_prompt", 1, 32, 8, 128, 2, 32, 128, 0, 8192),
        # capped scores, distance bias and a window; 8 bits, narrow heads, odd sizes
        _attend("attend_capped", 3, 16, 8, 64, 8, 64, 64, 5001, 777, lens="ragged", cap=30.0, window=2048, slopes=True),
        # proposals appended to branches of 8 sequences (the residual nearly full: each quantizes a block)
        dict(name="branch_7b_verify", op="branch", B=8, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=4096, n=4, times=1),
        # four continuations of each of four prompts, 500 tokens each
        dict(name="branch_gqa_chunk", op="branch", B=4, Hq=32, Hkv=8, D=128, bits=4, G=128, R=128, L=8192, n=500, times=4),
        # the newest 1000 tokens of three sequences
        dict(name="read_tail", op="read", B=3, Hq=8, Hkv=8, D=64, bits=8, G=64, R=64, L=2777, first=1777, count=1000),
        # the whole 7B layer, to be kept elsewhere in fp16
        dict(name="read_7b", op="read", B=8, Hq=32, Hkv=32, D=128, bits=2, G=32, R=128, L=4096, first=0, count=4096),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["attend", "attend", "attend", "branch", "read"])
    D = rng.choice([64, 128])
    G = rng.choice([g for g in (32, 64, 128) if g <= D])
    R = G * rng.choice([1, 1, 2]) if G > 32 else rng.choice([32, 64, 96, 128])
    Hkv = rng.choice([1, 2, 5, 8, 16, 32])
    nq = rng.choice([1, 2, 4])
    shape = dict(op=op, Hq=nq * Hkv, Hkv=Hkv, D=D, bits=rng.choice([2, 4, 8]), G=G, R=R)
    if op == "attend":
        n = min(spread(1, 4096), math.isqrt((1 << 30) // shape["Hq"]))
        B = spread(1, max(1, min(64, 2048 // n)))
        pairs = 1 << 29                             # (query head, query) x key pairs, with the chunk's within the listed cases'
        most = min(131072, (1 << 21) // (B * Hkv), pairs // (B * nq * Hkv * n))
        L = 0 if most < 2 or rng.random() < 0.1 else spread(1, most)
        fancy = rng.random() < 0.3
        return dict(shape, B=B, L=L, n=n, lens=rng.choice(["equal", "ragged", "first"]), ragged=rng.random() < 0.4,
                    cap=rng.choice([0.0, 20.0, 50.0]) if fancy else 0.0,
                    window=spread(1, 8192) if fancy and rng.random() < 0.5 else 0,
                    slopes=fancy and rng.random() < 0.5)
    times = spread(1, 8) if op == "branch" else 1
    B = spread(1, max(1, 32 // times))
    L = spread(1, min(65536, (1 << 20) // (B * Hkv)))
    if op == "branch":
        return dict(shape, B=B, L=L, n=spread(1, max(2, min(4096, (1 << 19) // (B * times * Hkv)))), times=times)
    first = rng.randint(0, L - 1)
    return dict(shape, B=B, L=L, first=first, count=rng.randint(1, L - first))


# ---- the shapes of a case ---------------------------------------------------------------------------


def _lengths(c):
    """Cached tokens of each sequence: all L, or spread evenly around L."""
    if not c.get("ragged"):
        return [c["L"]] * c["B"]
    return [c["L"] * (2 * i + 1) // c["B"] for i in range(c["B"])]


def _chunks(c):
    """New tokens of each sequence: n each; n of the first and one of the others; or from n downwards."""
    if c.get("lens") == "first":
        return [c["n"]] + [1] * (c["B"] - 1)
    if c.get("lens") == "ragged":
        return [max(1, c["n"] * (c["B"] - i) // c["B"]) for i in range(c["B"])]
    return [c["n"]] * c["B"]


def _split(n, c):
    """(quantized blocks, residual rows) of a prompt of n tokens."""
    blocks = (max(n - c["R"], 0) + c["G"] - 1) // c["G"]
    return blocks, n - blocks * c["G"]


def _after(c):
    """(quantized blocks, residual rows) of a sequence of the case when its chunk is appended."""
    return _split(c["L"] + c["n"], c)


def _token_bytes(c):
    """Bytes of one quantized token of one head, keys and values."""
    return (2 * c["G"] * c["D"] * c["bits"] // 8 + 8 * c["D"]) / c["G"]


def work(c):
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "attend":
        bytes_ = flops = 0
        for past, n in zip(_lengths(c), _chunks(c)):
            low = max(0, past + 1 - c["window"]) if c["window"] else 0        # the oldest token that any query sees
            quantized = _split(past, c)[0] * c["G"]
            bytes_ += Hkv * (max(0, quantized - low) * _token_bytes(c) + (past - max(quantized, low)) * 4 * D)
            bytes_ += n * (2 * Hkv + 2 * Hq) * 2 * D
            seen = c["window"] or past + n
            whole = max(0, min(n, seen - past))                               # queries that the window cuts nothing from
            flops += 4 * D * Hq * (whole * past + whole * (whole + 1) // 2 + (n - whole) * seen)
        return {"bytes": bytes_, "flops": flops}
    if c["op"] == "branch":
        copies = c["B"] * c["times"] * Hkv
        blocks, rows = _split(c["L"], c)
        new, left = _after(c)
        fresh = (new - blocks) * c["G"]
        # the residual and the chunk read, the new blocks and residual rows written; and all of that read back as fp16
        moved = (rows + c["n"]) * 4 * D + fresh * _token_bytes(c) + left * 4 * D
        back = fresh * _token_bytes(c) + left * 4 * D + (fresh + left) * 4 * D
        return {"bytes": copies * (moved + back), "flops": copies * fresh * D * 8}
    quantized = _split(c["L"], c)[0] * c["G"]
    old = max(0, min(quantized, c["first"] + c["count"]) - c["first"])
    rows = c["B"] * Hkv
    return {"bytes": rows * (old * _token_bytes(c) + (c["count"] - old) * 4 * D + c["count"] * 4 * D),
            "flops": rows * old * D * 4}


# ---- inputs -----------------------------------------------------------------------------------------


def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + tag)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _sinks(c, seed):
    """Each kv head's sink direction."""
    u = _randn((c["B"], c["Hkv"], c["D"]), _gen(seed, 1))
    return u / u.norm(dim=-1, keepdim=True)


def _queries(c, seed, u):
    """Queries of the new tokens, packed over the sequences: [tokens][Hq][D] fp16."""
    g = _gen(seed, 2)
    group = c["Hq"] // c["Hkv"]
    return torch.cat([_randn((n, c["Hq"], c["D"]), g) + 0.5 * math.sqrt(c["D"]) * u[i].repeat_interleave(group, dim=0)
                      for i, n in enumerate(_chunks(c))]).half()


def _keys_values(c, seed, i, n, u, more=0):
    """K, V [Hkv][n + more][D] fp16 of sequence i: four outlier channels per head, token 0 along the sink direction."""
    g = _gen(seed, 10 + i)
    scale = torch.ones(c["Hkv"], c["D"], device="cuda")
    at = torch.rand(c["Hkv"], c["D"], generator=g, device="cuda").argsort(dim=1)[:, :4]
    scale.scatter_(1, at, 10 + 40 * torch.rand(c["Hkv"], 4, generator=g, device="cuda"))
    k = _randn((c["Hkv"], n + more, c["D"]), g) * scale[:, None]
    k[:, 0] = 40.0 * u[i]
    return k.half(), _randn((c["Hkv"], n + more, c["D"]), g).half()


def _branch_rows(c, seed):
    """The new tokens of every branch, packed: k, v [B * times * n][Hkv][D] fp16."""
    g = _gen(seed, 3)
    shape = (c["B"] * c["times"] * c["n"], c["Hkv"], c["D"])
    return (3 * _randn(shape, g)).half(), _randn(shape, g).half()


def _slopes(c):
    """One slope per query head, a geometric sequence."""
    return torch.tensor([2.0 ** (-8 * (h + 1) / c["Hq"]) for h in range(c["Hq"])], device="cuda") if c["slopes"] else None


def prepare(c, seed):
    u = _sinks(c, seed)
    past = _lengths(c)
    s = dict(c=c)
    chunks = _chunks(c) if c["op"] == "attend" else [0] * c["B"]
    kv = [_keys_values(c, seed, i, past[i], u, chunks[i]) for i in range(c["B"])]
    if c["op"] == "attend":
        s["q"], s["slopes"], s["lens"] = _queries(c, seed, u), _slopes(c), chunks
        s["k"], s["v"] = (torch.cat([x[j][:, p:].transpose(0, 1) for x, p in zip(kv, past)]).contiguous() for j in (0, 1))
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "branch":
        s["k"], s["v"] = _branch_rows(c, seed)
    if c["op"] != "attend":
        count = c["count"] if c["op"] == "read" else c["L"] + c["n"] - _split(c["L"], c)[0] * c["G"]
        shape = (c["B"] * c.get("times", 1), c["Hkv"], count, c["D"])
        s["out"] = tuple(torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2))
    if own:
        _prepare_cache(s, c, kv, past)
    else:
        _prepare_plain(s, c, kv, past)
    return s


def _prepare_cache(s, c, kv, past):
    """The package's paged cache, holding the prompts."""
    from bit_kivi_kv_gb300.kivi import KiviPagedCache
    blocks = [_split(n, c)[0] for n in past]
    more = max(blocks) + 1
    pages = sum(blocks) + 1
    seqs = c["B"]
    if c["op"] == "branch":
        new = _after(c)[0] - blocks[0]
        more, pages, seqs = more + new, pages + c["B"] * c["times"] * new, c["B"] * (1 + c["times"])
    cache = KiviPagedCache(seqs, c["Hq"], c["Hkv"], c["D"], c["bits"], c["G"], c["R"], more, pages)
    s["seqs"] = [cache.add(k[:, :n].contiguous(), v[:, :n].contiguous()) for (k, v), n in zip(kv, past)]
    s["cache"] = cache


def _levels(x, dim, bits):
    """Step and zero (fp16) of groups along dim, and the code of every value."""
    x = x.float()
    lo, hi = x.amin(dim, keepdim=True) + 0.0, x.amax(dim, keepdim=True) + 0.0
    step, zero = ((hi - lo) / (2 ** bits - 1)).half(), lo.half()
    code = ((x - zero.float()) / step.float()).round().clamp(0, 2 ** bits - 1)
    return step, zero, torch.where(step == 0, torch.zeros_like(code), code).to(torch.uint8)


def _key_levels(k, c):
    """Steps, zeros [...][blocks][1][D] and codes [...][blocks][G][D] of keys [...][blocks * G][D]."""
    return _levels(k.unflatten(-2, (-1, c["G"])), -2, c["bits"])


def _value_levels(v, c):
    """Steps, zeros [...][blocks][G][D / G][1] and codes [...][blocks][G][D / G][G] of values [...][blocks * G][D]."""
    return _levels(v.unflatten(-2, (-1, c["G"])).unflatten(-1, (-1, c["G"])), -1, c["bits"])


def _prepare_plain(s, c, kv, past):
    """The same cache as plain tensors: codes, steps and zeros per block and the residual rows, padded to the longest."""
    B, H, D, G = c["B"], c["Hkv"], c["D"], c["G"]
    split = [_split(n, c) for n in past]
    most, rows = max(b for b, _ in split), max(r for _, r in split)
    half = dict(dtype=torch.float16, device="cuda")
    s["kc"] = torch.zeros(B, H, most, G, D, dtype=torch.uint8, device="cuda")
    s["vc"] = torch.zeros(B, H, most, G, D // G, G, dtype=torch.uint8, device="cuda")
    s["ks"], s["kz"] = torch.zeros(B, H, most, 1, D, **half), torch.zeros(B, H, most, 1, D, **half)
    s["vs"], s["vz"] = torch.zeros(B, H, most, G, D // G, 1, **half), torch.zeros(B, H, most, G, D // G, 1, **half)
    s["kr"], s["vr"] = torch.zeros(B, H, rows, D, **half), torch.zeros(B, H, rows, D, **half)
    for i, ((k, v), n, (b, r)) in enumerate(zip(kv, past, split)):
        if b:
            s["ks"][i, :, :b], s["kz"][i, :, :b], s["kc"][i, :, :b] = _key_levels(k[:, :b * G], c)
            s["vs"][i, :, :b], s["vz"][i, :, :b], s["vc"][i, :, :b] = _value_levels(v[:, :b * G], c)
        s["kr"][i, :, :r], s["vr"][i, :, :r] = k[:, b * G:n], v[:, b * G:n]
    if c["op"] == "attend":
        chunks = s["lens"]
        n = max(chunks)
        ones = lambda xs: torch.tensor(xs, device="cuda")[:, None]  # noqa: E731
        at = torch.arange(n, device="cuda")
        there = at < ones(chunks)                                                         # [B][n]
        s["rows"] = there.flatten().nonzero()[:, 0]                                       # packed tokens in [B * n]
        # where each key of [blocks | residual | chunk] stands in its sequence (-1: nowhere), and each query
        quantized, length = ones([b * G for b, _ in split]), ones(past)
        t, j = torch.arange(most * G, device="cuda"), torch.arange(rows, device="cuda")
        nowhere = torch.tensor(-1, device="cuda")
        s["key_at"] = torch.cat([torch.where(t < quantized, t, nowhere), torch.where(quantized + j < length, quantized + j, nowhere),
                                 torch.where(there, length + at, nowhere)], dim=1)
        s["query_at"] = length + at


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    c = s["c"]
    if own:
        return _own(s, c)
    return {"attend": _plain_attend, "branch": _plain_branch, "read": _plain_read}[c["op"]](s, c)


def _own(s, c):
    cache = s["cache"]
    if c["op"] == "attend":
        return cache.chunk_attn(s["seqs"], s["lens"], s["q"], s["k"], s["v"], out=s["out"], cap=c["cap"],
                                window=c["window"], slopes=s["slopes"])
    if c["op"] == "read":
        return cache.read(s["seqs"], c["first"], c["count"], out=s["out"])
    branches = cache.fork(s["seqs"] * c["times"])
    cache.append_chunk(branches, [c["n"]] * len(branches), s["k"], s["v"])
    out = cache.read(branches, _split(c["L"], c)[0] * c["G"], s["out"][0].shape[2], out=s["out"])
    for b in reversed(branches):
        cache.release(b)
    return out


def _dequantized(code, step, zero):
    return code.float() * step.float() + zero.float()


def _cached(s):
    """Keys and values of the quantized blocks in 32 bits, [B][Hkv][blocks * G][D]."""
    return (_dequantized(s["kc"], s["ks"], s["kz"]).flatten(2, 3),
            _dequantized(s["vc"], s["vs"], s["vz"]).flatten(4, 5).flatten(2, 3))


def _padded(x, s, c):
    """Packed [tokens][heads][D] as [B][heads][n][D], zeros behind a sequence's last token."""
    n = s["query_at"].shape[1]
    y = torch.zeros(c["B"] * n, *x.shape[1:], device=x.device)
    y[s["rows"]] = x.float()
    return y.unflatten(0, (c["B"], n)).transpose(1, 2)


def _plain_attend(s, c):
    H = c["Hkv"]
    k, v = _cached(s)
    k = torch.cat([k, s["kr"].float(), _padded(s["k"], s, c)], dim=2)
    v = torch.cat([v, s["vr"].float(), _padded(s["v"], s, c)], dim=2)
    q = _padded(s["q"], s, c).unflatten(1, (H, -1))                                       # [B][Hkv][group][n][D]
    group, n = q.shape[2:4]
    x = (q.flatten(2, 3) @ k.transpose(2, 3) / math.sqrt(c["D"])).unflatten(2, (group, n))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    key, query = s["key_at"][:, None], s["query_at"][:, :, None]                          # [B][n][keys]
    seen = (key >= 0) & (key <= query)
    if c["window"]:
        seen = seen & (key > query - c["window"])
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, H, group, 1, 1) * (key - query)[:, None, None].float()
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (group, n)).flatten(1, 2)                      # [B][Hq][n][D]
    return o.transpose(1, 2).flatten(0, 1)[s["rows"]].half()


def _plain_branch(s, c):
    def rows(resid, new):
        new = new.unflatten(0, (c["times"] * c["B"], c["n"])).transpose(1, 2)
        return torch.cat([resid.repeat(c["times"], 1, 1, 1), new], dim=2)

    k, v = rows(s["kr"], s["k"]), rows(s["vr"], s["v"])
    fresh = (_after(c)[0] - _split(c["L"], c)[0]) * c["G"]
    if not fresh:
        return k, v
    step, zero, code = _key_levels(k[:, :, :fresh], c)
    k_hat = _dequantized(code, step, zero).flatten(2, 3)
    step, zero, code = _value_levels(v[:, :, :fresh], c)
    v_hat = _dequantized(code, step, zero).flatten(4, 5).flatten(2, 3)
    return torch.cat([k_hat.half(), k[:, :, fresh:]], dim=2), torch.cat([v_hat.half(), v[:, :, fresh:]], dim=2)


def _plain_read(s, c):
    part = slice(c["first"], c["first"] + c["count"])
    return tuple(torch.cat([x.half(), r], dim=2)[:, :, part].contiguous() for x, r in zip(_cached(s), (s["kr"], s["vr"])))


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def exact(c, seed):
    return {"attend": _exact_attend, "branch": _exact_branch, "read": _exact_read}[c["op"]](c, seed)


def _f32(x):
    return x.float().double()


def _exact_hat(x, dim, bits):
    """Values of groups along dim after quantization, with the format's single-precision roundings of steps and codes."""
    lo, hi = x.double().amin(dim, keepdim=True), x.double().amax(dim, keepdim=True)
    lo = torch.where(lo == 0, torch.zeros_like(lo), lo)
    step, zero = _f32(_f32(hi - lo) / (2 ** bits - 1)).half().double(), lo.half().double()
    code = torch.round(_f32(_f32(x.double() - zero) / step)).clamp(0, 2 ** bits - 1)
    return torch.where(step == 0, torch.zeros_like(code), code) * step + zero


def _exact_tokens(k, v, n, c):
    """One head's keys and values [tokens][D] with the first n of them quantized."""
    D, G = c["D"], c["G"]
    if not n:
        return k.double(), v.double()
    kh = _exact_hat(k[:n].reshape(-1, G, D), 1, c["bits"]).reshape(-1, D)
    vh = _exact_hat(v[:n].reshape(n, D // G, G), 2, c["bits"]).reshape(-1, D)
    return torch.cat([kh, k[n:].double()]), torch.cat([vh, v[n:].double()])


def _exact_attend(c, seed):
    u = _sinks(c, seed)
    q = _queries(c, seed, u)
    slopes, group = _slopes(c), c["Hq"] // c["Hkv"]
    out, first = [], 0
    for i, (past, n) in enumerate(zip(_lengths(c), _chunks(c))):
        k, v = _keys_values(c, seed, i, past, u, n)
        distance = torch.arange(past, past + n, device="cuda")[:, None] - torch.arange(past + n, device="cuda")
        hidden = distance < 0
        if c["window"]:
            hidden |= distance >= c["window"]
        heads = []
        for h in range(c["Hq"]):
            if h % group == 0:
                keys, vals = _exact_tokens(k[h // group], v[h // group], _split(past, c)[0] * c["G"], c)
            x = q[first:first + n, h].double() @ keys.T * c["D"] ** -0.5
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if slopes is not None:
                x -= float(slopes[h]) * distance
            heads.append(torch.softmax(x.masked_fill_(hidden, -math.inf), dim=1) @ vals)
        out.append(torch.stack(heads, dim=1))
        first += n
    return torch.cat(out)


def _exact_branch(c, seed):
    u = _sinks(c, seed)
    kn, vn = (x.unflatten(0, (c["times"], c["B"], c["n"])) for x in _branch_rows(c, seed))
    old, new = _split(c["L"], c)[0] * c["G"], _after(c)[0] * c["G"]
    outs = [[], []]
    prompts = [_keys_values(c, seed, i, c["L"], u) for i in range(c["B"])]
    for j in range(c["times"]):
        for i, (k, v) in enumerate(prompts):
            heads = [_exact_tokens(torch.cat([k[h, old:], kn[j, i, :, h]]), torch.cat([v[h, old:], vn[j, i, :, h]]), new - old, c)
                     for h in range(c["Hkv"])]
            for o, x in zip(outs, zip(*heads)):
                o.append(torch.stack(x))
    return tuple(torch.stack(o) for o in outs)


def _exact_read(c, seed):
    u = _sinks(c, seed)
    outs = [[], []]
    for i in range(c["B"]):
        k, v = _keys_values(c, seed, i, c["L"], u)
        heads = [_exact_tokens(k[h], v[h], _split(c["L"], c)[0] * c["G"], c) for h in range(c["Hkv"])]
        for o, x in zip(outs, zip(*heads)):
            o.append(torch.stack(x)[:, c["first"]:c["first"] + c["count"]])
    return tuple(torch.stack(o) for o in outs)
