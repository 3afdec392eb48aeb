"""The 4-bit latent cache: writing rows into it, reading rows back, and the sparse attention over it.

Cases of three operators: ``write`` (bf16 latent rows quantised into the slots of a cache), ``read`` (cache rows,
picked by number, back to bf16) and ``attend`` (MLA attention of every query head over the query's selected rows of the
cache).  Where ``own`` is false the operators are computed in their plain form; where it is true they are the
framework's entry points.

The cache row of a latent row of D columns, the first Dv of them values: Dv four-bit integers u = c + 8 with c in
-7..7 (of eight columns, the even ones in nibbles 0-3 and the odd ones in nibbles 4-7 of a little-endian 32-bit word),
the D - Dv rope columns as bf16, one E4M3 scale per 16 value columns, one byte e + 127; the first three sections padded
to 16 bytes, the row too.  A value is c * scale * 2^e.  A row with a NaN or an infinity among its values has the byte
255 and stands for NaN in every value column.
"""
import math

import torch

own = False

MAX_SCALED = 7 * 448            # the largest |x| / 2^e of a row
E_MIN, E_MAX = -124, 114        # of the row's power of two
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def up16(n):
    return (n + 15) // 16 * 16


def layout(D, Dv):
    """Byte offsets of the rope columns, the scales, the exponent, and the row's bytes."""
    rope = up16(Dv // 2)
    scales = rope + up16(2 * (D - Dv))
    exponent = scales + (Dv + 15) // 16
    return rope, scales, exponent, up16(exponent + 1)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of one request, written into its page, the page read back
        {"name": "write_1", "op": "write", "rows": 1, "cache_rows": 64, "D": 576, "Dv": 512, "stride": 576},
        # one new token of each request of a decode batch
        {"name": "write_61", "op": "write", "rows": 61, "cache_rows": 1024, "D": 576, "Dv": 512, "stride": 576},
        # a prefill chunk; the latent is a slice of a wider projection output
        {"name": "write_8000", "op": "write", "rows": 8000, "cache_rows": 8192, "D": 576, "Dv": 512, "stride": 2112},
        # a long request in one piece
        {"name": "write_65536", "op": "write", "rows": 65536, "cache_rows": 65536, "D": 576, "Dv": 512, "stride": 576},
        # the rows one query selected, back in bf16
        {"name": "read_2048", "op": "read", "rows": 2048, "cache_rows": 65536, "D": 576, "Dv": 512},
        # a batch's rows in request order out of a scattered cache, some slots empty
        {"name": "read_100003", "op": "read", "rows": 100003, "cache_rows": 131072, "D": 576, "Dv": 512},
        # one token of one long request
        {"name": "attend_1", "op": "attend", "queries": 1, "context": 65536, "topk": 2048, "H": 128, "chunk": False,
         "ragged": False, "sink": False},
        # a small decode batch with short and empty contexts, a tensor-parallel rank's heads
        {"name": "attend_7_ragged", "op": "attend", "queries": 7, "context": 8000, "topk": 2048, "H": 32,
         "chunk": False, "ragged": True, "sink": True},
        # a decode batch, all heads on one GPU; the cache is larger than the L2
        {"name": "attend_64", "op": "attend", "queries": 64, "context": 8192, "topk": 2048, "H": 128, "chunk": False,
         "ragged": False, "sink": True},
        # a decode batch, 16 heads per rank
        {"name": "attend_64_h16", "op": "attend", "queries": 64, "context": 8192, "topk": 2048, "H": 16,
         "chunk": False, "ragged": False, "sink": False},
        # a decode batch that is no multiple of the SM pairs
        {"name": "attend_200", "op": "attend", "queries": 200, "context": 3000, "topk": 2048, "H": 64,
         "chunk": False, "ragged": True, "sink": False},
        # a prefill chunk of one request, all heads
        {"name": "attend_chunk_2048", "op": "attend", "queries": 2048, "context": 8192, "topk": 2048, "H": 128,
         "chunk": True, "ragged": False, "sink": True},
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of lo..hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    if op != "attend":
        rows = _spread(rng, 1, 60000)
        # the shapes of the DeepSeek-V3.2 latent, and small odd ones
        D, Dv = rng.choice([(576, 512), (576, 512), (64, 48), (200, 136)])
        case = {"op": op, "rows": rows, "cache_rows": up16(rows + rng.randint(0, max(16, rows // 8))), "D": D, "Dv": Dv}
        if op == "write":
            case["stride"] = D + 8 * rng.randint(0, 40)
        return case
    queries = _spread(rng, 1, 600)
    chunk = rng.random() < 0.25
    context = _spread(rng, 300, 9000)
    if chunk:
        context = max(context, queries)
    return {"op": op, "queries": queries, "context": context,
            "topk": rng.choice([64, 500, 1024, 2048, 2048, rng.randint(1, 2048)]),
            "H": rng.choice([8, 16, 24, 32, 64, 128, 128, rng.randint(1, 128)]), "chunk": chunk,
            "ragged": not chunk and rng.random() < 0.5, "sink": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _rows(n, D, g):
    """Latent rows as a normalised latent has them, N(0, 1) with a spread of row magnitudes."""
    x = torch.randn(n, D, device="cuda", generator=g)
    return (x * torch.exp(0.3 * torch.randn(n, 1, device="cuda", generator=g))).to(BF16)


def _lengths(case, g):
    """KV length of each query's request (ragged: log-uniform, the first one empty)."""
    n, ctx = case["queries"], case["context"]
    if not case["ragged"]:
        return torch.full((n,), ctx, device="cuda")
    u = torch.rand(n, device="cuda", generator=g)
    lens = torch.exp(u * math.log(ctx)).round().clamp(1, ctx).long()
    lens[0] = 0
    lens[-1] = ctx
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] in ("write", "read"):
        D, Dv, n, R = case["D"], case["Dv"], case["rows"], case["cache_rows"]
        state = {"case": dict(case), "cache": plain_quantise(_rows(R, D, g), Dv)}
        if case["op"] == "write":
            wide = _rows(n, case["stride"], g)
            off = (case["stride"] - D) // 16 * 8   # the latent's columns of the wider tensor
            state["kv"] = wide[:, off:off + D]
            state["slots"] = torch.randperm(R, device="cuda", generator=g)[:n].to(torch.int32)
        else:
            rows = torch.randint(0, R, (n,), device="cuda", generator=g)
            holes = torch.rand(n, device="cuda", generator=g) < 0.02
            state["rows"] = torch.where(holes, -1, rows).to(torch.int32)
        return state
    n, ctx, topk, H, D = case["queries"], case["context"], case["topk"], case["H"], 576
    R = ctx if case["chunk"] else n * ctx
    cache = torch.cat([plain_quantise(_rows(min(1 << 18, R - r), D, g), 512) for r in range(0, R, 1 << 18)])
    if case["chunk"]:    # the queries are the last positions of one request
        seen, base = ctx - n + 1 + torch.arange(n, device="cuda"), torch.zeros(n, dtype=torch.long, device="cuda")
    else:                # every query is the newest token of its own request
        seen, base = _lengths(case, g), torch.arange(n, device="cuda") * ctx
    score = torch.rand(n, max(ctx, topk), device="cuda", generator=g)
    score.masked_fill_(torch.arange(score.shape[1], device="cuda") >= seen[:, None], -1.0)
    val, pos = score.topk(topk, dim=1)
    pos = torch.where(val < 0, score.shape[1], pos).sort(dim=1).values   # ascending, the unused entries last
    # the cache's rows lie scattered: KV row r is at slot slots[r]
    state = {"case": dict(case), "cache": cache, "slots": torch.randperm(R, device="cuda", generator=g).to(torch.int32),
             "idx": torch.where(pos < score.shape[1], pos + base[:, None], -1).to(torch.int32),
             "q": torch.randn(n, H, D, device="cuda", generator=g).to(BF16),
             "sink": torch.randn(H, device="cuda", generator=g) if case["sink"] else None}
    return state


# ------------------------------------------------------------------ the plain form

def plain_quantise(kv, Dv):
    """Cache rows uint8 [n, row_bytes] of bf16 rows."""
    n, D = kv.shape
    rope, scales, exponent, row_bytes = layout(D, Dv)
    nb = (Dv + 15) // 16
    x = torch.nn.functional.pad(kv[:, :Dv].to(F32), (0, nb * 16 - Dv))
    fine = torch.isfinite(x).all(1, keepdim=True)
    x = torch.where(fine, x, 0.0)
    m, k = torch.frexp(x.abs().amax(1, keepdim=True))
    e = torch.where(m <= MAX_SCALED / 4096, k - 12, k - 11).clamp(E_MIN, E_MAX)
    e = torch.where(m == 0, E_MIN, e)
    x = torch.ldexp(x, -e).view(n, nb, 16).to(F64)    # quotients are met with half steps: in 64 bits
    s8 = (x.abs().amax(2) / 7).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(F64)[:, :, None]
    c = torch.where(s > 0, torch.round(x / s), 0.0).clamp(-7, 7)
    u = (c.view(n, nb * 16)[:, :Dv] + 8).to(torch.uint8).view(n, Dv // 8, 4, 2).transpose(2, 3).reshape(n, Dv // 2, 2)
    row = torch.zeros(n, row_bytes, dtype=torch.uint8, device=kv.device)
    row[:, :Dv // 2] = u[:, :, 0] | (u[:, :, 1] << 4)
    row[:, rope:rope + 2 * (D - Dv)] = kv[:, Dv:].contiguous().view(torch.uint8)
    row[:, scales:scales + nb] = s8.view(torch.uint8)
    row[:, exponent] = torch.where(fine, e + 127, 255)[:, 0].to(torch.uint8)
    return row


def plain_values(row, D, Dv):
    """The fp32 values [n, D] that cache rows stand for."""
    n = row.shape[0]
    rope, scales, exponent, _ = layout(D, Dv)
    nb = (Dv + 15) // 16
    b = row[:, :Dv // 2]
    u = torch.stack([b & 15, b >> 4], 2).view(n, Dv // 8, 2, 4).transpose(2, 3).reshape(n, Dv)
    s = row[:, scales:scales + nb].contiguous().view(torch.float8_e4m3fn).to(F32)
    e = row[:, exponent:exponent + 1].to(torch.int32)
    s = torch.where(e == 255, float("nan"), torch.ldexp(s, e - 127))
    v = (u.to(F32) - 8) * s.repeat_interleave(16, 1)[:, :Dv]
    return torch.cat([v, row[:, rope:rope + 2 * (D - Dv)].contiguous().view(BF16).to(F32)], 1)


def plain_attend(q, cache, idx, scale, Dv, sink, slots):
    n, H, D = q.shape
    used = idx >= 0
    rows = slots[idx.clamp(min=0).long()].long()
    k = plain_values(cache[rows.view(-1)], D, Dv).view(n, -1, D)
    l = torch.matmul(q.to(F32), k.transpose(1, 2)) * scale
    l = l.masked_fill(~used[:, None, :], float("-inf"))
    top = l.amax(2, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(l - top)
    den = p.sum(2, keepdim=True)
    if sink is not None:
        den = den + torch.exp(sink[None, :, None] - top)
    return torch.where(den > 0, torch.matmul(p, k[:, :, :Dv]) / den, 0.0).to(BF16)


SCALE = 192 ** -0.5


def run(state):
    case = state["case"]
    if own:
        import sparse_attention_prefill_cp_gb300 as dsa
        if case["op"] == "write":
            dsa.dsa_kv_int4_quantize(state["kv"], case["Dv"], state["cache"], slots=state["slots"])
            return dsa.dsa_kv_int4_dequantize(state["cache"], case["D"], case["Dv"])
        if case["op"] == "read":
            return dsa.dsa_kv_int4_dequantize(state["cache"], case["D"], case["Dv"], rows=state["rows"])
        return dsa.dsa_sparse_attn_int4kv(state["q"], state["cache"], state["idx"], SCALE, 512,
                                          attn_sink=state["sink"], slots=state["slots"])
    if case["op"] == "write":
        state["cache"][state["slots"].long()] = plain_quantise(state["kv"], case["Dv"])
        return plain_values(state["cache"], case["D"], case["Dv"]).to(BF16)
    if case["op"] == "read":
        rows = state["rows"].long()
        got = plain_values(state["cache"][rows.clamp(min=0)], case["D"], case["Dv"])
        return torch.where(rows[:, None] < 0, 0.0, got).to(BF16)
    return plain_attend(state["q"], state["cache"], state["idx"], SCALE, 512, state["sink"], state["slots"])


def work(case):
    if case["op"] in ("write", "read"):
        row = layout(case["D"], case["Dv"])[3]
        if case["op"] == "write":
            return {"bytes": (case["rows"] + case["cache_rows"]) * (row + 2 * case["D"]) + 4 * case["rows"], "flops": 0}
        return {"bytes": case["rows"] * (row + 2 * case["D"] + 4), "flops": 0}
    n, H, ctx, topk = case["queries"], case["H"], case["context"], case["topk"]
    if case["chunk"]:
        entries = sum(min(topk, ctx - n + 1 + i) for i in range(n))
        rows = min(entries, ctx)
    else:   # ragged lengths are log-uniform: the mean of min(topk, length)
        t = min(topk, ctx)
        mean = ((t - 1) + t * math.log(ctx / t)) / math.log(ctx) if case["ragged"] else t
        entries = rows = n * mean
    return {"bytes": rows * (layout(576, 512)[3] + 4) + n * topk * 4 + n * H * 2 * (576 + 512),
            "flops": 2 * (576 + 512) * H * entries}


# ------------------------------------------------------------------ in 64 bits, from the definition

def _e4m3_values(device):
    """The value of every E4M3 byte."""
    b = torch.arange(256, device=device)
    ex, man = (b >> 3) & 15, (b & 7).to(F64)
    mag = torch.where(ex == 0, man / 512, (1 + man / 8) * torch.exp2(ex.to(F64) - 7))
    mag = torch.where((b & 127) == 127, float("nan"), mag)
    return torch.where(b >= 128, -mag, mag)


def _decode64(row, D, Dv):
    rope, scales, exponent, _ = layout(D, Dv)
    col = torch.arange(Dv, device=row.device)
    nibble = col // 8 * 8 + (col % 8) // 2 + 4 * (col % 2)
    code = (row[:, nibble // 2].long() >> (4 * (nibble % 2))) % 16 - 8
    s = _e4m3_values(row.device)[row[:, scales + col // 16].long()]
    e = row[:, exponent:exponent + 1].to(F64)
    v = code.to(F64) * s * torch.where(e == 255, math.nan, torch.exp2(e - 127))
    return torch.cat([v, row[:, rope:rope + 2 * (D - Dv)].contiguous().view(BF16).to(F64)], 1)


def _stored64(kv, D, Dv):
    """What a latent row reads back as: every value to the nearest c * s * 2^e."""
    x = kv[:, :Dv].to(F64)
    top = x.abs().amax(1)
    e = torch.ceil(torch.log2(top / MAX_SCALED))
    e = torch.where(top > MAX_SCALED * torch.exp2(e), e + 1, e)       # log2 may have rounded
    e = torch.where(top <= MAX_SCALED * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
    grid = _e4m3_values(kv.device)[:127]
    out = torch.empty(x.shape[0], Dv, dtype=F64, device=kv.device)
    for b in range(0, Dv, 16):
        y = x[:, b:b + 16] * torch.exp2(-e)[:, None]
        want = y.abs().amax(1) / 7
        hi = torch.searchsorted(grid, want).clamp(1, 126)
        lo = hi - 1
        down, up = want - grid[lo], grid[hi] - want
        pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
        s = grid[pick][:, None]
        c = torch.where(s > 0, torch.round(y / s), 0.0).clamp(-7, 7)
        out[:, b:b + 16] = c * s * torch.exp2(e)[:, None]
    return torch.cat([out, kv[:, Dv:].to(F64)], 1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        out = _decode64(state["cache"], case["D"], case["Dv"])
        out[state["slots"].long()] = _stored64(state["kv"], case["D"], case["Dv"])
        return out
    if case["op"] == "read":
        rows = state["rows"].long()
        out = _decode64(state["cache"], case["D"], case["Dv"])[rows]
        out[rows < 0] = 0
        return out
    outs = []
    for i in range(0, case["queries"], 64):      # a few queries at a time
        idx = state["idx"][i:i + 64].long()
        k = _decode64(state["cache"][state["slots"][idx.clamp(min=0)].long().view(-1)], 576, 512)
        k = k.view(idx.shape[0], -1, 576)
        l = torch.einsum("nhd,nsd->nhs", state["q"][i:i + 64].to(F64), k) * SCALE
        l = torch.where(idx[:, None, :] >= 0, l, -math.inf)
        if state["sink"] is not None:
            sink = state["sink"].to(F64)[None, :, None].expand(l.shape[0], -1, 1)
            p = torch.softmax(torch.cat([l, sink], 2), 2)[:, :, :-1]
        else:
            p = torch.nan_to_num(torch.softmax(l, 2), nan=0.0)
        outs.append(torch.einsum("nhs,nsd->nhd", p, k[:, :, :512]))
    return torch.cat(outs)
