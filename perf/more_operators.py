"""Serving from a paged latent-KV cache: its page tables, writing rows, choosing blocks, and attending.

Cases of four operators.  ``pages``: the page table of a batch grown to new lengths out of a list of free pages, the
slots that its new rows get, and the pages given back.  ``append``: latent rows and index keys written to their slots,
and the mean key of every page that they complete.  ``select``: for every query the pages worth reading, by the
lightning-indexer score of the pages' mean keys.  ``attend``: MLA attention of every query head over its request's
paged rows, all of them or those of the selected pages.  Where ``own`` is false the operators are computed in their
plain form; where it is true they are the framework's entry points.

A page holds P rows; position p of request b lies in slot page_table[b][p // P] * P + p % P of the cache.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
D, DV, HI, DI = 576, 512, 64, 128
SCALE = 192 ** -0.5


def pages_of(n, P):
    return (n + P - 1) // P


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: every request grows by a token, a few by a page
        {"name": "pages_step_64", "op": "pages", "requests": 64, "context": 8192, "grow": 1, "P": 64},
        # a mixed prompt batch admitted at once (184,265 tokens in the framework's own batch of 16 requests)
        {"name": "pages_admit_16", "op": "pages", "requests": 16, "context": 32768, "grow": 0, "P": 64},
        # one new token of each request of a decode batch
        {"name": "append_61", "op": "append", "rows": 61, "requests": 61, "P": 64, "stride": 576},
        # a prefill chunk of one request; the latent is a slice of a wider projection output
        {"name": "append_8000", "op": "append", "rows": 8000, "requests": 1, "P": 64, "stride": 2112},
        # a decode batch of long requests: 1,024 blocks each, 32 chosen
        {"name": "select_64", "op": "select", "queries": 64, "requests": 64, "context": 65536, "P": 64, "nsel": 32,
         "ragged": False},
        # a prefill chunk at the end of a long request
        {"name": "select_chunk_2048", "op": "select", "queries": 2048, "requests": 1, "context": 65536, "P": 64,
         "nsel": 32, "ragged": False},
        # one token of one long request, all heads on one GPU
        {"name": "attend_1", "op": "attend", "queries": 1, "requests": 1, "context": 65536, "P": 64, "H": 128,
         "nsel": 0, "ragged": False, "sink": False},
        # a small decode batch with short and empty contexts in small pages, a tensor-parallel rank's heads
        {"name": "attend_7_ragged", "op": "attend", "queries": 7, "requests": 7, "context": 8000, "P": 16, "H": 32,
         "nsel": 0, "ragged": True, "sink": True},
        # a decode batch, 16 heads per rank; the cache is larger than the L2
        {"name": "attend_64_h16", "op": "attend", "queries": 64, "requests": 64, "context": 8192, "P": 64, "H": 16,
         "nsel": 0, "ragged": False, "sink": False},
        # a decode batch, all heads on one GPU
        {"name": "attend_64", "op": "attend", "queries": 64, "requests": 64, "context": 8192, "P": 64, "H": 128,
         "nsel": 0, "ragged": False, "sink": True},
        # a decode batch of long and short requests, each token reading 32 blocks
        {"name": "attend_blocks_64", "op": "attend", "queries": 64, "requests": 64, "context": 16384, "P": 64,
         "H": 128, "nsel": 32, "ragged": True, "sink": False},
        # a prefill chunk, every token reading the 32 blocks that it chose
        {"name": "attend_blocks_2048", "op": "attend", "queries": 2048, "requests": 1, "context": 8192, "P": 64,
         "H": 128, "nsel": 32, "ragged": False, "sink": True},
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of lo..hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "select", "attend", "attend", "attend"])
    P = rng.choice([16, 32, 64, 64, 128])
    if op == "pages":
        requests = _spread(rng, 1, 300)
        return {"op": op, "requests": requests, "context": _spread(rng, 16, 400000 // requests + 16),
                "grow": rng.choice([0, 1, rng.randint(2, 100)]), "P": P}
    if op == "append":
        rows = _spread(rng, 1, 9000)
        requests = rng.choice([1, rng.randint(1, min(rows, 64)), rows if rows <= 500 else 3])
        return {"op": op, "rows": rows, "requests": min(requests, rows), "P": P, "stride": D + 8 * rng.randint(0, 190)}
    if op == "select":
        queries = _spread(rng, 1, 1500)
        requests = rng.choice([1, queries]) if queries <= 64 else 1
        context = max(_spread(rng, 32 * P, 40000), queries)
        return {"op": op, "queries": queries, "requests": requests, "context": context, "P": P,
                "nsel": rng.randint(8, min(64, context // P // 2)), "ragged": requests > 1 and rng.random() < 0.5}
    nsel = rng.choice([0, 0, rng.randint(1, 2048 // P)])
    queries = _spread(rng, 1, 64 if not nsel else 600)
    requests = rng.choice([1, queries, max(1, queries // 2)]) if queries <= 64 else 1
    context = max(_spread(rng, 1, 12000), queries)
    return {"op": op, "queries": queries, "requests": requests, "context": context, "P": P,
            "H": rng.choice([8, 16, 24, 32, 64, 128, 128, rng.randint(1, 128)]), "nsel": nsel,
            "ragged": requests > 1 and rng.random() < 0.6, "sink": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return x.to(torch.int32)


def _perm(n, g):
    return torch.randperm(n, device="cuda", generator=g)


def _log_uniform(n, top, g):
    """n lengths spread evenly over the logarithm of 1..top, in random order, the longest last."""
    u = torch.arange(1, n + 1, device="cuda") / n
    lens = torch.exp(u * math.log(max(top, 1))).round().clamp(1, top).long()
    return torch.cat([lens[:-1][_perm(n - 1, g)], lens[-1:]])


def _rows(n, d, g):
    """Latent rows as a normalised latent has them, N(0, 1) with a spread of row magnitudes."""
    x = torch.randn(n, d, device="cuda", generator=g)
    return (x * torch.exp(0.3 * torch.randn(n, 1, device="cuda", generator=g))).to(BF16)


def _grid(shape, std, step, g):
    """Normal values rounded to multiples of ``step``, as index operands held in 8 bits have them: sums of their
    products are exact in 32 bits in any order, and equal scores do occur."""
    return (torch.randn(*shape, device="cuda", generator=g) * (std / step)).round().clamp(-127, 127) * step


def _requests(case, g):
    """Lengths of the requests, their page table over a pool in random order, the pool's size."""
    B, ctx, P = case["requests"], case["context"], case["P"]
    lens = torch.full((B,), ctx, device="cuda")
    if case["ragged"]:
        lens = _log_uniform(B, ctx, g)
        lens[0] = 0
    width = pages_of(ctx, P)
    pool = B * width
    table = _perm(pool, g).view(B, width)
    table = torch.where(torch.arange(width, device="cuda") < pages_of(lens, P)[:, None], table, -1)
    return lens, table, pool


def _queries(case, lens):
    """Request and visible length of every query: the last tokens of its request (a request may be shorter)."""
    n, B = case["queries"], case["requests"]
    per = (n + B - 1) // B
    i = torch.arange(n, device="cuda")
    req = (i // per).clamp(max=B - 1)
    back = per - 1 - (i - req * per)
    return req, (lens[req] - back).clamp(min=0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, P = case["op"], case["P"]
    state = {"case": dict(case)}
    if op == "pages":
        B, ctx = case["requests"], case["context"]
        seq = _log_uniform(B, ctx, g)
        held = (seq - case["grow"]).clamp(min=0) if case["grow"] else torch.zeros_like(seq)
        width = pages_of(ctx, P) + 2
        used = pages_of(held, P)
        pool = int(pages_of(seq, P).sum()) + 32
        order = _perm(pool, g)
        col = torch.arange(width, device="cuda")
        mine = col[None, :] < used[:, None]
        k = (torch.cumsum(mine.view(-1).long(), 0) - 1).view(B, width)
        taken = int(used.sum())
        state.update(held=_i32(held), seq=_i32(seq), table=_i32(torch.where(mine, order[k.clamp(min=0)], -1)),
                     free=_i32(torch.cat([order[taken:], torch.zeros(taken, dtype=torch.long, device="cuda")])),
                     count=torch.full((1,), pool - taken, dtype=torch.int32, device="cuda"),
                     rows=int((seq - held).sum()))
        return state
    if op == "append":
        n, B = case["rows"], case["requests"]
        per = torch.full((B,), n // B, device="cuda")
        per[:n - n // B * B] += 1
        first = torch.randint(0, 4 * P, (B,), device="cuda", generator=g)
        width = pages_of(4 * P + n // B + 1, P)
        table = _perm(B * width, g).view(B, width)
        start = torch.cumsum(per, 0) - per
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), per, output_size=n)
        pos = first[req] + torch.arange(n, device="cuda") - start[req]
        pool = B * width
        wide = _rows(n, case["stride"], g)
        off = (case["stride"] - D) // 16 * 8      # the latent's columns of the wider tensor
        state.update(kv=wide[:, off:off + D], k_idx=torch.randn(n, DI, device="cuda", generator=g).to(BF16),
                     slots=_i32(table[req, pos // P] * P + pos % P),
                     cache=_rows(pool * P, D, g).view(pool, P, D),
                     keys=torch.randn(pool, P, DI, device="cuda", generator=g).to(BF16),
                     block_keys=torch.zeros(pool, DI, dtype=BF16, device="cuda"))
        return state
    lens, table, pool = _requests(case, g)
    req, seen = _queries(case, lens)
    state.update(table=_i32(table), req=_i32(req), lens=_i32(seen))
    if case["queries"] == case["requests"]:
        state["req"] = None                       # every query has a request of its own
    if op == "select":
        n = case["queries"]
        state.update(q=_grid((n, HI, DI), 1.0, 0.25, g).to(BF16), w=_grid((n, HI), HI ** -0.5, 1 / 32, g),
                     block_keys=_grid((pool, DI), 0.5, 1 / 32, g).to(BF16))
        return state
    n, nsel, H = case["queries"], case["nsel"], case["H"]
    cache = torch.cat([_rows(min(1 << 18, pool * P - r), D, g) for r in range(0, pool * P, 1 << 18)]).view(pool, P, D)
    # rows behind a request's last one hold whatever memory held
    last = table.gather(1, (pages_of(lens, P) - 1).clamp(min=0)[:, None])[:, 0]
    tail = (lens % P != 0) & (last >= 0)
    for b in torch.nonzero(tail)[:, 0].tolist()[:64]:
        cache[int(last[b]), int(lens[b]) % P:] = math.nan
    state.update(cache=cache, q=torch.randn(n, H, D, device="cuda", generator=g).to(BF16),
                 sink=torch.randn(H, device="cuda", generator=g) if case["sink"] else None, blocks=None)
    if nsel:
        width = table.shape[1]
        have = pages_of(seen, P)[:, None]
        col = torch.arange(width, device="cuda")
        score = torch.rand(n, width, device="cuda", generator=g)
        score = torch.where((col == 0) | (col == have - 1), 2.0, score).masked_fill(col >= have, -1.0)
        if width < nsel:
            score = torch.nn.functional.pad(score, (0, nsel - width), value=-1.0)
        val, at = score.topk(nsel, dim=1)
        at = torch.where(val < 0, 1 << 30, at).sort(dim=1).values
        state["blocks"] = _i32(torch.where(at < 1 << 30, at, -1))
    return state


# ------------------------------------------------------------------ the plain form

def plain_update(table, held, seq, free, count, P):
    """Pages taken and given back, in place."""
    had, need = pages_of(held.long(), P), pages_of(seq.long(), P)
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    gone, new = (col >= need[:, None]) & (col < had[:, None]), (col >= had[:, None]) & (col < need[:, None])
    nth = lambda m: torch.cumsum(m.reshape(-1).long(), 0).view(m.shape) - 1
    R, G, c = gone.sum(), new.sum(), count.long()
    at = torch.where(gone, c + R - 1 - nth(gone), free.numel())
    pool = torch.cat([free, free.new_zeros(1)]).scatter(0, at.view(-1), table.reshape(-1))[:-1]
    taken = pool[torch.where(new, c + R - 1 - nth(new), 0)]
    table.copy_(torch.where(new, taken, torch.where(gone, -1, table)))
    free.copy_(pool)
    count.add_(_i32(R - G))


def plain_slots(table, first, seq, P, n):
    per = (seq - first).long()
    end = torch.cumsum(per, 0)
    t = torch.arange(n, device=table.device)
    b = torch.searchsorted(end, t, right=True)
    inside = b < seq.numel()
    b = b.clamp(max=seq.numel() - 1)
    pos = first[b].long() + t - (end - per)[b]
    page = table[b, torch.where(inside, pos // P, 0)].long()
    return _i32(torch.where(inside & (page >= 0), page * P + pos % P, -1))


def plain_append(kv, k_idx, slots, cache, keys, block_keys):
    P = cache.shape[1]
    s = slots.long()
    cache.view(-1, D)[s] = kv
    keys.view(-1, DI)[s] = k_idx
    page = s // P
    mean = (keys[page].to(F32).sum(1) / P if page.numel() <= 4096 else
            torch.cat([keys[p].to(F32).sum(1) / P for p in page.split(4096)]))
    done = s % P == P - 1
    # pages that got no last row keep their key: written to a row behind the others
    grown = torch.cat([block_keys, block_keys.new_zeros(1, DI)])
    grown[torch.where(done, page, block_keys.shape[0])] = mean.to(BF16)
    block_keys.copy_(grown[:-1])


def plain_select(q, w, block_keys, table, lens, req, P, nsel, keep_first=1, keep_last=1):
    out = []
    for i in range(0, q.shape[0], 64):
        t = table[i:i + 64] if req is None else table[req[i:i + 64].long()]
        t = t.long()
        have = pages_of(lens[i:i + 64].long(), P)[:, None]
        col = torch.arange(t.shape[1], device=t.device)
        if req is None:
            dots = torch.einsum("nhd,nbd->nhb", q[i:i + 64].to(F32), block_keys[t.clamp(min=0)].to(F32))
        else:                                     # the queries of one request share its keys
            b = req[i:i + 64].long()
            rows = block_keys[table[b[0]].long().clamp(min=0)].to(F32)
            dots = torch.matmul(q[i:i + 64].to(F32), rows.T)
            for r in range(int(b[0]) + 1, int(b[-1]) + 1):
                rows = block_keys[table[r].long().clamp(min=0)].to(F32)
                dots = torch.where((b == r)[:, None, None], torch.matmul(q[i:i + 64].to(F32), rows.T), dots)
        score = (dots.clamp(min=0) * w[i:i + 64, :, None]).sum(1)
        score = torch.where((col < keep_first) | (col >= have - keep_last), math.inf, score)
        score = torch.where(col < have, score, -math.inf)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :nsel]
        order = torch.where(order < have, order, 1 << 30).sort(dim=1).values
        order = torch.nn.functional.pad(order, (0, max(0, nsel - order.shape[1])), value=1 << 30)
        out.append(_i32(torch.where(order < 1 << 30, order, -1)))
    return torch.cat(out)


def plain_attend(q, cache, table, lens, req, blocks, sink):
    n, H, _ = q.shape
    P = cache.shape[1]
    out = []
    width = table.shape[1] if blocks is None else blocks.shape[1]
    step = max(1, (1 << 20) // (width * P))
    for i in range(0, n, step):
        t = (table[i:i + step] if req is None else table[req[i:i + step].long()]).long()
        b = torch.arange(width, device=q.device).expand(t.shape[0], -1) if blocks is None else blocks[i:i + step].long()
        page = torch.where(b >= 0, t.gather(1, b.clamp(min=0)), -1)
        pos = (b[:, :, None] * P + torch.arange(P, device=q.device)).view(t.shape[0], -1)
        used = (pos < lens[i:i + step, None]) & (pos >= 0) & (page >= 0).repeat_interleave(P, 1)
        k = cache[page.clamp(min=0)].view(t.shape[0], -1, D).to(F32).masked_fill(~used[:, :, None], 0.0)
        l = torch.matmul(q[i:i + step].to(F32), k.transpose(1, 2)) * SCALE
        l = l.masked_fill(~used[:, None, :], -math.inf)
        top = l.amax(2, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(l - top)
        den = p.sum(2, keepdim=True)
        some = den > 0
        if sink is not None:
            den = den + torch.exp(sink[None, :, None] - top)
        out.append(torch.where(some, torch.matmul(p, k[:, :, :DV]) / den, 0.0).to(BF16))
    return torch.cat(out)


def run(state):
    case = state["case"]
    P = case["P"]
    if case["op"] == "pages":
        # a step and its end: the new rows' pages are taken, named, and given back
        table, held, seq, free, count = (state[k] for k in ("table", "held", "seq", "free", "count"))
        if own:
            import sparse_attention_prefill_cp_gb300 as dsa
            dsa.dsa_pages_update(table, held, seq, free, count, P)
            slots = dsa.dsa_pages_slots(table, held, seq, P, state["rows"])
            dsa.dsa_pages_update(table, seq, held, free, count, P)
        else:
            plain_update(table, held, seq, free, count, P)
            slots = plain_slots(table, held, seq, P, state["rows"])
            plain_update(table, seq, held, free, count, P)
        return slots, table, free, count
    if case["op"] == "append":
        args = [state[k] for k in ("kv", "k_idx", "slots", "cache", "keys", "block_keys")]
        if own:
            import sparse_attention_prefill_cp_gb300 as dsa
            dsa.dsa_pages_append(*args)
        else:
            plain_append(*args)
        return tuple(args[3:])
    if case["op"] == "select":
        if own:
            import sparse_attention_prefill_cp_gb300 as dsa
            return dsa.dsa_block_select(state["q"], state["w"], state["block_keys"], state["table"], state["lens"], P,
                                        case["nsel"], req=state["req"])
        return plain_select(state["q"], state["w"], state["block_keys"], state["table"], state["lens"], state["req"], P,
                            case["nsel"])
    if own:
        import sparse_attention_prefill_cp_gb300 as dsa
        return dsa.dsa_paged_attn(state["q"], state["cache"], state["table"], state["lens"], SCALE, DV,
                                  blocks=state["blocks"], req=state["req"], attn_sink=state["sink"])
    return plain_attend(state["q"], state["cache"], state["table"], state["lens"], state["req"], state["blocks"],
                        state["sink"])


def _lengths(case):
    """Mean and sum over the requests of their lengths (ragged ones are log-uniform, the first empty)."""
    ctx = case["context"]
    mean = ctx / max(math.log(ctx), 1.0) if case.get("ragged") else ctx
    return mean, mean * case["requests"]


def work(case):
    op, P = case["op"], case["P"]
    if op == "pages":
        B, ctx = case["requests"], case["context"]
        mean = ctx / max(math.log(ctx), 1.0)      # log-uniform lengths
        rows = B * (min(case["grow"], mean) if case["grow"] else mean)
        pages = rows / P
        # twice the lengths and the pages taken or given back (free list and table), and a slot for every row
        return {"bytes": 2 * (8 * B + 12 * pages) + 4 * rows + 8 * B, "flops": 0}
    if op == "append":
        n = case["rows"]
        # a page's key costs its page's keys and the key itself; most of them are this call's own rows
        keys = n / P * (2 * DI + (2 * DI * P if n < case["requests"] * P else 0))
        # the caches come back whole, but what no slot names is not touched
        return {"bytes": n * (2 * (2 * D + 2 * DI) + 4) + keys, "flops": n * DI}
    n = case["queries"]
    if op == "select":
        mean, total = _lengths(case)
        return {"bytes": total / P * (2 * DI + 4) + n * (2 * HI * DI + 4 * HI + 4 * case["nsel"]),
                "flops": 2 * HI * DI * n * mean / P}
    H, ctx = case["H"], case["context"]
    mean, total = _lengths(case)
    per = mean
    if case["nsel"]:
        t = min(case["nsel"] * P, ctx)
        per = t if not case["ragged"] else ((t - 1) + t * math.log(ctx / t)) / max(math.log(ctx), 1.0)
        if not case["ragged"] and case["requests"] < n:    # a chunk's early queries see less
            per = min(t, ctx - n / case["requests"] / 2)
        total = min(total, n * per)
    return {"bytes": total * (2 * D + 4 / P) + n * (2 * H * (D + DV) + 4 * case["nsel"] + 4),
            "flops": 2 * (D + DV) * H * n * per}


# ------------------------------------------------------------------ in 64 bits, from the definition

def exact(case, seed):
    state = prepare(case, seed)
    op, P = case["op"], case["P"]
    dev = "cuda"
    if op == "pages":
        table, held, seq = state["table"].tolist(), state["held"].tolist(), state["seq"].tolist()
        free, count = state["free"].tolist(), int(state["count"])
        slots = []
        for b in range(len(seq)):
            for k in range(-(-held[b] // P), -(-seq[b] // P)):
                count -= 1
                table[b][k] = free[count]
            slots += [table[b][p // P] * P + p % P for p in range(held[b], seq[b])]
        # given back: the list is as it was, the table too
        return (torch.tensor(slots, dtype=torch.int32, device=dev), state["table"], state["free"], state["count"])
    if op == "append":
        cache, keys = state["cache"].to(F64), state["keys"].to(F64)
        means = state["block_keys"].to(F64)
        slots = state["slots"].tolist()
        at = torch.tensor(slots, device=dev)
        cache.view(-1, D)[at] = state["kv"].to(F64)
        keys.view(-1, DI)[at] = state["k_idx"].to(F64)
        ended = [s // P for s in slots if (s + 1) % P == 0]
        if ended:
            means[ended] = keys[ended].mean(1)
        return cache, keys, means
    lens, n = state["lens"].tolist(), case["queries"]
    req = list(range(n)) if state["req"] is None else state["req"].tolist()
    if op == "select":
        out = torch.full((n, case["nsel"]), -1, dtype=torch.int32, device=dev)
        for b in range(case["requests"]):
            mine = [i for i in range(n) if req[i] == b]
            have = [-(-lens[i] // P) for i in mine]
            if not mine or max(have) == 0:
                continue
            k = state["block_keys"][state["table"][b, :max(have)].long()].to(F64)
            for i0 in range(0, len(mine), 64):
                part = mine[i0:i0 + 64]
                s = torch.einsum("nhd,bd->nhb", state["q"][part].to(F64), k).relu()
                s = torch.einsum("nhb,nh->nb", s, state["w"][part].to(F64)).tolist()
                for row, i, m in zip(s, part, have[i0:i0 + 64]):
                    kept = {0, m - 1} if m else set()
                    rest = sorted((x for x in range(m) if x not in kept), key=lambda x: (-row[x], x))
                    chosen = sorted(list(sorted(kept)) + rest[:max(0, case["nsel"] - len(kept))])[:case["nsel"]]
                    out[i, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        return out
    H = case["H"]
    out = torch.zeros(n, H, DV, dtype=F64, device=dev)
    blocks = None if state["blocks"] is None else state["blocks"].tolist()
    flat = state["cache"].view(-1, D)
    shared = None                                 # (request, its rows in 64 bits)
    for i in range(n):
        if lens[i] == 0:
            continue
        if blocks is None:
            pos = torch.arange(lens[i], device=dev)
        else:
            pos = torch.tensor([b for b in blocks[i] if b >= 0], device=dev)
            pos = (pos[:, None] * P + torch.arange(P, device=dev)).view(-1)
            pos = pos[pos < lens[i]]
        if shared is None or shared[0] != req[i]:
            have = -(-max(l for l, r in zip(lens, req) if r == req[i]) // P)
            p = torch.arange(have * P, device=dev)
            shared = (req[i], flat[state["table"][req[i], p // P].long() * P + p % P].to(F64))
        k = shared[1][pos]
        l = torch.matmul(state["q"][i].to(F64), k.T) * SCALE
        if state["sink"] is not None:
            l = torch.cat([l, state["sink"].to(F64)[:, None]], 1)
        p = torch.softmax(l, 1)[:, :pos.numel()]
        out[i] = torch.matmul(p, k[:, :DV])
    return out
