"""The paged latent cache at the borders of what its calls allow."""
import glob
import os

import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from conftest import ROOT
from oracle import dsa_oracle as O
from sparse_attention_prefill_cp_gb300 import _lib
from test_paged_gpu import D, DV, INF, NAN, SCALE, attend64, bounds, gen, grid, i32, near, paged, randn

CSRC = os.path.join(ROOT, "sparse_attention_prefill_cp_gb300", "csrc")
A = 0x10000     # an aligned address, never read


@pytest.fixture(autouse=True)
def _gpu(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    dsa.dsa_poll_device_error()


# ------------------------------------------------------------------ kernels launched while the one before still runs

def test_overlapped_kernels_read_with_plain_loads():
    """A kernel that is there while its inputs are still being written may not read them as data that nobody writes."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path, encoding="utf-8").read()
        if "launch_overlapped(" not in text:
            continue
        seen += 1
        assert "griddepcontrol.wait" in text, path
        for form in ("__ldg(", "ld.global.nc"):
            assert form not in text, f"{os.path.basename(path)} reads with {form}"
    assert seen >= 4

# ------------------------------------------------------------------ rows in any order

@pytest.mark.gpu
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("rows", [300, 3000])
def test_rows_in_any_order_make_the_same_keys(P, rows):
    # one call in order, in a random order with rows that have no slot between, and token by token over several requests
    pages, DI = -(-rows // P) + 4, 128
    kv, ki = randn(rows, D, seed=1).cuda(), randn(rows, DI, seed=2).cuda()
    slots = torch.randperm(pages, generator=gen(P))[torch.arange(rows) // P] * P + torch.arange(rows) % P
    half = slots % P < 5                             # the first rows of every page are there before

    def write(order, before=None):
        cache = torch.zeros(pages, P, D, dtype=torch.bfloat16, device="cuda")
        keys = torch.zeros(pages, P, DI, dtype=torch.bfloat16, device="cuda")
        means = torch.zeros(pages, DI, dtype=torch.bfloat16, device="cuda")
        for part in ([] if before is None else [before]) + [order]:
            # an odd start, so that the list begins off a 16-byte boundary
            s = torch.cat([torch.full((1,), -1), torch.where(part >= 0, slots[part.clamp(min=0)], -1)]).int().cuda()[1:]
            at = part.clamp(min=0).cuda()
            dsa.dsa_pages_append(kv[at], ki[at], s, cache, keys, means)
        return cache, keys, means

    every = torch.arange(rows)
    want = write(every)
    assert want[2].any(1).sum() == rows // P
    shuffled = every[torch.randperm(rows, generator=gen(3))]
    holes = torch.full((2 * rows + 3,), -1)
    holes[torch.randperm(2 * rows + 3, generator=gen(4))[:rows].sort().values] = shuffled
    per = rows // 4                                  # four requests, a token of each by turns
    turns = torch.cat([every[:4 * per].view(4, per).t().reshape(-1), every[4 * per:]])
    for order, before in ((shuffled, None), (every.flip(0), None), (holes, None), (turns, None),
                          (every[~half], every[half]), (every[~half].flip(0), every[half])):
        got = write(order, before)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ attention over chosen pages

def attend_lists(lists, lens, have, P, H, req=None):
    """The attention over these lists of pages against the one in 64 bits."""
    cache, table, rows = paged(have, P, seed=P + H)
    q, sink = randn(len(lens), H, D, seed=H), torch.randn(H, generator=gen(6))
    blocks = torch.tensor(lists, dtype=torch.int32)
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, blocks=blocks.cuda(),
                             req=None if req is None else i32(req), attn_sink=sink.cuda())
    near(got, *attend64(q, rows, lens, req, lists, P, sink))
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("H", [16, 32, 128])
def test_pages_that_a_query_does_not_see_name_nothing(P, H):
    # more entries than pages: some of pages behind the query's last ahead of those that it sees, negative ones between
    have = [10 * P] * 4
    got = attend_lists([[3, 9, 8, 7, 6, 5, 4, 2, 1, 0, -1, -1], [9, 0, -1, 8, 1, -1, -1, 7, -5, 6, 2, 5],
                        [-1] * 11 + [0], [4, -1, 3, -1, 2, 9, 8, 7, 6, -1, -1, 5]],
                       [P - 3, 2 * P + 1, 1, 5 * P], have, P, H)
    assert all(got[i].any() for i in range(4))
    # as many entries as pages, or fewer
    got = attend_lists([[9, 1], [-1, 2], [5, 0], [9, 8]], [2 * P, 3 * P, P - 1, 2 * P], have, P, H)
    assert not got[3].any()


@pytest.mark.gpu
@pytest.mark.parametrize("P,nsel", [(16, 70), (32, 33), (64, 9)])
def test_a_list_shared_by_a_chunk(P, nsel):
    # every query sees more than the one before, all have the same list, in falling order
    n, have = 90, 70 * P + 5
    pages = -(-have // P)
    chosen = torch.randperm(pages, generator=gen(nsel))[:nsel].sort(descending=True).values.tolist()
    lens = [1 + i * (have - 1) // (n - 1) for i in range(n)]
    attend_lists([chosen] * n, lens, [have], P, 24, req=[0] * n)


# ------------------------------------------------------------------ choosing among pages that are none

def select(lens, table, keys, nsel, q=None, w=None, **kw):
    n = len(lens)
    q = grid(n, 64, 128, std=1, step=0.25, seed=2) if q is None else q
    w = grid(n, 64, std=0.125, step=1 / 32, seed=3).abs() if w is None else w
    return dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(),
                                i32(lens), 16, nsel, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [-1, 40])
@pytest.mark.parametrize("queries", [1, 400])
def test_a_page_that_is_none_is_reported_where_all_are_taken(page, queries):
    # no more pages than a list takes, so none is scored; alone, and among queries that share the request
    width, nsel = 6, 8
    keys = grid(40, 128, std=0.5, step=1 / 32, seed=4)
    table = torch.arange(2 * width, dtype=torch.int32).view(2, width)
    req = [0] * (queries // 2) + [1] * (queries - queries // 2)
    lens, want = [16 * width - 3] * queries, i32([0, 1, 2, 3, 4, 5, -1, -1])
    got = select(lens, table, keys, nsel, req=i32(req))
    dsa.dsa_poll_device_error()
    assert (got == want).all()
    table[1, 4] = page
    select([16 * 4] * queries, table, keys, nsel, req=i32(req))
    dsa.dsa_poll_device_error()                      # behind what the queries see
    got = select(lens, table, keys, nsel, req=i32(req))
    assert bounds(57) >= queries // 2
    assert (got == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("queries", [1, 400])
def test_a_page_that_is_none_ranks_behind_scores_that_are_no_numbers(queries):
    width, nsel = 12, 6
    keys = grid(40, 128, std=0.5, step=1 / 32, seed=4)
    keys[5:width - 1] = NAN                          # of pages 1 .. 10 four have a score
    table = torch.arange(width, dtype=torch.int32)[None].clone()
    table[0, 1:4] = torch.tensor([-1, 40, -7])       # pages 1 to 3 are none: one score is left
    got = select([16 * width] * queries, table, keys, nsel, req=i32([0] * queries))
    bounds(57)
    assert (got == i32([0, 4, 5, 6, 7, 11])).all()


@pytest.mark.gpu
def test_forced_pages_are_taken_whatever_they_are():
    width, nsel = 12, 4
    keys = grid(40, 128, std=0.5, step=1 / 32, seed=4)
    table = torch.arange(width, dtype=torch.int32)[None].clone()
    table[0, 0] = 40
    keys[11] = NAN
    got = select([16 * width], table, keys, nsel)
    assert bounds(57) == 0
    q, w = grid(1, 64, 128, std=1, step=0.25, seed=2), grid(1, 64, std=0.125, step=1 / 32, seed=3).abs()
    score = (w[0].double()[:, None] * (q[0].double() @ keys[:width].double().T).clamp(min=0)).sum(0)
    best = sorted(range(1, 11), key=lambda b: (-score[b].item(), b))[:2]
    assert got[0].tolist() == [0] + sorted(best) + [11]


@pytest.mark.gpu
@pytest.mark.parametrize("queries", [3, 400])
@pytest.mark.parametrize("HI", [1, 5, 16, 33, 48, 63, 64])
def test_infinite_keys_with_any_number_of_index_heads(HI, queries):
    # the score of a page with an infinite key is infinite (or no number), whatever the number of heads
    width, nsel = 150, 5
    keys = grid(width, 128, std=0.5, step=1 / 32, seed=4)
    q = grid(1, HI, 128, std=1, step=0.25, seed=2)
    q[0, :, 7] = 1.0
    w = grid(1, HI, std=0.125, step=1 / 32, seed=3).abs() + 1 / 32
    keys[9, 7], keys[140, 7] = INF, INF              # the highest scores
    keys[3, 7] = -INF                                # relu(-inf) = 0: the lowest
    q[0, 0, 8] = 0.0
    keys[11, 8] = INF                                # 0 * inf: no number
    s = (w[0].double()[:, None] * (q[0].double() @ keys.double().T).clamp(min=0)).sum(0)
    assert s[9] == s[140] == INF and s[3] == 0 and torch.isnan(s[11])
    rest = sorted((b for b in range(1, width - 1) if not torch.isnan(s[b])), key=lambda b: (-s[b].item(), b))
    want = sorted([0, width - 1] + rest[:nsel - 2])
    table = torch.arange(width, dtype=torch.int32)[None]
    got = select([16 * width] * queries, table, keys, nsel, q=q.expand(queries, -1, -1).contiguous(),
                 w=w.expand(queries, -1).contiguous(), req=i32([0] * queries))
    assert (got == i32(want)).all()


# ------------------------------------------------------------------ lengths that are no lengths

@pytest.mark.gpu
def test_a_length_below_zero_counts_as_zero_whatever_the_first_position():
    table = i32([[0, 1], [2, 3], [4, 5]])
    for first, length in ((2 ** 31 - 1, -2), (2 ** 31 - 1, -2 ** 31), (1, -2 ** 31), (-2 ** 31, -2 ** 31), (2 ** 31 - 1, 5)):
        got = dsa.dsa_pages_slots(table, i32([0, first, 1]), i32([2, length, 3]), 16, 6).tolist()
        if length < 0 or first < 0:
            assert bounds(52) == 1
        assert got == [0, 1, 65, 66, -1, -1]


@pytest.mark.gpu
def test_as_many_rows_as_a_call_may_have():
    # 2^31 - 1 rows, of which four have a slot
    n, P = 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("needs 50 GB")
    kv = torch.empty(n, 8, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    cache = torch.zeros(2, P, 8, dtype=torch.bfloat16, device="cuda")
    want = torch.zeros(2, P, 8, dtype=torch.bfloat16)
    for k, (at, slot) in enumerate(((0, 3), (7, 17), (n - 8, 31), (n - 1, 0))):
        x = randn(8, seed=k)
        kv[at], slots[at] = x.cuda(), slot
        want.view(-1, 8)[slot] = x
    dsa.dsa_pages_append(kv, None, slots, cache)
    assert torch.equal(cache.cpu(), want)
    del kv, slots
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the example of a step

@pytest.mark.gpu
def test_the_example_of_a_step_gives_back_every_page():
    """README's example as it stands: after its last call the pages of the requests that stay and the free ones are all
    there are."""
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    code = next(b for b in text.split("```python\n")[1:] if "dsa_pages_update" in b).split("```")[0]
    batch, P, num_pages, max_pages = 4, 64, 40, 8
    held, new, left = [0, 63, 64, 130], [100, 64, 65, 131], [0, 64, 0, 131]
    rows = sum(new) - sum(held)
    req = [b for b in range(batch) for _ in range(new[b] - held[b])]
    seen = [p + 1 for b in range(batch) for p in range(held[b], new[b])]
    bf16 = lambda *shape, seed: randn(*shape, seed=seed).cuda()
    at = code.index("dsa.dsa_pages_update")
    env = dict(torch=torch, dsa=dsa, batch=batch, num_pages=num_pages, max_pages=max_pages, new_rows=rows,
               held_lens=i32(held), seq_lens=i32(new), remaining_lens=i32(left), lens=i32(seen), req=i32(req),
               kv=bf16(rows, D, seed=1), k_idx=bf16(rows, 128, seed=2), q=bf16(rows, 128, D, seed=3),
               q_idx=bf16(rows, 64, 128, seed=4), w=torch.randn(rows, 64, device="cuda"), sink=torch.zeros(128, device="cuda"))
    exec(code[:at], env)
    zero = i32([0] * batch)
    dsa.dsa_pages_update(env["table"], zero, env["held_lens"], env["free"], env["count"], P)
    for name in ("cache", "key_cache", "block_keys"):
        env[name].zero_()
    exec(code[at:], env)
    dsa.dsa_poll_device_error()
    owned = [page for row, n in zip(env["table"].tolist(), left) for page in row[:-(-n // P)]]
    assert sorted(owned + env["free"].tolist()[:env["count"].item()]) == list(range(num_pages))
    assert (env["table"] >= 0).sum().item() == len(owned)


# ------------------------------------------------------------------ every kernel that a call may take

def oracle_choice(i, q, w, keys, row, length, P, nsel):
    return O.block_select(q[i].numpy(), w[i].numpy(), keys.numpy(), row, length, P, nsel)


@pytest.mark.gpu
@pytest.mark.parametrize("n,shared,width", [(152, False, 40), (153, False, 40), (200, False, 200), (304, True, 40),
                                            (700, False, 130), (320, True, 4097), (320, True, 4096)])
def test_selection_of_many_requests_and_of_wide_tables(n, shared, width):
    # up to an SM each, two to an SM, more than that with a request each; queries that share requests in tables too wide
    # for groups of four
    P, nsel, pages = 16, 9, 600
    requests = 3 if shared else n
    g = gen(n + width)
    table = torch.randint(0, pages, (requests, width), generator=g, dtype=torch.int32)
    req = [i * 3 // n for i in range(n)] if shared else list(range(n))
    lens = torch.randint(0, min(width, 300) * P + 1, (n,), generator=g).tolist()
    lens[0], lens[1], lens[2], lens[n - 1] = 0, -1, width * P, 1
    q, w = grid(n, 64, 128, std=1, step=0.25, seed=2), grid(n, 64, std=0.125, step=1 / 32, seed=3)
    keys = grid(pages, 128, std=0.5, step=1 / 32, seed=4)
    out = torch.full((n, nsel), -9, dtype=torch.int32, device="cuda")
    dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(), i32(lens), P,
                         nsel, req=i32(req) if shared else None, out=out)
    got = out.tolist()
    for i in sorted({*range(0, n, 7), 1, 2, n - 2, n - 1}):
        want = [-9] * nsel if lens[i] < 0 else oracle_choice(i, q, w, keys, table[req[i]].tolist(), lens[i], P, nsel)
        assert got[i] == want, i


def widest_table():
    """The most pages of a request that a selection takes, from the host's own check."""
    lib = _lib.load()
    takes = lambda width: lib.dsa_block_select(A, A, 0, 64, 128, A, 8, 16, A, 1, width, A, None, 4, 1, 1, A, None) == 0
    lo, hi = 1, 1 << 17
    assert takes(lo) and not takes(hi)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if takes(mid) else (lo, mid)
    return lo


def test_the_widest_table_is_what_the_header_says():
    assert 37000 <= widest_table() < 40000


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 5])
def test_selection_of_the_widest_table(n):
    width, P, nsel, pages = widest_table(), 16, 64, 5000
    table = torch.randint(0, pages, (1, width), generator=gen(1), dtype=torch.int32)
    q, w = grid(n, 64, 128, std=1, step=0.25, seed=2), grid(n, 64, std=0.125, step=1 / 32, seed=3)
    keys = grid(pages, 128, std=0.5, step=1 / 32, seed=4)
    lens = [width * P - i * 40000 for i in range(n)]
    got = dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(),
                               i32(lens), P, nsel, req=i32([0] * n))
    for i in range(n):
        assert got[i].tolist() == oracle_choice(i, q, w, keys, table[0].tolist(), lens[i], P, nsel), i


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 128])
def test_steps_over_a_wide_table(H):
    """Steps of a batch whose table is as wide as long requests need, so that the heads stay in groups of 64: each step
    against 64 bits, and captured and replayed."""
    P, B, width, pool, nsel = 16, 3, 800, 40, 3
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = B * width * P // 128
    assert blocks * 2 * (H // 64) > sms
    assert dsa.dsa_paged_attn_workspace_size(B, H, width, 0, P) == \
        min(blocks, sms * 64 // H) * (2 * H * (4 * DV + 8) + 16)      # a unit per group of 64 heads
    lens = [130, 1, 47]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count, held, seq = i32(list(range(pool))), i32([pool]), i32([0] * B), i32(lens)
    cache = torch.full((pool, P, D), NAN, dtype=torch.bfloat16, device="cuda")
    keys = torch.zeros(pool, P, 128, dtype=torch.bfloat16, device="cuda")
    means = torch.zeros(pool, 128, dtype=torch.bfloat16, device="cuda")
    rows = [randn(n, D, seed=10 + b) for b, n in enumerate(lens)]
    dsa.dsa_pages_update(table, held, seq, free, count, P)
    slots = dsa.dsa_pages_slots(table, held, seq, P, sum(lens))
    dsa.dsa_pages_append(torch.cat(rows).cuda(), randn(sum(lens), 128, seed=20).cuda(), slots, cache, keys, means)
    held.copy_(seq)
    kv, ki = torch.zeros(B, D, dtype=torch.bfloat16, device="cuda"), randn(B, 128, seed=21).cuda()
    q, qi = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"), randn(B, 64, 128, seed=22).cuda()
    w = torch.ones(B, 64, device="cuda")

    def step():
        seq.add_(1)
        dsa.dsa_pages_update(table, held, seq, free, count, P)
        dsa.dsa_pages_append(kv, ki, dsa.dsa_pages_slots(table, held, seq, P, B), cache, keys, means)
        chosen = dsa.dsa_block_select(qi, w, means, table, seq, P, nsel)
        held.copy_(seq)
        return chosen, dsa.dsa_paged_attn(q, cache, table, seq, SCALE, DV, blocks=chosen), \
            dsa.dsa_paged_attn(q, cache, table, seq, SCALE, DV)

    graph = None
    for t in range(20):
        new = randn(B, D, seed=100 + t)
        kv.copy_(new)
        q.copy_(randn(B, H, D, seed=200 + t))
        rows = [torch.cat([r, new[b:b + 1]]) for b, r in enumerate(rows)]
        if t == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step()
        if graph is None:
            got = step()
        else:
            graph.replay()
        now = [len(r) for r in rows]
        wide = [r.cuda().double() for r in rows]
        assert seq.tolist() == now
        near(got[1], *attend64(q.cpu(), wide, now, blocks=got[0].tolist(), P=P))
        near(got[2], *attend64(q.cpu(), wide, now))


# ------------------------------------------------------------------ many queries, none, and rows of any width

@pytest.mark.gpu
@pytest.mark.parametrize("H", [2, 33])
def test_many_more_queries_than_a_block_has_threads(H):
    have, P, n = [60, 200], 32, 1500
    cache, table, rows = paged(have, P, seed=H)
    g = gen(8)
    req = torch.randint(0, 2, (n,), generator=g).tolist()
    lens = [int(torch.randint(-1, have[r] + 1, (1,), generator=g)) for r in req]
    q = randn(n, H, D, seed=H)
    out = torch.full((n, H, DV), 3.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, req=i32(req), out=out)
    near(out, *attend64(q, rows, lens, req))
    none = [i for i in range(n) if lens[i] < 0]
    assert none and (out[none] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 128])
def test_calls_without_any_query(H):
    cache, table, _ = paged([100, 40], 16, seed=1)
    q, out = randn(2, H, D, seed=2).cuda(), torch.full((2, H, DV), 3.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_paged_attn(q, cache, table, i32([-1, -2 ** 31]), SCALE, DV, out=out)
    dsa.dsa_paged_attn(q, cache, table, i32([-1, -5]), SCALE, DV, blocks=i32([[0, 1], [0, 1]]), out=out)
    assert (out == 3.0).all()
    blocks = torch.full((2, 3), -9, dtype=torch.int32, device="cuda")
    dsa.dsa_block_select(randn(2, 64, 128, seed=3).cuda(), torch.ones(2, 64, device="cuda"), randn(20, 128, seed=4).cuda(),
                         table, i32([-1, -2 ** 31]), 16, 3, out=blocks)
    assert (blocks == -9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [8, 760, 768, 776, 2000, 4096])
@pytest.mark.parametrize("rows,DI", [(37, 8), (1100, 72)])
def test_rows_of_any_width(width, rows, DI):
    P, pages = 16, 80
    kv, ki = randn(rows, width, seed=1).cuda(), randn(rows, DI, seed=2).cuda()
    slots = torch.randperm(pages * P, generator=gen(width))[:rows].int().cuda()
    cache = torch.zeros(pages, P, width, dtype=torch.bfloat16, device="cuda")
    keys = torch.zeros(pages, P, DI, dtype=torch.bfloat16, device="cuda")
    means = torch.full((pages, DI), 5.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_pages_append(kv, ki, slots, cache, keys, means)
    want, want_keys = torch.zeros_like(cache), torch.zeros_like(keys)
    want.view(-1, width)[slots.long()] = kv
    want_keys.view(-1, DI)[slots.long()] = ki
    assert torch.equal(cache, want) and torch.equal(keys, want_keys)
    ended = torch.zeros(pages, dtype=torch.bool, device="cuda")
    ended[slots[slots % P == P - 1].long() // P] = True
    x = keys.double()
    # half a step of bf16, and P fp32 additions
    tol = 2.0 ** -8 * x.mean(1).abs() + 1.01 * P * 2.0 ** -24 * x.abs().mean(1)
    assert ((means.double() - x.mean(1)).abs() <= tol)[ended].all() and (means[~ended] == 5.0).all()
