"""The paged latent cache on the GPU: page tables and slots, writing rows and
block keys, choosing blocks and attending, alone and together.

Tolerance of the attention, elementwise, from the roundings.  With p_j the exact
weights over L rows:
  the result to bf16:                          2^-8 of it
  each P to bf16 for the product:              2^-8 p_j |v_j|
  a logit off by d_j, in the weight itself and in the denominator:
                                               expm1(d_j) p_j (|v_j| + |out|)
  exp2 (2 ulp), and fp32 sums of L terms in steps of an MMA that each round 16
  products and the sum so far, aligned to the largest of the 17, below 2^-24 of
  it:                                          (2^-21 + L / 16 * 17 * 2^-24) p_j (|v_j| + |out|)
and 2^-6 of the sum of these for their products.  d_j: q.k likewise, 36 steps,
36 * 17 * 2^-24 < 2^-14.7 of sum_d |q_d k_d| at the worst, and 2^-21 of the
largest logit for the scale and the exponent's fma.
"""
import numpy as np
import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from oracle import dsa_oracle as O

pytestmark = pytest.mark.gpu
D, DV, SCALE = 576, 512, 192 ** -0.5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    dsa.dsa_poll_device_error()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def randn(*shape, seed):
    return torch.randn(*shape, generator=gen(seed)).to(torch.bfloat16)


def paged(lens, P, seed, width=None, spare=2, fill=NAN):
    """(cache, table, rows per request in 64 bits): requests of these lengths in
    pages in random order; what no request owns is ``fill``."""
    width = width or max(1, max(-(-n // P) for n in lens))
    pages = sum(-(-n // P) for n in lens)
    order = torch.randperm(pages + spare, generator=gen(seed))
    cache = torch.full((pages + spare, P, D), fill, dtype=torch.bfloat16)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    rows, at = [], 0
    for b, n in enumerate(lens):
        x = randn(n, D, seed=seed * 1000 + b)
        rows.append(x.cuda().double())
        for k in range(-(-n // P)):
            page = order[at]
            at += 1
            part = x[k * P:(k + 1) * P]
            cache[page, :part.shape[0]] = part
            table[b, k] = page
    return cache.cuda(), table.cuda(), rows


def attend64(q, rows, lens, req=None, blocks=None, P=None, sink=None):
    """(out, tolerance) of the attention in 64 bits, a query at a time; NaN marks a query that is none."""
    n, H = q.shape[:2]
    out = torch.zeros(n, H, DV, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for i in range(n):
        if lens[i] < 0:
            out[i] = NAN
            continue
        k = rows[req[i] if req is not None else i][:lens[i]]
        if blocks is not None:
            pos = [b * P + x for b in blocks[i] if b >= 0 for x in range(P)]
            k = k[[p for p in pos if p < k.shape[0]]]
        L = k.shape[0]
        if L == 0:
            continue
        x = q[i].cuda().double()
        l = SCALE * (x @ k.T)
        m = l.amax(1, keepdim=True)
        p = torch.exp(l - m)
        den = p.sum(1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink.cuda().double()[:, None] - m)
        p = p / den
        v = k[:, :DV]
        out[i] = p @ v
        d = 2 ** -14.7 * SCALE * (x.abs() @ k.abs().T) + 2.0 ** -21 * l.abs().amax(1, keepdim=True)
        e = torch.expm1(d) + 2.0 ** -21 + L / 16 * 17 * 2.0 ** -24
        a = out[i].abs()
        tol[i] = (1 + 2 ** -6) * (2.0 ** -8 * a + 2.0 ** -8 * (p @ v.abs()) + (p * e) @ v.abs() +
                                  (p * e).sum(1, keepdim=True) * a) + 2.0 ** -133
    return out, tol


def near(got, want, tol):
    there = ~torch.isnan(want)
    worst = ((got.double() - want).abs() - tol)[there]
    assert worst.numel() == 0 or (worst <= 0).all(), f"{worst.max().item()} beyond the tolerance"


# ------------------------------------------------------------------ attention

RAGGED = [0, 1, 15, 16, 17, 100, 127, 128, 129, 257, 640]


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [1, 16, 17, 32, 33, 64, 65, 128])
def test_ragged_lengths(H, P):
    cache, table, rows = paged(RAGGED, P, seed=P + H)
    q = randn(len(RAGGED), H, D, seed=H)
    sink = torch.randn(H, generator=gen(3)) if H % 2 else None
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(RAGGED), SCALE, DV,
                             attn_sink=None if sink is None else sink.cuda())
    assert not got[0].any()
    near(got, *attend64(q, rows, RAGGED, sink=sink))


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("lens", [[9001], [5000, 3, 0, 2049, 64]], ids=["one", "few"])
def test_long_requests_over_all_units(H, lens):
    cache, table, rows = paged(lens, 64, seed=H)
    q = randn(len(lens), H, D, seed=H + 1)
    sink = torch.randn(H, generator=gen(4))
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, attn_sink=sink.cuda())
    near(got, *attend64(q, rows, lens, sink=sink))


@pytest.mark.parametrize("H", [16, 24, 64, 128])
def test_many_queries_of_few_requests(H):
    # every query sees one position more than the one before; some are none, and their rows of out stay
    have, n = [700, 130], 330
    cache, table, rows = paged(have, 64, seed=H)
    req = [0] * 230 + [1] * 100
    lens = [471 + i for i in range(230)] + [31 + i for i in range(100)]
    for i in (0, 7, 229, 329):
        lens[i] = -1
    q = randn(n, H, D, seed=H + 2)
    out = torch.full((n, H, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, req=i32(req), out=out)
    assert got is out
    near(got, *attend64(q, rows, lens, req))
    assert all((got[i] == 7.0).all() for i in (0, 7, 229, 329))


@pytest.mark.parametrize("P,nsel", [(16, 1), (16, 37), (32, 5), (64, 3), (64, 32), (128, 2)])
@pytest.mark.parametrize("H", [16, 128])
def test_selected_blocks(P, nsel, H):
    have, n = [1500, 90], 40
    cache, table, rows = paged(have, P, seed=P)
    g = gen(nsel)
    req, lens, blocks = [], [], torch.full((n, nsel), -1, dtype=torch.int32)
    for i in range(n):
        r = int(i % 5 == 0)
        req.append(r)
        lens.append(int(torch.randint(0, have[r] + 1, (1,), generator=g)))
        pages = -(-lens[i] // P)
        pick = torch.randperm(pages, generator=g)[:max(0, nsel - i % 3)]
        if i % 2:
            pick = pick.sort().values      # the order does not matter
        blocks[i, :pick.numel()] = pick
    q = randn(n, H, D, seed=H)
    sink = torch.randn(H, generator=gen(5))
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, blocks=blocks.cuda(), req=i32(req),
                             attn_sink=sink.cuda())
    want, tol = attend64(q, rows, lens, req, blocks.tolist(), P, sink)
    near(got, want, tol)
    empty = [i for i in range(n) if lens[i] == 0 or (blocks[i] < 0).all()]
    assert not got[empty].any()


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("order", ["rising", "falling", "peak"])
def test_the_reference_moves(H, order):
    # logits that grow by hundreds from block to block: sums and O are rescaled again and again
    L, P = 1100, 64
    step = torch.arange(L) // 128
    size = {"rising": step, "falling": 8 - step, "peak": (step == 5) * 8.0}[order].float()
    unit = randn(1, D, seed=1).float()
    k = (randn(L, D, seed=2).float() * 0.1 + size[:, None] * unit).to(torch.bfloat16)
    cache, table, _ = paged([L], P, seed=3, fill=NAN)
    flat = cache.view(-1, D)
    slots = dsa.dsa_pages_slots(table, None, i32([L]), P, L)
    flat[slots.long()] = k.cuda()
    q = (unit * torch.linspace(-1, 1, H)[:, None])[None].to(torch.bfloat16)
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32([L]), SCALE, DV)
    near(got, *attend64(q, [k.cuda().double()], [L]))


def test_values_that_are_not_finite():
    lens, P, H = [300, 300, 300], 64, 32
    cache, table, rows = paged(lens, P, seed=9)
    flat = cache.view(-1, D)
    at = lambda b, p: int(table[b, p // P]) * P + p % P
    flat[at(0, 200), 5] = NAN                        # a NaN row makes every head of that request NaN
    flat[at(1, 250), DV - 1] = INF                   # an infinite value: where its weight is not 0
    q = randn(3, H, D, seed=10)
    q[1, :, DV - 1] = 0
    q[1, :, 0] = q[1, :, 0].abs()
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV)
    assert torch.isnan(got[0]).all()
    assert torch.isnan(got[1]).all()                 # 0 * inf in q.k
    want, tol = attend64(q, rows, lens)
    near(got[2:], want[2:], tol[2:])
    # shorter contexts do not see those rows
    short = [200, 250, 300]
    near(dsa.dsa_paged_attn(q.cuda(), cache, table, i32(short), SCALE, DV), *attend64(q, rows, short))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_query_that_is_not_finite_spoils_its_head_alone(bad):
    lens, P, H = [1000, 300], 64, 40
    cache, table, rows = paged(lens, P, seed=29)
    q = randn(2, H, D, seed=30)
    clean = q.clone()
    q[0, 33, 7] = bad
    q[1, 2, 575] = bad
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV)
    assert torch.isnan(got[0, 33]).all() and torch.isnan(got[1, 2]).all()
    want, tol = attend64(clean, rows, lens)
    want[0, 33] = want[1, 2] = NAN
    near(got, want, tol)


def test_sinks_of_every_size():
    lens, P, H = [200, 0, 1], 32, 4
    cache, table, rows = paged(lens, P, seed=11)
    q = randn(3, H, D, seed=12)
    sink = torch.tensor([-INF, 0.0, 30.0, -200.0])
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV, attn_sink=sink.cuda())
    near(got, *attend64(q, rows, lens, sink=sink))
    assert not got[1].any()


def test_strided_cache():
    lens, P, H = [130, 77], 64, 16
    cache, table, rows = paged(lens, P, seed=13)
    wide = torch.full((cache.shape[0], P + 3, 648), NAN, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 2:2 + P, 64:64 + D]
    view.copy_(cache)
    q = randn(2, H, D, seed=14)
    got = dsa.dsa_paged_attn(q.cuda(), view, table, i32(lens), SCALE, DV)
    assert torch.equal(got, dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV))
    near(got, *attend64(q, rows, lens))


def test_pages_beyond_32_bits():
    # the last pages of a cache of more than 2^32 bytes and 2^31 values
    P, pages, lens = 128, 30000, [300]
    assert pages * P * D > 2 ** 31
    cache = torch.empty(pages, P, D, dtype=torch.bfloat16, device="cuda")
    table = i32([[pages - 1, pages - 3, pages - 2]])
    x = randn(300, D, seed=15)
    slots = dsa.dsa_pages_slots(table, None, i32(lens), P, 300)
    dsa.dsa_pages_append(x.cuda(), None, slots, cache)
    q = randn(1, 16, D, seed=16)
    near(dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV), *attend64(q, [x.cuda().double()], lens))


def test_same_bits_whatever_runs_beside_it():
    lens, P = [3000, 10, 700, 0, 128], 64
    cache, table, _ = paged(lens, P, seed=17)
    for H in (16, 128):
        q = randn(5, H, D, seed=18).cuda()
        args = (q, cache, table, i32(lens), SCALE, DV)
        want = dsa.dsa_paged_attn(*args)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams * 3:                        # workspaces of their own
            got.append(dsa.dsa_paged_attn(*args, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        # captured and replayed, with new lengths in the same tensor
        static = i32(lens)
        out = torch.zeros_like(want)
        ws = torch.empty(dsa.dsa_paged_attn_workspace_size(5, H, table.shape[1], 0, P), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dsa.dsa_paged_attn(q, cache, table, static, SCALE, DV, out=out, workspace=ws)
        for new in ([2999, 10, 3, 0, 1], lens):
            static.copy_(i32(new))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, dsa.dsa_paged_attn(q, cache, table, i32(new), SCALE, DV))


def bounds(site):
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_poll_device_error()
    assert e.value.status == 7 and e.value.detail[0] == site, e.value
    return e.value.detail[1]


@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_a_page_that_is_none(page):
    lens, P = [200, 200, 200], 64
    cache, table, rows = paged(lens, P, seed=19)
    table[1, 2] = page
    q = randn(3, 16, D, seed=20)
    got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32(lens), SCALE, DV)
    assert bounds(57) == 1
    rows[1] = torch.cat([rows[1][:128], rows[1][192:]])
    near(got, *attend64(q, rows, [200, 136, 200]))


def test_a_request_or_length_that_is_none():
    lens, P = [200, 130], 64
    cache, table, rows = paged(lens, P, seed=21)
    q = randn(3, 16, D, seed=22)
    for req in ([0, 2, 1], [0, -1, 1]):
        got = dsa.dsa_paged_attn(q.cuda(), cache, table, i32([200, 50, 130]), SCALE, DV, req=i32(req))
        assert bounds(58) == 1 and not got[1].any()
        near(got[[0, 2]], *attend64(q[[0, 2]], rows, lens))
    got = dsa.dsa_paged_attn(q[:1].cuda(), cache, table, i32([4 * P + 1]), SCALE, DV)
    assert bounds(58) == 0                           # longer than the table: what it has is used
    assert torch.isnan(got).all()                    # and the rows behind the request's last are NaN here
    near(dsa.dsa_paged_attn(q[:2].cuda(), cache, table, i32(lens), SCALE, DV), *attend64(q[:2], rows, lens))


def test_attention_refusals():
    lens, P = [200, 130], 64
    cache, table, _ = paged(lens, P, seed=23)
    q, ln = randn(2, 16, D, seed=24).cuda(), i32(lens)
    call = lambda q=q, cache=cache, table=table, ln=ln, **kw: dsa.dsa_paged_attn(q, cache, table, ln, SCALE, DV, **kw)
    bad = [dict(q=q.float()), dict(q=q[0]), dict(q=q[:, :, :512]), dict(q=q.cpu()), dict(q=q.transpose(0, 1)),
           dict(cache=cache.float()), dict(cache=cache[:, :24]), dict(cache=cache[0]), dict(cache=cache[:, :, 4:]),
           dict(cache=cache[:, :, ::2]), dict(table=table.long()), dict(table=table[0]), dict(table=table[:, :0]),
           dict(ln=ln.long()), dict(ln=ln[:1]), dict(ln=None), dict(req=ln[:1]), dict(table=table[:1]), dict(blocks=ln),
           dict(blocks=i32([[0]])), dict(blocks=torch.zeros(2, 0, dtype=torch.int32, device="cuda")),
           dict(attn_sink=torch.zeros(8, device="cuda")),
           dict(out=torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda")),
           dict(workspace=torch.zeros(64, device="cuda"))]
    for k, kw in enumerate(bad):
        with pytest.raises(ValueError):
            call(**kw)
            pytest.fail(f"case {k} was taken")
    with pytest.raises(dsa.DSAError) as e:
        call(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_paged_attn(randn(2, 129, D, seed=1).cuda(), cache, table, ln, SCALE, DV)
    assert e.value.status == 3
    empty = dsa.dsa_paged_attn(q[:0], cache, table, ln[:0], SCALE, DV)
    assert tuple(empty.shape) == (0, 16, DV)


# ------------------------------------------------------------------ page tables and slots

def test_page_tables_follow_the_oracle():
    rng = np.random.default_rng(2)
    for B, width, P in ((1, 3, 16), (5, 9, 64), (70, 40, 32), (1300, 4, 128)):
        pool = B * width * 2 // 3 + 1
        ref = ([[-1] * width for _ in range(B)], [int(x) for x in rng.permutation(pool)], pool)
        lens = [0] * B
        table, free, count = i32(ref[0]), i32(ref[1]), i32([ref[2]])
        done = 0
        for step in range(12):
            new = [int(x) for x in rng.integers(0, width * P + 1, B)] if step % 3 == 0 else \
                [min(n + int(rng.integers(-3, 5)), width * P) if n > 3 else n + 2 for n in lens]
            got = O.pages_update(*[ref[0], lens, new, ref[1], ref[2]], P)
            dsa.dsa_pages_update(table, i32(lens), i32(new), free, count, P)
            if got is None:
                bounds(54)
            else:
                ref, lens, done = got, new, done + 1
            assert table.tolist() == ref[0] and free.tolist() == ref[1] and count.item() == ref[2]
            n = sum(lens)
            assert dsa.dsa_pages_slots(table, None, i32(lens), P, n + 5).tolist() == \
                O.pages_slots(ref[0], None, lens, P, n + 5)
            first = [int(rng.integers(0, x + 1)) for x in lens]
            n -= sum(first)
            assert dsa.dsa_pages_slots(table, i32(first), i32(lens), P, n).tolist() == \
                O.pages_slots(ref[0], first, lens, P, n)
        assert done >= 6


@pytest.mark.parametrize("held,seq,site,detail", [([0, 0], [16, 65], 52, 1), ([0, 0], [-1, 3], 52, 0),
                                                  ([-5, 0], [1, 3], 52, 0), ([0, 33], [0, 0], 53, 1),
                                                  ([0, 0], [64, 49], 54, 8)])
def test_page_tables_change_not_at_all_or_wholly(held, seq, site, detail):
    table, free, count = i32([[3, -1, -1, -1], [9, 1, -1, -1]]), i32(list(range(10))), i32([7])
    before = [t.clone() for t in (table, free, count)]
    dsa.dsa_pages_update(table, i32(held), i32(seq), free, count, 16)
    assert bounds(site) == detail
    assert all(torch.equal(a, b) for a, b in zip((table, free, count), before))
    # a stack that says it holds as many pages as it can, and one comes back
    dsa.dsa_pages_update(table, i32([16, 0]), i32([0, 0]), free, i32([10]), 16)
    bounds(54)
    assert torch.equal(table, before[0])


def test_slots_beyond_the_table_or_the_output():
    table = i32([[2, -1], [0, 1]])
    assert dsa.dsa_pages_slots(table, None, i32([17, 2]), 16, 20).tolist() == list(range(32, 48)) + [-1, 0, 1, -1]
    got = dsa.dsa_pages_slots(table, None, i32([17, 2]), 16, 18).tolist()
    assert bounds(55) == 2 and got == list(range(32, 48)) + [-1, 0]
    got = dsa.dsa_pages_slots(table, i32([0, 31]), i32([1, 34]), 16, 5).tolist()
    assert bounds(52) == 1 and got == [32, 31, -1, -1, -1]
    got = dsa.dsa_pages_slots(table, i32([-2, 0]), i32([1, 1]), 16, 3).tolist()
    assert bounds(52) == 0 and got == [32, 0, -1]
    assert dsa.dsa_pages_slots(table[:0], None, i32([]), 16, 3).tolist() == [-1, -1, -1]
    assert dsa.dsa_pages_slots(table, None, i32([0, 0]), 16, 0).numel() == 0


def test_page_table_refusals():
    table, free, count, ln = i32([[0, -1]]), i32([1, 2, 3]), i32([3]), i32([4])
    for kw in (dict(table=table.long()), dict(table=table[0]), dict(ln=ln.long()), dict(ln=i32([1, 2])),
               dict(free=free[:, None]), dict(count=i32([1, 2])), dict(P=17), dict(table=table.cpu())):
        a = dict(table=table, ln=ln, free=free, count=count, P=16)
        a.update(kw)
        with pytest.raises(ValueError):
            dsa.dsa_pages_update(a["table"], a["ln"], ln, a["free"], a["count"], a["P"])
    for kw in (dict(n=-1), dict(n=1 << 31), dict(first=i32([1, 2])), dict(out=i32([1, 2])), dict(P=0)):
        a = dict(first=None, n=4, out=None, P=16)
        a.update(kw)
        with pytest.raises(ValueError):
            dsa.dsa_pages_slots(table, a["first"], ln, a["P"], a["n"], out=a["out"])


# ------------------------------------------------------------------ writing rows

@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("DI", [128, 32])
def test_rows_and_block_keys(P, DI):
    # the same rows in one call, in odd pieces and one by one: the same bytes, and the mean of every full page
    lens = [3 * P + 5, P - 1, 2 * P, 1]
    B, width = len(lens), 4
    pages = B * width
    table = torch.randperm(pages, generator=gen(P)).view(B, width).to(torch.int32).cuda()
    rows = [(randn(n, D, seed=b), randn(n, DI, seed=50 + b)) for b, n in enumerate(lens)]

    def write(cuts):
        cache = torch.full((pages, P, D), 3.0, dtype=torch.bfloat16, device="cuda")
        keys = torch.full((pages, P, DI), 4.0, dtype=torch.bfloat16, device="cuda")
        means = torch.full((pages, DI), 5.0, dtype=torch.bfloat16, device="cuda")
        held = [0] * B
        for c in cuts:
            new = [min(n, c) for n in lens]
            n = sum(new) - sum(held)
            slots = dsa.dsa_pages_slots(table, i32(held), i32(new), P, n)
            kv = torch.cat([r[0][h:m] for r, h, m in zip(rows, held, new)])
            ki = torch.cat([r[1][h:m] for r, h, m in zip(rows, held, new)])
            wide = torch.full((n, 648), NAN, dtype=torch.bfloat16)
            wide[:, 64:64 + D] = kv
            dsa.dsa_pages_append(wide.cuda()[:, 64:64 + D], ki.cuda(), slots, cache, keys, means)
            held = new
        return cache, keys, means

    one = write([max(lens)])
    for cuts in ([1, 7, P, P + 1, 3 * P, 3 * P + 5], list(range(1, 3 * P + 6))):
        assert all(torch.equal(a, b) for a, b in zip(write(cuts), one)), cuts
    cache, keys, means = (t.cpu() for t in one)
    table = table.cpu()
    named = set()
    for b, n in enumerate(lens):
        for p in range(n):
            page = int(table[b, p // P])
            assert torch.equal(cache[page, p % P], rows[b][0][p]) and torch.equal(keys[page, p % P], rows[b][1][p])
            named.add((page, p % P))
        for k in range(n // P):
            page = int(table[b, k])
            x = rows[b][1][k * P:(k + 1) * P].double()
            # half a step of bf16, and P fp32 additions
            tol = 2.0 ** -8 * x.mean(0).abs() + 1.01 * P * 2.0 ** -24 * x.abs().mean(0)
            assert ((means[page].double() - x.mean(0)).abs() <= tol).all()
    for page in range(pages):
        for r in range(P):
            if (page, r) not in named:
                assert (cache[page, r] == 3.0).all() and (keys[page, r] == 4.0).all()
        if (page, P - 1) not in named:
            assert (means[page] == 5.0).all()


def test_rows_without_a_slot_stay():
    P, pages = 16, 3
    cache = torch.zeros(pages, P, D, dtype=torch.bfloat16, device="cuda")
    x = randn(4, D, seed=1).cuda()
    dsa.dsa_pages_append(x, None, i32([5, -1, 47, -7]), cache)
    want = torch.zeros_like(cache)
    want.view(-1, D)[[5, 47]] = x[[0, 2]]
    assert torch.equal(cache, want)
    dsa.dsa_pages_append(x, None, i32([5, 48, 6, -7]), cache)
    assert bounds(56) == 1
    want.view(-1, D)[[5, 6]] = x[[0, 2]]
    assert torch.equal(cache, want)
    # rewritten rows of a page that was full: its key is that of the rows it holds now
    keys = torch.zeros(pages, P, 128, dtype=torch.bfloat16, device="cuda")
    means = torch.zeros(pages, 128, dtype=torch.bfloat16, device="cuda")
    a, b = randn(P, 128, seed=2).cuda(), randn(3, 128, seed=3).cuda()
    dsa.dsa_pages_append(randn(P, D, seed=4).cuda(), a, i32(list(range(16, 32))), cache, keys, means)
    dsa.dsa_pages_append(randn(3, D, seed=5).cuda(), b, i32([29, 30, 31]), cache, keys, means)
    whole = torch.zeros_like(means)
    dsa.dsa_pages_append(randn(P, D, seed=4).cuda(), torch.cat([a[:13], b]), i32(list(range(16, 32))), cache, keys, whole)
    assert torch.equal(means, whole) and means[1].any()


def test_append_refusals():
    P = 16
    cache = torch.zeros(3, P, D, dtype=torch.bfloat16, device="cuda")
    keys = torch.zeros(3, P, 128, dtype=torch.bfloat16, device="cuda")
    means = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    x, k, s = randn(4, D, seed=1).cuda(), randn(4, 128, seed=1).cuda(), i32([0, 1, 2, 3])
    for args in ((x.float(), k, s, cache, keys, means), (x[:, :512], k, s, cache, keys, means), (x, k, s, cache),
                 (x, k, s[:3], cache, keys, means), (x, k, s.long(), cache, keys, means), (x, k, s, cache, keys[:2], means),
                 (x, k, s, cache, keys, means[:, :64]), (x, k, s, cache[:, :9], keys, means), (x, None, s, cache, keys, None),
                 (x, k.t(), s, cache, keys, means), (x.cpu(), k, s, cache, keys, means), (x, k, None, cache, keys, means)):
        with pytest.raises(ValueError):
            dsa.dsa_pages_append(*args)
    dsa.dsa_pages_append(x[:0], k[:0], s[:0], cache, keys, means)
    assert not cache.any()


# ------------------------------------------------------------------ choosing blocks

def grid(*shape, std, step, seed):
    """Normal values on multiples of a power of two: their scores are exact in fp32 in any order, and ties occur."""
    return (torch.randn(*shape, generator=gen(seed)) * (std / step)).round() * step


@pytest.mark.parametrize("HI", [64, 5])
@pytest.mark.parametrize("P,nsel,keep", [(64, 8, (1, 1)), (16, 40, (2, 3)), (128, 1, (0, 1)), (32, 130, (0, 2))])
def test_selection_follows_the_oracle(P, nsel, keep, HI):
    lens = [0, 1, P, 8 * P, 8 * P + 1, 300 * P, 129 * P - 3, 128 * P, 200 * P, -1]
    B, width = len(lens), 301
    pages = B * width
    table = torch.randperm(pages, generator=gen(1)).view(B, width).to(torch.int32)
    q, w = grid(B, HI, 128, std=1, step=0.25, seed=2), grid(B, HI, std=0.125, step=1 / 32, seed=3)
    keys = grid(pages, 128, std=0.5, step=1 / 32, seed=4)
    w[8] = 0                                       # all scores equal: the lowest pages
    out = torch.full((B, nsel), -9, dtype=torch.int32, device="cuda")
    got = dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(),
                               i32(lens), P, nsel, *keep, out=out)
    for i in range(B - 1):
        want = O.block_select(q[i].numpy(), w[i].numpy(), keys.numpy(), table[i].tolist(), lens[i], P, nsel, *keep)
        assert got[i].tolist() == want, i
    assert (got[B - 1] == -9).all()


def test_selection_of_many_queries_of_few_requests():
    # more queries than SMs: four of a group share their request's keys, but for groups at a request's border
    P, nsel, n = 16, 12, 611
    have = [150 * P, 40 * P, 5 * P]
    pages, width = 500, 150
    table = torch.stack([torch.randperm(pages, generator=gen(b))[:width] for b in range(3)]).to(torch.int32)
    req = [0] * 401 + [1] * 150 + [2] * 60
    lens = [have[r] - (i * 7) % (4 * P) for i, r in enumerate(req)]
    lens[5] = lens[403] = -1
    lens[610] = 0
    q, w = grid(n, 64, 128, std=1, step=0.25, seed=2), grid(n, 64, std=0.125, step=1 / 32, seed=3)
    keys = grid(pages, 128, std=0.5, step=1 / 32, seed=4)
    args = (q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(), i32(lens), P, nsel)
    out = torch.full((n, nsel), -9, dtype=torch.int32, device="cuda")
    got = dsa.dsa_block_select(*args, req=i32(req), out=out)
    for i in list(range(0, n, 13)) + [4, 5, 400, 401, 402, 403, 404, 550, 551, 552, 610]:
        if lens[i] < 0:
            assert (got[i] == -9).all()
            continue
        want = O.block_select(q[i].numpy(), w[i].numpy(), keys.numpy(), table[req[i]].tolist(), lens[i], P, nsel)
        assert got[i].tolist() == want, i
    # a query alone gives the same list
    for i in (0, 402, 600):
        alone = dsa.dsa_block_select(args[0][i:i + 1], args[1][i:i + 1], args[2], args[3], i32([lens[i]]), P, nsel,
                                     req=i32([req[i]]))
        assert torch.equal(alone[0], got[i])


def test_long_contexts_are_chosen_from():
    P, width, nsel = 64, 20011, 64
    table = torch.randperm(width, generator=gen(1)).to(torch.int32)[None]
    q, w = grid(1, 64, 128, std=1, step=0.25, seed=2), grid(1, 64, std=0.125, step=1 / 32, seed=3)
    keys = grid(width, 128, std=0.5, step=1 / 32, seed=4)
    got = dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(),
                               i32([width * P - 5]), P, nsel)
    assert got[0].tolist() == O.block_select(q[0].numpy(), w[0].numpy(), keys.numpy(), table[0].tolist(), width * P - 5,
                                             P, nsel)


def test_scores_that_are_no_numbers_and_pages_that_are_none():
    P, nsel, width = 16, 4, 30
    table = torch.arange(width, dtype=torch.int32)[None].repeat(2, 1)
    q, w = grid(2, 64, 128, std=1, step=0.25, seed=2), grid(2, 64, std=0.125, step=1 / 32, seed=3).abs()
    keys = grid(width, 128, std=0.5, step=1 / 32, seed=4)
    w[0, 3] = NAN                                   # every score of that query
    keys[11, 5] = NAN                               # the scores of that page
    table[1, 7] = -1                                # ranks last
    table[1, 9] = width
    lens = [width * P] * 2
    got = dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table.cuda(),
                               i32(lens), P, nsel)
    assert bounds(57) == 1
    assert got[0].tolist() == [0, 1, 2, 29]
    keep = [b for b in range(width) if b not in (7, 9, 11)]
    want = O.block_select(q[1].numpy(), w[1].numpy(), keys.numpy(), keep, len(keep) * P, P, nsel)
    assert got[1].tolist() == [keep[b] for b in want]
    dsa.dsa_block_select(q.to(torch.bfloat16).cuda(), w.cuda(), keys.to(torch.bfloat16).cuda(), table[:1].cuda(),
                         i32([P, P]), P, nsel, req=i32([0, 1]))
    assert bounds(58) == 1


def test_selection_refusals():
    q, w, keys = randn(2, 64, 128, seed=1).cuda(), torch.zeros(2, 64, device="cuda"), randn(9, 128, seed=2).cuda()
    table, ln = i32([[0, 1], [2, 3]]), i32([20, 3])
    for a in ((q.float(), w, keys, table, ln, 16, 4), (q, w.half(), keys, table, ln, 16, 4),
              (q, w[:, :3], keys, table, ln, 16, 4), (q, w, keys[:, :64], table, ln, 16, 4), (q, w, keys, table[:1], ln, 16, 4),
              (q, w, keys, table, ln[:1], 16, 4), (q, w, keys, table, ln, 15, 4), (q[0], w, keys, table, ln, 16, 4),
              (q, w, keys, table.long(), ln, 16, 4), (q, w, keys, table, None, 16, 4)):
        with pytest.raises(ValueError):
            dsa.dsa_block_select(*a)
    for nsel, first, last, status in ((1, 1, 1, 2), (0, 0, 1, 2), (4, 1, 0, 2), (4, -1, 1, 2)):
        with pytest.raises(dsa.DSAError) as e:
            dsa.dsa_block_select(q, w, keys, table, ln, 16, nsel, first, last)
        assert e.value.status == status
    assert dsa.dsa_block_select(q[:0], w[:0], keys, table, ln[:0], 16, 4).numel() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("H,P", [(16, 16), (128, 64)])
def test_serving_steps(H, P):
    """Prompts admitted, then steps of one token a request: pages, rows and block keys, the blocks chosen, attention
    over them and over everything, one request leaving and another taking its pages; and the 4-bit cache over the same
    slots."""
    lens, width, nsel = [5 * P + 3, 1, 9 * P - 1], 12, 4
    B, pool = len(lens), 24
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = i32(list(range(pool))), i32([pool])
    cache = torch.full((pool, P, D), NAN, dtype=torch.bfloat16, device="cuda")
    keys = torch.zeros(pool, P, 128, dtype=torch.bfloat16, device="cuda")
    means = torch.zeros(pool, 128, dtype=torch.bfloat16, device="cuda")
    small = torch.zeros(pool * P, dsa.dsa_kv_int4_row_bytes(D, DV), dtype=torch.uint8, device="cuda")
    held, rows = [0] * B, [torch.zeros(0, D, dtype=torch.bfloat16) for _ in range(B)]
    seed = 100
    for step in range(6):
        if step == 3:                              # request 0 leaves; a shorter one takes its place
            dsa.dsa_pages_update(table, i32(held), i32([0] + held[1:]), free, count, P)
            held[0], rows[0], lens = 0, rows[0][:0], [2 * P + 7] + lens[1:]
        elif step:
            lens = [n + 1 for n in lens]
        new = sum(lens) - sum(held)
        dsa.dsa_pages_update(table, i32(held), i32(lens), free, count, P)
        slots = dsa.dsa_pages_slots(table, i32(held), i32(lens), P, new)
        fresh = []
        for b in range(B):
            fresh.append(randn(lens[b] - held[b], D, seed=seed + b))
            rows[b] = torch.cat([rows[b], fresh[b]])
        kv = torch.cat(fresh).cuda()
        ki = grid(new, 128, std=1, step=0.25, seed=seed + 50).to(torch.bfloat16).cuda()
        dsa.dsa_pages_append(kv, ki, slots, cache, keys, means)
        dsa.dsa_kv_int4_quantize(kv, DV, out=small, slots=slots)
        held, seed = list(lens), seed + 100
        q, qi = randn(B, H, D, seed=seed + 60), randn(B, 64, 128, seed=seed + 61)
        w = torch.randn(B, 64, generator=gen(seed + 62))
        ln = i32(lens)
        blocks = dsa.dsa_block_select(qi.cuda(), w.cuda(), means, table, ln, P, nsel)
        for b in range(B):                         # the choice is right up to what fp32 sums leave open
            have = -(-lens[b] // P)
            chosen = [x for x in blocks[b].tolist() if x >= 0]
            assert len(chosen) == min(have, nsel) and chosen == sorted(set(chosen))
            assert chosen[0] == 0 and chosen[-1] == have - 1
            k = means[table[b, :have].long()].cpu().double()
            s = (w[b].double()[:, None] * (qi[b].double() @ k.T).clamp(min=0)).sum(0)
            size = (w[b].double().abs()[:, None] * (qi[b].double().abs() @ k.abs().T)).sum(0).max() * 2.0 ** -14
            rest = [x for x in range(have) if x not in chosen]
            if rest and len(chosen) > 2:
                assert s[chosen[1:-1]].min() >= s[rest].max() - size
        wide = [r.cuda().double() for r in rows]
        near(dsa.dsa_paged_attn(q.cuda(), cache, table, ln, SCALE, DV, blocks=blocks),
             *attend64(q, wide, lens, blocks=blocks.tolist(), P=P))
        near(dsa.dsa_paged_attn(q.cuda(), cache, table, ln, SCALE, DV), *attend64(q, wide, lens))
        # the 4-bit cache through the slots of all rows, entries numbered request by request
        every = dsa.dsa_pages_slots(table, None, ln, P, sum(lens))
        top = max(lens)
        idx = torch.full((B, top), -1, dtype=torch.int32)
        for b in range(B):
            idx[b, :lens[b]] = torch.arange(lens[b]) + sum(lens[:b])
        got = dsa.dsa_sparse_attn_int4kv(q.cuda(), small, idx.cuda(), SCALE, DV, slots=every)
        back = dsa.dsa_kv_int4_dequantize(small, D, DV, rows=every).double()
        near(got, *attend64(q, list(torch.split(back, lens)), lens))
    owned = sum(-(-n // P) for n in lens)
    assert count.item() == pool - owned
    dsa.dsa_pages_update(table, i32(lens), i32([0] * B), free, count, P)
    assert count.item() == pool and sorted(free.tolist()) == list(range(pool)) and (table == -1).all()


@pytest.mark.parametrize("H", [16, 128])
def test_steps_in_a_graph(H):
    """A whole step captured once and replayed: lengths grow, pages are taken, rows written, blocks chosen and attended
    over, all by what lies in the step's own tensors; every replay against the calls one by one."""
    P, B, width, pool, nsel, steps = 16, 3, 8, 20, 3, 40
    start = [15, 0, 47]

    def fresh():
        s = dict(table=torch.full((B, width), -1, dtype=torch.int32, device="cuda"), free=i32(list(range(pool))),
                 count=i32([pool]), held=i32([0] * B), seq=i32(start),
                 cache=torch.full((pool, P, D), NAN, dtype=torch.bfloat16, device="cuda"),
                 keys=torch.zeros(pool, P, 128, dtype=torch.bfloat16, device="cuda"),
                 means=torch.zeros(pool, 128, dtype=torch.bfloat16, device="cuda"),
                 kv=torch.zeros(B, D, dtype=torch.bfloat16, device="cuda"),
                 ki=torch.zeros(B, 128, dtype=torch.bfloat16, device="cuda"),
                 q=torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                 qi=torch.zeros(B, 64, 128, dtype=torch.bfloat16, device="cuda"),
                 w=torch.ones(B, 64, device="cuda"))
        n = sum(start)
        dsa.dsa_pages_update(s["table"], s["held"], s["seq"], s["free"], s["count"], P)
        slots = dsa.dsa_pages_slots(s["table"], s["held"], s["seq"], P, n)
        dsa.dsa_pages_append(randn(n, D, seed=1).cuda(), randn(n, 128, seed=2).cuda(), slots, s["cache"], s["keys"],
                             s["means"])
        s["held"].copy_(s["seq"])
        return s

    def step(s):
        s["seq"].add_(1)
        dsa.dsa_pages_update(s["table"], s["held"], s["seq"], s["free"], s["count"], P)
        slots = dsa.dsa_pages_slots(s["table"], s["held"], s["seq"], P, B)
        dsa.dsa_pages_append(s["kv"], s["ki"], slots, s["cache"], s["keys"], s["means"])
        blocks = dsa.dsa_block_select(s["qi"], s["w"], s["means"], s["table"], s["seq"], P, nsel)
        out = dsa.dsa_paged_attn(s["q"], s["cache"], s["table"], s["seq"], SCALE, DV, blocks=blocks)
        s["held"].copy_(s["seq"])
        return blocks, out

    def inputs(s, t):
        for k, name in enumerate(("kv", "ki", "q", "qi")):
            s[name].copy_(randn(*s[name].shape, seed=100 * t + k))

    a, b = fresh(), fresh()
    step(fresh())                                    # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for t in range(steps):
        inputs(a, t)
        inputs(b, t)
        graph.replay()
        want = step(b)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), t
    for name in ("table", "free", "count", "keys", "means"):
        assert torch.equal(a[name], b[name])
    assert a["seq"].tolist() == [n + steps for n in start] and not torch.isnan(got[1]).any()
