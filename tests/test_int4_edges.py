"""The attention over the 4-bit cache in every division of a call (pairs of
SMs, groups of 16 and of 32 heads, each with and without splits of the
entries), where its answer must not depend on the division.

Tolerance, elementwise, from the roundings.  With p_j the exact weights:
  the result to bf16:                          2^-8 of it
  each P to bf16 for the product:              2^-8 p_j |v_j|
  a logit off by d_j, in the weight itself and in the denominator:
                                               expm1(d_j) p_j (|v_j| + |out|)
  exp2 and fp32 sums of up to 2048 terms:      2^-14 p_j |v_j|
and 2^-6 of the sum of these for their products.  d_j: q.k is summed in fp32,
36 steps of an MMA that each round 16 products and the sum so far, aligned to
the largest of the 17, below 2^-24 of it: 36 * 17 * 2^-24 < 2^-14.7 of
sum_d |q_d k_d| at the very worst.  Where q and k are integers whose sums stay
below 2^24, q.k is exact and d_j is what the scale and the exponent's fma
round, 2^-21 of the largest logit.
"""
import numpy as np
import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa

D, DV, SCALE = 576, 512, 192 ** -0.5
INF = float("inf")

# n, H, topk of a call in every division on 152 SMs
DIVISIONS = {"pairs": (90, 128, 130), "pairs, split": (8, 128, 2048), "pairs, longest first": (152, 128, 1100),
             "groups of 16": (160, 16, 300), "groups of 16, split": (1, 16, 2048),
             "groups of 32": (160, 32, 300), "groups of 32, split": (6, 32, 2048)}
every_division = pytest.mark.parametrize("n,H,topk", DIVISIONS.values(), ids=DIVISIONS.keys())


@pytest.fixture(autouse=True)
def _gpu(request):
    if request.node.get_closest_marker("gpu") is None:
        yield
        return
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    dsa.dsa_poll_device_error()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def latent(n, seed):
    return torch.randn(n, D, generator=gen(seed)).to(torch.bfloat16)


def store(kv):
    """(cache, the values it stands for in 64 bits)."""
    cache = dsa.dsa_kv_int4_quantize(kv.cuda(), DV)
    return cache, dsa.dsa_kv_int4_dequantize(cache, D, DV).double()


def attend64(q, rows, idx, sink=None, slots=None, exact_sums=False):
    """(out, tolerance) of the attention in 64 bits, a query at a time."""
    q, rows, idx = q.cuda().double(), rows.cuda(), idx.cuda()
    n, H = q.shape[:2]
    out = torch.zeros(n, H, DV, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for i in range(n):
        pick = idx[i].long()
        pick = pick[pick >= 0]
        if slots is not None:
            pick = slots[pick].long()
            pick = pick[pick >= 0]
        if not pick.numel():
            continue
        k = rows[pick]
        l = SCALE * (q[i] @ k.T)
        m = l.amax(1, keepdim=True)
        p = torch.exp(l - m)
        den = p.sum(1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink.double()[:, None] - m)
        p = p / den
        out[i] = p @ k[:, :DV]
        if exact_sums:
            d = 2.0 ** -21 * l.abs().amax(1, keepdim=True).expand_as(l)
        else:
            d = SCALE * 2.0 ** -14.7 * (q[i].abs() @ k.abs().T)
        off = p * torch.expm1(d)
        v = k[:, :DV].abs()
        t = (p * (2.0 ** -8 + 2.0 ** -14) + off) @ v + out[i].abs() * (2.0 ** -8 + off.sum(1, keepdim=True))
        tol[i] = t * (1 + 2.0 ** -6) + 1e-30
    return out, tol


def check(got, ref, tol):
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), (off / tol).nan_to_num(nan=INF).max().item()
    # the roundings are independent: their norm stays well below the sum of their bounds
    norm = ref.norm()
    assert norm == 0 or (got.double() - ref).norm() / norm <= 1e-2


def division(n, H, topk):
    splits, heads, first = dsa.dsa_sparse_attn_int4kv_division(n, H, topk)
    return ("pairs" if heads == 0 else f"groups of {heads}") + (", split" if splits > 1 else "") + \
        (", longest first" if first else "")


@pytest.mark.gpu
def test_divisions_are_what_their_names_say():
    """What is tested below in every division is: the rule that divides a call may move, the tests then move along."""
    for name, (n, H, topk) in DIVISIONS.items():
        assert division(n, H, topk) == name


# ------------------------------------------------------------------ queries without a row

@pytest.mark.gpu
@every_division
def test_entries_that_lead_to_no_row_give_zeros(n, H, topk):
    """Every third query names KV rows whose slot is negative, and nothing else: zeros, whatever the sink.  The last
    one names a row that holds a NaN beside them: NaN, whatever the sink."""
    R = 200
    kv = latent(R, 1)
    kv[R - 1, 7] = float("nan")
    cache, rows = store(kv)
    slots = torch.arange(R, dtype=torch.int32)
    slots[150:R - 1] = -1
    idx = torch.randint(0, 150, (n, topk), generator=gen(2)).to(torch.int32)
    none = [i for i in range(0, n, 3) if i == 0 or i < n - 1]
    idx[none] = torch.randint(150, R - 1, (len(none), topk), generator=gen(3)).to(torch.int32)
    if n > 1:
        idx[n - 1] = 160
        idx[n - 1, topk // 2] = R - 1
    use = max(n - 1, 1)
    q = torch.randn(n, H, D, generator=gen(4)).to(torch.bfloat16).cuda()
    idx, slots = idx.cuda(), slots.cuda()
    for level in (None, 2.0, INF, -INF):
        sink = None if level is None else torch.full((H,), level, device="cuda")
        got = dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, attn_sink=sink, slots=slots)
        assert not got[none].any()                      # a NaN counts as something
        if n > 1:
            assert torch.isnan(got[n - 1]).all()
        ref, tol = attend64(q[:use], rows, idx[:use], sink, slots)
        check(got[:use], ref, tol)


@pytest.mark.gpu
@every_division
def test_entries_out_of_range_give_zeros(n, H, topk):
    """A query whose entries are all out of range has none: reported, and zeros under a sink of -inf."""
    cache, rows = store(latent(64, 5))
    idx = torch.randint(0, 64, (n, topk), generator=gen(6)).to(torch.int32)
    idx[0] = 64
    q = torch.randn(n, H, D, generator=gen(7)).to(torch.bfloat16).cuda()
    sink = torch.full((H,), -INF, device="cuda")
    got = dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, attn_sink=sink)
    with pytest.raises(dsa.DSAError) as err:
        dsa.dsa_poll_device_error()
    assert err.value.status == 7 and err.value.detail[0] == 50
    idx[0] = -1
    ref, tol = attend64(q, rows, idx, sink)
    check(got, ref, tol)
    assert not got[0].any()


# ------------------------------------------------------------------ sums of q.k

@pytest.mark.gpu
@every_division
@pytest.mark.parametrize("size", [8, 64])
def test_halves_of_q_k_that_cancel(n, H, topk, size):
    """q.k whose halves over columns 0-255 and 256-511 are large (some 12,000 with size 8, 99,000 with size 64) and
    cancel to a few units: integers, exact in 32 bits."""
    R = 300
    kv = torch.empty(R, D)
    sign = torch.where(torch.rand(DV // 2, generator=gen(8)) < 0.5, -1.0, 1.0)
    kv[:, :256] = 6 * sign
    kv[:, :256:16] = 7 * sign[::16]
    kv[:, 256:DV] = kv[:, :256]
    kv[:, DV:] = 0
    # a row differs from the others in the rope columns, and in a few values on either side
    kv[:, DV:] = torch.randint(-2, 3, (R, D - DV), generator=gen(9)).float() / size
    flip = torch.randint(1, 16, (R, 2), generator=gen(10))
    for side in range(2):
        at = 256 * side + 16 * torch.randint(0, 16, (R,), generator=gen(11 + side)) + flip[:, side]
        kv[torch.arange(R), at] -= sign[at % 256] * torch.randint(0, 3, (R,), generator=gen(13 + side))
    cache, rows = store(kv.to(torch.bfloat16))
    assert torch.equal(rows.cpu(), kv.double())
    q = torch.empty(n, H, D)
    q[:, :, :256] = size * sign
    q[:, :, 256:DV] = -size * sign
    q[:, :, DV:] = torch.randint(-size, size + 1, (n, H, D - DV), generator=gen(15)).float()
    q = q.to(torch.bfloat16)
    idx = torch.randint(0, R, (n, topk), generator=gen(16)).to(torch.int32).cuda()
    s0 = (q[0, 0, :256].double() @ kv[:, :256].double().T).abs()
    assert s0.min() > 1300 * size                       # 65504 is left behind with size 64
    got = dsa.dsa_sparse_attn_int4kv(q.cuda(), cache, idx, SCALE, DV)
    ref, tol = attend64(q, rows, idx, exact_sums=True)
    check(got, ref, tol)


@pytest.mark.gpu
@every_division
def test_one_softmax_for_all_value_columns(n, H, topk):
    """Rows whose value columns 256-511 repeat columns 0-255: so does every result, bit for bit, although q differs."""
    kv = latent(500, 17)
    kv[:, 256:DV] = kv[:, :256]
    cache, rows = store(kv)
    q = (2 * torch.randn(n, H, D, generator=gen(18))).to(torch.bfloat16).cuda()
    idx = torch.randint(-20, 500, (n, topk), generator=gen(19)).clamp(min=-1).to(torch.int32).cuda()
    got = dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV)
    assert torch.equal(got[:, :, :256], got[:, :, 256:])
    ref, tol = attend64(q, rows, idx)
    check(got, ref, tol)


@pytest.mark.gpu
@every_division
def test_infinite_rope_columns(n, H, topk):
    """A selected row with an infinite rope column: a logit of +inf makes NaN of the whole head, one of -inf is an
    entry of no weight."""
    kv = latent(400, 20)
    kv[7, DV + 3] = INF                                 # in the share of one SM of a pair,
    kv[8, DV + 40] = -INF                               # in that of the other
    cache, rows = store(kv)
    q = torch.randn(n, H, D, generator=gen(21)).to(torch.bfloat16)
    q[:, :, DV + 3] = -q[:, :, DV + 3].abs() - 1        # -inf for every head ...
    q[:, :, DV + 40] = q[:, :, DV + 40].abs() + 1
    q[:, 0, DV + 3] = 2                                 # ... but the first and the last
    q[:, H - 1, DV + 40] = -2
    idx = torch.randint(9, 400, (n, topk), generator=gen(22)).to(torch.int32)
    idx[:, 5], idx[:, topk - 2] = 7, 8
    got = dsa.dsa_sparse_attn_int4kv(q.cuda(), cache, idx.cuda(), SCALE, DV)
    assert torch.isnan(got[:, 0]).all() and torch.isnan(got[:, H - 1]).all()
    used = idx.clone()
    used[:, 5] = used[:, topk - 2] = -1
    ref, tol = attend64(q[:, 1:H - 1], rows, used)
    check(got[:, 1:H - 1], ref, tol)


# ------------------------------------------------------------------ what splits and their join have to hold

# n, H, topk: decode batches whose entries are split, but for the first between pairs; odd head counts and lengths
SPLIT = [(5, 128, 2048), (8, 128, 2048), (16, 128, 2048), (38, 128, 2048), (32, 64, 2048), (12, 100, 1500),
             (11, 127, 1999), (7, 128, 9001)]


def lists(n, topk, R, seed, kind):
    g = gen(seed)
    idx = torch.randint(0, R, (n, topk), generator=g).to(torch.int32)
    if kind == "ragged":            # most splits of most queries have no entry, some queries none at all
        lens = torch.exp(torch.rand(n, generator=g) * np.log(topk)).long()
        lens[0], lens[n // 2] = topk, 0
        idx[torch.arange(topk)[None] >= lens[:, None]] = -1
    elif kind == "holes":
        idx[torch.rand(n, topk, generator=g) < 0.5] = -1
    elif kind == "tail only":       # the entries of the last split alone, one of them in the first query
        idx[:, :topk - 3] = -1
        idx[0, :topk - 1] = -1
    return idx


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["full", "ragged", "holes", "tail only"])
@pytest.mark.parametrize("n,H,topk", SPLIT)
def test_split_entries(n, H, topk, kind):
    """Slots (some without a row), q rows in another order, a sink; eager, again, and replayed over other lists."""
    assert division(n, H, topk) == ("groups of 32, split" if n == 5 else "pairs, split")
    R, KV, m = 4000, 3000, n + 3
    cache, rows = store(latent(R, 30))
    g = gen(31 + n)
    slots = torch.randperm(R, generator=g)[:KV].to(torch.int32)
    slots[::53] = -1
    slots = slots.cuda()
    q_rows = torch.randperm(m, generator=g)[:n].to(torch.int32)
    q_rows[n - 1] = -1
    at = q_rows[:n - 1].long().cuda()
    q_rows = q_rows.cuda()
    q = torch.randn(m, H, D, generator=g).to(torch.bfloat16).cuda()
    sink = torch.randn(H, generator=g).cuda()
    idx = lists(n, topk, KV, 32, kind).cuda()
    out = torch.full((m, H, DV), 5.0, dtype=torch.bfloat16, device="cuda")

    def run():
        return dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, attn_sink=sink, slots=slots, q_rows=q_rows, out=out)

    def verify():
        ref, tol = attend64(q[at], rows, idx[:n - 1], sink, slots)
        check(out[at], ref, tol)
        rest = torch.ones(m, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (out[rest] == 5.0).all()

    run()
    verify()
    first = out.clone()
    run()
    assert torch.equal(out, first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    out.fill_(5.0)
    idx.copy_(lists(n, topk, KV, 33, "ragged" if kind == "full" else "full"))
    graph.replay()
    verify()


@pytest.mark.gpu
@every_division
def test_bad_entries_of_every_division(n, H, topk):
    """An entry past the cache, past the slots, a slot past the cache and a q row past q: reported, and unused."""
    cache, rows = store(latent(100, 34))
    q = torch.randn(n, H, D, generator=gen(35)).to(torch.bfloat16)
    idx = torch.randint(0, 100, (n, topk), generator=gen(36)).to(torch.int32)
    fine = idx.clone()
    at = (n - 1, topk - 1)
    idx[at], fine[at] = 100, -1
    ref, tol = attend64(q, rows, fine)
    q, idx, fine = q.cuda(), idx.cuda(), fine.cuda()

    def reported(site, got, ref, tol):
        with pytest.raises(dsa.DSAError) as err:
            dsa.dsa_poll_device_error()
        assert err.value.status == 7 and err.value.detail[0] == site
        check(got, ref, tol)

    reported(50, dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV), ref, tol)
    slots = torch.arange(100, dtype=torch.int32).cuda()
    reported(49, dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, slots=slots), ref, tol)
    slots = torch.arange(101, dtype=torch.int32).cuda()
    reported(50, dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, slots=slots), ref, tol)
    out = torch.zeros(n, H, DV, dtype=torch.bfloat16, device="cuda")
    q_rows = torch.arange(n, dtype=torch.int32)
    q_rows[0] = n
    ref[0] = 0
    reported(51, dsa.dsa_sparse_attn_int4kv(q, cache, fine, SCALE, DV, q_rows=q_rows.cuda(), out=out), ref, tol)


@pytest.mark.gpu
@every_division
def test_large_logits_of_every_division(n, H, topk):
    """Logits of hundreds, whose sums are exact (multiples of 2^-6 below 2^18): the running maximum moves in every block (later rows
    larger), or the first entry outweighs the rest; a sink far above every logit, at their level, and far below."""
    R = min(topk, 700)
    size = torch.linspace(1, 7, R).round()
    kv = torch.randint(0, 2, (R, D), generator=gen(37)).float() * 2 - 1
    kv[:, :DV] *= size[:, None]
    cache, rows = store(kv.to(torch.bfloat16))
    assert torch.equal(rows * 64, (rows * 64).round()) and rows.abs().sum(1).max() * 16 < 2 ** 18
    q = (torch.randint(0, 2, (n, H, D), generator=gen(38)) * 32 - 16).to(torch.bfloat16)
    up = (torch.arange(topk) * R // topk).to(torch.int32).repeat(n, 1).cuda()
    for idx in (up, up.flip(1).contiguous()):
        for level in (None, -1e4, 300.0, 1e4):
            sink = None if level is None else torch.full((H,), level).cuda()
            got = dsa.dsa_sparse_attn_int4kv(q.cuda(), cache, idx, SCALE, DV, attn_sink=sink)
            ref, tol = attend64(q, rows, idx, sink, exact_sums=True)
            check(got, ref, tol)
