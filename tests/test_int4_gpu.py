"""The 4-bit latent cache on the GPU against the fp64 oracle: bytes written,
values read back (both exact), the attention over it, and a run of them
together.

Tolerance of the attention, elementwise, from its roundings.  With W = sum_j
p_j |v_j| the exact weighted magnitude:
  the result to bf16:                     2^-8 |out|
  each P to bf16 for the product:         2^-8 W
  a logit off by d changes p_j and the denominator by e^d - 1 each: 2 (e^d - 1) W
  fp32 sums of up to 2048 products, exp2 and the logit's fma: 2^-14 W
where d is half an fp16 step of the half of q.k that the pair exchanges,
scale * 2^-11 * max(|S_0|, |S_1|), and 2^-18 of scale * sum_d |q_d k_d| for the
fp32 sum of q.k.
"""
import numpy as np
import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from sparse_attention_prefill_cp_gb300.pipeline import DSAPrefill
from oracle import dsa_oracle as O
from workloads import HEAD_TAIL, IN_SEQ_SPLIT, LONG_8K, ROUND_ROBIN, TINY, draw_inputs

pytestmark = pytest.mark.gpu
D, DV, SCALE = 576, 512, 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    dsa.load()
    yield
    dsa.dsa_poll_device_error()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def latent(n, d, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, d, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))).to(torch.bfloat16)


# ------------------------------------------------------------------ writing and reading back

def special_rows(D, Dv):
    """Rows at the edges of the format: zeros, one value, signed zeros, half steps, huge, tiny, NaN, infinities."""
    g = torch.Generator().manual_seed(D)
    x = torch.randn(14, D, generator=g)
    x[0] = 0
    x[1] = 0
    x[1, Dv - 1] = -3.0
    x[2] = -0.0
    x[3] = torch.randint(-14, 15, (D,), generator=g) / 2          # many half steps: 7 / 7 = 1 a step
    x[3, 0] = 7
    x[4] = torch.randint(-119, 120, (D,), generator=g).float()    # 119 / 7 = 17: midpoints of E4M3
    x[5] *= 3e37
    x[6] = 3.38e38
    x[7] *= 1e-38
    x[8] = 9.2e-41                                                # a bf16 subnormal
    x[9, 3] = float("nan")
    x[10, Dv - 1] = float("inf")
    x[11, 0] = -float("inf")
    x[12, :Dv // 2] *= 1e-6                                       # blocks far below the row's largest
    x[13, Dv:] = float("nan")                                     # rope columns are kept as they are
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("D,Dv,n", [(576, 512, 300), (576, 512, 1), (64, 48, 77), (200, 136, 33), (24, 24, 9),
                                    (8, 8, 3), (1160, 1032, 21)])
def test_bytes_and_values(D, Dv, n):
    x = torch.cat([special_rows(D, Dv), latent(n, D, n)])
    cache = dsa.dsa_kv_int4_quantize(x.cuda(), Dv)
    back = dsa.dsa_kv_int4_dequantize(cache, D, Dv)
    dsa.dsa_poll_device_error()
    ref = O.kv_int4_quantize(x.float().numpy(), Dv)
    assert np.array_equal(cache.cpu().numpy(), ref)
    assert np.array_equal(f64(back), O.kv_int4_dequantize(ref, D, Dv), equal_nan=True)


def test_every_code_scale_and_exponent_reads_back():
    """Rows of every exponent byte the writer leaves, each with all 127 scales and every code."""
    rope, scales, exponent, rb = O.kv_int4_layout(2048, 2040)
    e = np.r_[3:242, 255]
    cache = np.zeros((e.size, rb), dtype=np.uint8)
    cache[:, :1020] = np.random.default_rng(1).integers(0, 256, (e.size, 1020)) | 0x11   # no code 0 ...
    codes = cache[:, :1020]
    codes[(codes & 0xF0) == 0] |= 0x80                                                   # ... in either nibble
    cache[:, scales:scales + 128] = np.minimum(np.arange(128), 126)
    cache[:, exponent] = e
    got = dsa.dsa_kv_int4_dequantize(torch.from_numpy(cache).cuda(), 2048, 2040)
    dsa.dsa_poll_device_error()
    assert np.array_equal(f64(got), O.kv_int4_dequantize(cache, 2048, 2040), equal_nan=True)


def test_slots_and_strided_rows():
    n, R = 45, 128
    wide = latent(n, D + 40, 3).cuda()
    kv = wide[:, 24:24 + D]                                      # rows of a wider projection
    slots = torch.randperm(R, generator=torch.Generator().manual_seed(4))[:n].to(torch.int32)
    slots[5] = slots[17] = -1
    old = torch.randint(0, 256, (R, 432), dtype=torch.uint8, generator=torch.Generator().manual_seed(5))
    cache = old.cuda()
    assert dsa.dsa_kv_int4_quantize(kv, DV, cache, slots=slots.cuda()) is cache
    want = old.numpy().copy()
    ref = O.kv_int4_quantize(kv.float().cpu().numpy(), DV)
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s] = ref[i]
    assert np.array_equal(cache.cpu().numpy(), want)
    dsa.dsa_kv_int4_quantize(kv[:7], DV, cache)                  # rows 0..6, the others as they were
    want[:7] = ref[:7]
    assert np.array_equal(cache.cpu().numpy(), want)
    rows = torch.tensor([slots[0], -1, slots[0], slots[44], 0, -5], dtype=torch.int32).cuda()
    got = f64(dsa.dsa_kv_int4_dequantize(cache, D, DV, rows=rows))
    values = O.kv_int4_dequantize(want, D, DV)
    for i, r in enumerate(rows.tolist()):
        assert np.array_equal(got[i], values[r] if r >= 0 else np.zeros(D), equal_nan=True)
    dsa.dsa_poll_device_error()


def test_out_of_range_rows_are_reported_and_left_out():
    cache = torch.zeros(8, 432, dtype=torch.uint8, device="cuda")
    kv = latent(3, D, 6).cuda()
    dsa.dsa_kv_int4_quantize(kv, DV, cache, slots=torch.tensor([2, 8, 5], dtype=torch.int32, device="cuda"))
    with pytest.raises(dsa.DSAError) as err:
        dsa.dsa_poll_device_error()
    assert err.value.status == 7 and err.value.detail[:2] == (47, 1)
    ref = O.kv_int4_quantize(kv.float().cpu().numpy(), DV)
    want = np.zeros((8, 432), dtype=np.uint8)
    want[2], want[5] = ref[0], ref[2]
    assert np.array_equal(cache.cpu().numpy(), want)
    got = dsa.dsa_kv_int4_dequantize(cache, D, DV, rows=torch.tensor([5, 2147483647], dtype=torch.int32).cuda())
    with pytest.raises(dsa.DSAError) as err:
        dsa.dsa_poll_device_error()
    assert err.value.status == 7 and err.value.detail[:2] == (48, 1)
    assert np.array_equal(f64(got[0]), O.kv_int4_dequantize(want[5:6], D, DV)[0]) and not got[1].any()


def test_empty_calls():
    cache = dsa.dsa_kv_int4_quantize(torch.empty(0, D, dtype=torch.bfloat16, device="cuda"), DV)
    assert tuple(cache.shape) == (0, 432)
    assert tuple(dsa.dsa_kv_int4_dequantize(cache, D, DV).shape) == (0, D)
    some = torch.zeros(4, 432, dtype=torch.uint8, device="cuda")
    out = dsa.dsa_sparse_attn_int4kv(torch.empty(0, 16, D, dtype=torch.bfloat16, device="cuda"), some,
                                     torch.empty(0, 64, dtype=torch.int32, device="cuda"), SCALE, DV)
    assert tuple(out.shape) == (0, 16, DV)


def test_refusals():
    kv, cache = latent(4, D, 7).cuda(), torch.zeros(8, 432, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad in (kv.float(), kv.cpu(), kv[0], kv.t(), latent(4, D + 8, 7).cuda()[:, 1:1 + D],
                latent(4, D + 4, 7).cuda()[:, :D], kv[:1].expand(4, D)):
        with pytest.raises((ValueError, dsa.DSAError)):   # a transposed kv has another row size
            dsa.dsa_kv_int4_quantize(bad, DV, cache)
    for kw in (dict(slots=torch.zeros(4, **i32)), dict(out=cache[:3]), dict(out=cache[:, :431]),
               dict(out=cache, slots=torch.zeros(5, **i32)), dict(out=cache, slots=torch.zeros(4, device="cuda")),
               dict(out=cache, slots=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            dsa.dsa_kv_int4_quantize(kv, DV, **kw)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_kv_int4_quantize(kv, 500)
    for kw in (dict(rows=torch.zeros(2, 2, **i32)), dict(out=torch.empty(8, DV, dtype=torch.bfloat16, device="cuda")),
               dict(rows=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.dsa_kv_int4_dequantize(cache, D, DV, **kw)
    q, idx = torch.zeros(4, 16, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 64, **i32)
    for kw in (dict(q=q.float()), dict(q=q[:, :, :512].contiguous()), dict(q=q[:3]), dict(idx=idx.long()),
               dict(idx=idx[0]), dict(cache=cache[:, :400].contiguous()), dict(attn_sink=torch.zeros(15, device="cuda")),
               dict(slots=torch.zeros(4, 2, **i32)), dict(q_rows=torch.zeros(3, **i32)),
               dict(q_rows=torch.zeros(4, **i32)), dict(out=torch.zeros(4, 16, D, dtype=torch.bfloat16, device="cuda")),
               dict(workspace=torch.zeros(4, device="cuda"))):
        args = dict(q=q, cache=cache, idx=idx)
        args.update({k: v for k, v in kw.items() if k in args})
        with pytest.raises(ValueError):
            dsa.dsa_sparse_attn_int4kv(args["q"], args["cache"], args["idx"], SCALE, DV,
                                       **{k: v for k, v in kw.items() if k not in args})
    with pytest.raises(dsa.DSAError) as err:
        dsa.dsa_sparse_attn_int4kv(torch.zeros(4, 129, D, dtype=torch.bfloat16, device="cuda"), cache, idx, SCALE, DV)
    assert err.value.status == 3
    with pytest.raises(dsa.DSAError) as err:                     # one query of 2048 entries is split
        dsa.dsa_sparse_attn_int4kv(q[:1], cache, torch.zeros(1, 2048, **i32), SCALE, DV,
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert err.value.status == 4
    dsa.dsa_poll_device_error()


# ------------------------------------------------------------------ attention

def attend_ref(q, rows, idx, scale, sink=None, slots=None):
    """(out, tolerance) of the exact attention, computed on the GPU in 64 bits a query at a time."""
    q, rows = q.cuda().double(), rows.cuda()
    n, H = q.shape[:2]
    out = torch.zeros(n, H, DV, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    half = torch.arange(D, device="cuda")
    half = torch.where(half < DV, half // 256, (half - DV) // 32) == 0      # the dims of CTA 0
    for i in range(n):
        pick = idx[i].long()
        pick = pick[pick >= 0]
        if slots is not None:
            pick = slots[pick].long()
            pick = pick[pick >= 0]
        if not pick.numel():
            continue
        k = rows[pick]
        s0 = q[i][:, half] @ k[:, half].T
        s1 = q[i][:, ~half] @ k[:, ~half].T
        l = scale * (s0 + s1)
        m = l.amax(1, keepdim=True)
        p = torch.exp(l - m)
        den = p.sum(1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink.double()[:, None] - m)
        p = p / den
        out[i] = p @ k[:, :DV]
        W = p @ k[:, :DV].abs()
        d = scale * (2.0 ** -11 * torch.maximum(s0.abs(), s1.abs()) + 2.0 ** -18 * (q[i].abs() @ k.abs().T))
        d = d.amax(1, keepdim=True)
        tol[i] = 2.0 ** -8 * out[i].abs() + (2.0 ** -8 + 2 * torch.expm1(d) + 2.0 ** -14) * W + 1e-30
    return out, tol


def make_cache(R, seed):
    """(cache, the values it stands for as float64, both on the GPU)."""
    parts = [dsa.dsa_kv_int4_quantize(latent(min(R - r, 1 << 16), D, seed + r).cuda(), DV) for r in range(0, R, 1 << 16)]
    cache = torch.cat(parts)
    return cache, dsa.dsa_kv_int4_dequantize(cache, D, DV).double()


def draw_idx(n, topk, R, seed, holes="tail"):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, R, (n, topk), generator=g).to(torch.int32)
    if holes == "tail":
        lens = torch.randint(1, topk + 1, (n,), generator=g)
        idx[torch.arange(topk)[None] >= lens[:, None]] = -1
    elif holes == "scattered":
        idx[torch.rand(n, topk, generator=g) < 0.4] = -1
    elif holes == "head":       # whole blocks of unused entries before the first used one
        idx[:, :topk * 3 // 4] = -7
    return idx


CASES = [
    # n, H, topk, R, holes, sink: one token; every head count class; odd sizes; lists that end inside a block
    (1, 128, 2048, 5000, "none", True), (1, 1, 1, 1, "none", False), (1, 128, 64, 64, "none", False),
    (2, 16, 65, 200, "none", True), (3, 128, 2048, 4097, "tail", True), (5, 37, 131, 300, "scattered", False),
    (7, 32, 2048, 3000, "scattered", True), (4, 64, 1000, 900, "head", True), (9, 128, 513, 700, "head", False),
    (64, 128, 2048, 9000, "none", True), (70, 16, 2048, 9000, "tail", False), (77, 8, 200, 300, "tail", True),
    (160, 100, 700, 2000, "scattered", False), (300, 128, 130, 1000, "tail", True), (1, 128, 5003, 9000, "tail", True),
]


@pytest.mark.parametrize("n,H,topk,R,holes,with_sink", CASES)
def test_attention(n, H, topk, R, holes, with_sink):
    cache, rows = make_cache(R, n)
    g = torch.Generator().manual_seed(H)
    q = torch.randn(n, H, D, generator=g).to(torch.bfloat16).cuda()
    sink = torch.randn(H, generator=g).cuda() if with_sink else None
    idx = draw_idx(n, topk, R, topk, holes).cuda()
    got = dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, attn_sink=sink)
    dsa.dsa_poll_device_error()
    ref, tol = attend_ref(q, rows, idx, SCALE, sink)
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), (off / tol).max().item()
    again = dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, attn_sink=sink)
    assert torch.equal(got, again)
    # bf16 rounding alone is 2^-9 rms at most; the bound used for the other attention paths holds too
    norm = ref.norm()
    assert norm == 0 or (got.double() - ref).norm() / norm <= 1e-2


def test_reference_is_the_oracles():
    cache, rows = make_cache(90, 3)
    q = torch.randn(3, 5, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    sink = torch.randn(5, generator=torch.Generator().manual_seed(2))
    idx = draw_idx(3, 40, 90, 4, "scattered")
    idx[1] = -1
    slots = torch.randperm(90, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    slots[:9] = -1
    ref, _ = attend_ref(q, rows, idx.cuda(), SCALE, sink.cuda(), slots.cuda())
    want = O.sparse_attention_entries(f64(q), f64(rows), idx.numpy(), SCALE, DV, f64(sink), slots.numpy())
    assert np.abs(f64(ref) - want).max() < 1e-12


@pytest.mark.parametrize("n", [3, 200])
def test_rows_without_entries_and_masked_nan(n):
    """Queries with nothing to attend to get zeros, split or not, with a sink or without; what the unused rows of the
    cache and the unused entries hold does not matter."""
    cache, rows = make_cache(400, 8)
    bad = latent(4, D, 9)
    bad[:, 7] = float("nan")
    bad[:, 540] = float("inf")
    dsa.dsa_kv_int4_quantize(bad.cuda(), DV, cache[100:104])
    idx = draw_idx(n, 300, 100, 10, "scattered")
    idx[0] = -1
    idx[n - 1, 1:] = -2147483648
    idx[n - 1, 0] = -1
    idx[1, :] = -1
    idx[1, 299] = 5
    q = torch.randn(n, 128, D, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).cuda()
    for sink in (None, torch.full((128,), 2.0).cuda(), torch.full((128,), -float("inf")).cuda()):
        got = dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, attn_sink=sink)
        ref, tol = attend_ref(q, rows, idx.cuda(), SCALE, sink)
        assert ((got.double() - ref).abs() <= tol).all()
        assert not got[0].any() and not got[n - 1].any()
    sel = idx.cuda().clone()
    sel[2, 3] = 101                                    # a row that holds a NaN, selected by one query
    got = dsa.dsa_sparse_attn_int4kv(q, cache, sel, SCALE, DV)
    assert torch.isnan(got[2]).all() and torch.isfinite(torch.cat([got[:2], got[3:]])).all()
    dsa.dsa_poll_device_error()


@pytest.mark.parametrize("n", [2, 90])
def test_large_logits_and_a_dominant_sink(n):
    """Logits of hundreds: the running maximum moves block by block (later rows larger), or all but one entry
    vanishes; a sink far above every logit leaves nearly nothing, one far below changes nothing."""
    R = 640
    x = latent(R, D, 12, 0.0).float() * torch.linspace(0.05, 6, R)[:, None]
    cache = dsa.dsa_kv_int4_quantize(x.to(torch.bfloat16).cuda(), DV)
    rows = dsa.dsa_kv_int4_dequantize(cache, D, DV).double()
    q = (8 * torch.randn(n, 24, D, generator=torch.Generator().manual_seed(13))).to(torch.bfloat16).cuda()
    idx = torch.arange(R, dtype=torch.int32).repeat(n, 1).cuda()
    for order in (idx, idx.flip(1).contiguous()):
        for level in (None, -1e4, 1e4):
            sink = None if level is None else torch.full((24,), level).cuda()
            got = dsa.dsa_sparse_attn_int4kv(q, cache, order, SCALE, DV, attn_sink=sink)
            ref, tol = attend_ref(q, rows, order, SCALE, sink)
            assert ((got.double() - ref).abs() <= tol).all()
    dsa.dsa_poll_device_error()


@pytest.mark.parametrize("n", [4, 120])
def test_slots_and_query_rows(n):
    R, KV, H = 900, 700, 48
    cache, rows = make_cache(R, 14)
    g = torch.Generator().manual_seed(15)
    slots = torch.randperm(R, generator=g)[:KV].to(torch.int32)
    slots[50:60] = -1
    idx = draw_idx(n, 333, KV, 16, "tail")
    m = n + 5
    q = torch.randn(m, H, D, generator=g).to(torch.bfloat16).cuda()
    q_rows = torch.randperm(m, generator=g)[:n].to(torch.int32)
    q_rows[1] = -1
    out = torch.full((m, H, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    got = dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, slots=slots.cuda(), q_rows=q_rows.cuda(), out=out)
    assert got is out
    dsa.dsa_poll_device_error()
    keep = [i for i in range(n) if q_rows[i] >= 0]
    at = q_rows[keep].long().cuda()
    ref, tol = attend_ref(q[at], rows, idx[keep].cuda(), SCALE, None, slots.cuda())
    assert ((out[at].double() - ref).abs() <= tol).all()
    rest = torch.ones(m, dtype=torch.bool)
    rest[at.cpu()] = False
    assert (out[rest.cuda()] == 7.0).all()


@pytest.mark.parametrize("n", [2, 100])
def test_bad_entries_are_reported_and_unused(n):
    cache, rows = make_cache(100, 17)
    q = torch.randn(n, 16, D, generator=torch.Generator().manual_seed(18)).to(torch.bfloat16).cuda()
    idx = draw_idx(n, 200, 100, 19, "none")
    fine = idx.clone()
    idx[1, 70], fine[1, 70] = 100, -1
    ref, tol = attend_ref(q, rows, fine.cuda(), SCALE)

    def check(site, got, ref, tol):
        with pytest.raises(dsa.DSAError) as err:
            dsa.dsa_poll_device_error()
        assert err.value.status == 7 and err.value.detail[0] == site
        assert ((got.double() - ref).abs() <= tol).all()

    check(50, dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV), ref, tol)
    slots = torch.arange(100, dtype=torch.int32).cuda()
    check(49, dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, slots=slots), ref, tol)
    slots = torch.arange(101, dtype=torch.int32).cuda()
    check(50, dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, slots=slots), ref, tol)
    out = torch.zeros(n, 16, DV, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(n, dtype=torch.int32)
    at[0] = n
    ref[0] = 0
    check(51, dsa.dsa_sparse_attn_int4kv(q, cache, fine.cuda(), SCALE, DV, q_rows=at.cuda(), out=out), ref, tol)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: rows written, read and attended to behind that border."""
    R = (1 << 32) // 432 + 5000
    cache = torch.zeros(R, 432, dtype=torch.uint8, device="cuda")
    n = 300
    kv = latent(n, D, 20).cuda()
    slots = (R - 1 - 16 * torch.arange(n)).to(torch.int32).cuda()
    dsa.dsa_kv_int4_quantize(kv, DV, cache, slots=slots)
    small = dsa.dsa_kv_int4_quantize(kv, DV)
    assert torch.equal(cache[slots.long()], small)
    assert torch.equal(dsa.dsa_kv_int4_dequantize(cache, D, DV, rows=slots), dsa.dsa_kv_int4_dequantize(small, D, DV))
    q = torch.randn(2, 128, D, generator=torch.Generator().manual_seed(21)).to(torch.bfloat16).cuda()
    near = torch.arange(n, dtype=torch.int32, device="cuda").repeat(2, 1)
    far = slots.repeat(2, 1)
    assert torch.equal(dsa.dsa_sparse_attn_int4kv(q, cache, far, SCALE, DV),
                       dsa.dsa_sparse_attn_int4kv(q, small, near, SCALE, DV))
    dsa.dsa_poll_device_error()


def test_streams_and_graphs():
    """Calls on a side stream, and a captured decode step (write, attend) replayed over changed inputs."""
    cache, _ = make_cache(512, 22)
    q = torch.randn(3, 128, D, generator=torch.Generator().manual_seed(23)).to(torch.bfloat16).cuda()
    idx = draw_idx(3, 500, 512, 24, "scattered").cuda()
    kv = latent(3, D, 25).cuda()
    slots = torch.tensor([7, 300, 511], dtype=torch.int32, device="cuda")

    def step(stream=None):
        dsa.dsa_kv_int4_quantize(kv, DV, cache, slots=slots, stream=stream)
        return dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (26, 27):
        kv.copy_(latent(3, D, seed))
        idx.copy_(draw_idx(3, 500, 512, seed, "tail"))
        q.copy_(torch.randn(3, 128, D, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, step())
    dsa.dsa_poll_device_error()


def test_empty_slots_are_refused():
    """Slots without a row name none; they are not the call without slots."""
    cache, _ = make_cache(8, 40)
    q = torch.zeros(2, 16, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, slots=none)
    assert dsa.dsa_sparse_attn_int4kv(q[:0], cache, idx[:0], SCALE, DV, slots=none).shape == (0, 16, DV)


@pytest.mark.parametrize("n,H,topk", [(1, 100, 2048), (2, 64, 700), (1, 33, 64), (2, 128, 129), (1, 17, 9000),
                                      (1, 49, 4097), (2, 127, 2048)])
def test_a_query_or_two_of_many_heads(n, H, topk):
    """The division over groups of heads, the last of them partial, with a sink, slots and holes."""
    R, KV = 5000, 4000
    cache, rows = make_cache(R, 41)
    g = torch.Generator().manual_seed(42 + H)
    slots = torch.randperm(R, generator=g)[:KV].to(torch.int32)
    slots[::97] = -1
    idx = draw_idx(n, topk, KV, 43, "scattered")
    q = torch.randn(n, H, D, generator=g).to(torch.bfloat16).cuda()
    sink = torch.randn(H, generator=g).cuda()
    got = dsa.dsa_sparse_attn_int4kv(q, cache, idx.cuda(), SCALE, DV, attn_sink=sink, slots=slots.cuda())
    dsa.dsa_poll_device_error()
    ref, tol = attend_ref(q, rows, idx.cuda(), SCALE, sink, slots.cuda())
    assert ((got.double() - ref).abs() <= tol).all()


def test_two_streams_at_once():
    """Calls of different divisions on two streams, each with the workspace of its own stream."""
    cache, _ = make_cache(3000, 44)
    g = torch.Generator().manual_seed(45)
    calls = []
    for n, H, topk in ((3, 128, 2048), (5, 16, 2048), (90, 128, 300), (1, 64, 2048)):
        q = torch.randn(n, H, D, generator=g).to(torch.bfloat16).cuda()
        idx = draw_idx(n, topk, 3000, n, "scattered").cuda()
        calls.append((q, idx, dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            for q, idx, _want in calls if k == 0 else calls[::-1]:
                got[k].append(dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, stream=st))
    torch.cuda.synchronize()
    for k in range(2):
        order = calls if k == 0 else calls[::-1]
        for i, out in enumerate(got[k]):
            assert torch.equal(out, order[i % len(calls)][2])
    dsa.dsa_poll_device_error()


@pytest.mark.parametrize("n,H,topk", [(200, 128, 130), (160, 16, 300), (1, 128, 2048), (6, 32, 2048)])
def test_replays_of_every_division(n, H, topk):
    """A captured call replayed over changed inputs: pairs and groups, one pass and split with a join."""
    cache, _ = make_cache(2500, 46)
    g = torch.Generator().manual_seed(47)
    q = torch.randn(n, H, D, generator=g).to(torch.bfloat16).cuda()
    idx = draw_idx(n, topk, 2500, 48, "tail").cuda()
    dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV)
    for seed in (49, 50):
        q.copy_(torch.randn(n, H, D, generator=torch.Generator().manual_seed(seed)))
        idx.copy_(draw_idx(n, topk, 2500, seed, "scattered"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV))
    dsa.dsa_poll_device_error()


@pytest.mark.parametrize("n,H", [(152, 128), (181, 70), (304, 40), (305, 40)])
def test_ragged_lists_of_many_queries(n, H):
    """Two to four waves of long lists are taken longest first: lists of every length, empty and head-masked ones, rows
    without a query, and replays over other lengths, where the order has to be made anew."""
    R, m, topk = 3000, n + 3, 1100
    cache, rows = make_cache(R, 51)
    g = torch.Generator().manual_seed(52)

    def lists():
        idx = torch.randint(0, R, (n, topk), generator=g).to(torch.int32)
        lens = torch.exp(torch.rand(n, generator=g) * 7.2).long().clamp(max=topk)
        lens[:2] = torch.tensor([0, topk])
        idx[torch.arange(topk)[None] >= lens[:, None]] = -1
        idx[5, : topk - 3], idx[5, topk - 3 :] = -1, 7
        return idx.cuda()

    q_rows = torch.randperm(m, generator=g)[:n].to(torch.int32)
    q_rows[9] = -1
    q_rows = q_rows.cuda()
    q = torch.randn(m, H, D, generator=g).to(torch.bfloat16).cuda()
    out = torch.full((m, H, DV), 3.0, dtype=torch.bfloat16, device="cuda")
    idx = lists()

    def run():
        return dsa.dsa_sparse_attn_int4kv(q, cache, idx, SCALE, DV, q_rows=q_rows, out=out)

    def check():
        torch.cuda.synchronize()
        use = q_rows >= 0
        at = q_rows[use].long()
        ref, tol = attend_ref(q[at], rows, idx[use], SCALE)
        assert ((out[at].double() - ref).abs() <= tol).all()
        rest = torch.ones(m, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (out[rest] == 3.0).all()

    run()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        idx.copy_(lists())
        out.fill_(3.0)
        graph.replay()
        check()
    dsa.dsa_poll_device_error()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("page", [64, 16])
def test_prefill_then_decode_over_pages(page):
    """Three requests in pages scattered over one cache: the prompts' rows written in two chunks, then tokens one at a
    time -- each written, its query attending to a selection of its request's rows -- against the oracle's bytes and
    its attention over their values; pages of no request keep their bytes."""
    g = torch.Generator().manual_seed(28)
    prompts, steps, H, topk = [130, 1, 77], 4, 16, 96
    total = [p + steps for p in prompts]
    need = [-(-t // page) for t in total]
    pages = torch.randperm(sum(need) + 3, generator=g)
    R = pages.numel() * page
    table, at = [], 0
    for k in need:
        table.append(pages[at:at + k])
        at += k
    where = [torch.cat([t * page + torch.arange(page) for t in tb])[:n].to(torch.int32) for tb, n in zip(table, total)]
    kv = [latent(n, D, 29 + i) for i, n in enumerate(total)]
    old = torch.randint(0, 256, (R, 432), dtype=torch.uint8, generator=g)
    cache, want = old.cuda(), old.numpy().copy()
    for i, p in enumerate(prompts):
        for a, b in ((0, p // 2), (p // 2, p)):
            dsa.dsa_kv_int4_quantize(kv[i][a:b].cuda(), DV, cache, slots=where[i][a:b].cuda())
        want[where[i][:p].long()] = O.kv_int4_quantize(kv[i][:p].float().numpy(), DV)
    base = np.cumsum([0] + total)
    slots = torch.cat(where).cuda()                    # KV row (requests one after another) -> cache row
    for t in range(steps):
        new = torch.stack([kv[i][p + t] for i, p in enumerate(prompts)])
        at = torch.stack([where[i][p + t] for i, p in enumerate(prompts)])
        dsa.dsa_kv_int4_quantize(new.cuda(), DV, cache, slots=at.cuda())
        want[at.long()] = O.kv_int4_quantize(new.float().numpy(), DV)
        idx = torch.full((3, topk), -1, dtype=torch.int32)
        for i, p in enumerate(prompts):
            seen = p + t + 1
            pick = torch.randperm(seen, generator=g)[:topk].sort().values
            idx[i, :pick.numel()] = (pick + int(base[i])).to(torch.int32)
        q = torch.randn(3, H, D, generator=g).to(torch.bfloat16)
        got = dsa.dsa_sparse_attn_int4kv(q.cuda(), cache, idx.cuda(), SCALE, DV, slots=slots)
        rows = torch.from_numpy(O.kv_int4_dequantize(want, D, DV))
        ref, tol = attend_ref(q, rows, idx.cuda(), SCALE, None, slots)
        assert ((got.double() - ref).abs() <= tol).all()
    assert np.array_equal(cache.cpu().numpy(), want)
    dsa.dsa_poll_device_error()


@pytest.mark.parametrize("mode", [IN_SEQ_SPLIT, ROUND_ROBIN, HEAD_TAIL])
@pytest.mark.parametrize("wl", [TINY, LONG_8K.with_(name="int4-2x", lengths=(600, 2300, 5), cp_size=3, seed=31)],
                         ids=lambda w: w.name)
def test_prefill_pipeline_over_the_cache(wl, mode):
    """DSAPrefill(kv_int4=True) is DSAPrefill over the rows the cache stands for, in order or through slots."""
    x = {k: (v.cuda() if v is not None else None) for k, v in draw_inputs(wl).items()}
    args = (wl.lengths, wl.cp_size, mode, wl.H, wl.D, wl.Dv, wl.HI, wl.DI, wl.topk, wl.scale)
    cache = dsa.dsa_kv_int4_quantize(x["kv"], wl.Dv)
    rows = dsa.dsa_kv_int4_dequantize(cache, wl.D, wl.Dv)
    want = DSAPrefill(*args).run(x["q"], rows, x["q_idx"], x["k_idx"], x["w"], x["sink"])
    R = cache.shape[0]
    slots = torch.randperm(R + 40, generator=torch.Generator().manual_seed(32))[:R].to(torch.int32).cuda()
    paged = torch.empty(R + 40, cache.shape[1], dtype=torch.uint8, device="cuda")
    dsa.dsa_kv_int4_quantize(x["kv"], wl.Dv, paged, slots=slots)
    for kv, sl in ((cache, None), (paged, slots)):
        pipe = DSAPrefill(*args, kv_int4=True)
        got = pipe.run(x["q"], kv, x["q_idx"], x["k_idx"], x["w"], x["sink"], kv_slots=sl)
        assert torch.equal(got, want)
        if wl.D != D:
            continue
        for fused in (False, True):
            pipe = DSAPrefill(*args, kv_int4=True, kv_int4_direct=True, fused=fused, view_streams=2)
            got = pipe.run(x["q"], kv, x["q_idx"], x["k_idx"], x["w"], x["sink"], kv_slots=sl)
            for r in range(wl.cp_size):
                pos = pipe.md[r].token_pos.long()
                use = pos >= 0
                ref, tol = attend_ref(x["q"][pos[use]], rows.double(), pipe.topk_idx[r][use], wl.scale, x["sink"])
                assert ((got[pos[use]].double() - ref).abs() <= tol).all()
    dsa.dsa_poll_device_error()


def test_pipeline_refusals():
    args = (TINY.lengths, TINY.cp_size, 0, TINY.H, TINY.D, TINY.Dv, TINY.HI, TINY.DI, TINY.topk, TINY.scale)
    for kw in (dict(kv_int4=True, kv_fp8=True), dict(kv_int4_direct=True), dict(kv_int4=True, kv_int4_direct=True),
               dict(kv_int4=True, kv_int4_direct=True, window=4)):
        with pytest.raises(ValueError):
            DSAPrefill(*args, **kw)
    pipe = DSAPrefill(*args)
    x = {k: (v.cuda() if v is not None else None) for k, v in draw_inputs(TINY).items()}
    with pytest.raises(ValueError):
        pipe.run(x["q"], x["kv"], x["q_idx"], x["k_idx"], x["w"], kv_slots=torch.zeros(4, dtype=torch.int32).cuda())
