"""The 4-bit latent cache on the CPU: the oracle's row format against rows
worked by hand, what a stored value may be off by, and the entry points' host
checks (sizes, refusals) without a GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from sparse_attention_prefill_cp_gb300 import _lib
from oracle import dsa_oracle as O


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_row_worked_by_hand():
    # A = 7 * 448 * 2^-9 = 6.125: e = -9, the block's scale 448 (0x7e), step 448 * 2^-9 = 0.875
    x = np.zeros((1, 24))
    x[0, :16] = [6.125, -6.125, 0.875, -0.875, 1.3125, 0.4375, 0, -0.4375, 1.75, 2.625, 3.5, 4.375, 5.25, -1.75,
                 -2.625, -3.5]
    # codes: 1.3125 / 0.875 = 1.5 -> 2 (even), 0.4375 / 0.875 = 0.5 -> 0
    codes = [7, -7, 1, -1, 2, 0, 0, 0, 2, 3, 4, 5, 6, -2, -3, -4]
    x[0, 16:] = [1, -2, 0.5, 0, 3, -0.25, 8, 100]   # rope columns
    row = O.kv_int4_quantize(x, 16)[0]
    assert O.kv_int4_layout(24, 16) == (16, 32, 33, 48) and row.size == 48
    # byte 0: columns 0 and 2, byte 1: 4 and 6, byte 2: 1 and 3, byte 3: 5 and 7
    u = [c + 8 for c in codes]
    want = [u[0] | u[2] << 4, u[4] | u[6] << 4, u[1] | u[3] << 4, u[5] | u[7] << 4,
            u[8] | u[10] << 4, u[12] | u[14] << 4, u[9] | u[11] << 4, u[13] | u[15] << 4]
    assert list(row[:8]) == want and not row[8:16].any()
    assert row[32] == 0x7E and row[33] == 127 - 9 and not row[34:].any()
    assert list(row[16:32].view(np.uint16)) == [0x3F80, 0xC000, 0x3F00, 0, 0x4040, 0xBE80, 0x4100, 0x42C8]
    back = O.kv_int4_dequantize(row[None], 24, 16)[0]
    assert list(back[:16]) == [0.875 * c for c in codes] and list(back[16:]) == list(x[0, 16:])


def test_special_rows():
    x = np.zeros((4, 16))
    x[1, 3], x[2, 5] = np.nan, -np.inf
    x[3, 0] = 2.0 ** -133     # the least bf16
    row = O.kv_int4_quantize(x, 16)
    assert list(row[:, O.kv_int4_layout(16, 16)[2]]) == [3, 255, 255, 3]
    back = O.kv_int4_dequantize(row, 16, 16)
    assert not back[0].any() and np.isnan(back[1:3]).all()
    assert back[3, 0] in (0.0, 2.0 ** -133)


@pytest.mark.parametrize("D,Dv", [(576, 512), (64, 48), (200, 136), (24, 24)])
def test_values_are_bf16_and_near(D, Dv):
    rng = np.random.default_rng(D)
    x = O.bf16_round(rng.standard_normal((9, D)) * np.exp(3 * rng.standard_normal((9, 1)))).astype(np.float64)
    back = O.kv_int4_dequantize(O.kv_int4_quantize(x, Dv), D, Dv)
    assert np.array_equal(O.bf16_round(back), back.astype(np.float32))
    assert np.array_equal(back[:, Dv:], x[:, Dv:])
    for b in range(0, Dv, 16):
        blk = slice(b, min(b + 16, Dv))
        amax, rowmax = np.abs(x[:, blk]).max(1, keepdims=True), np.abs(x[:, :Dv]).max(1, keepdims=True)
        # the scale is off amax / 7 by at most 2^-4 of itself (E4M3), or half its least step, 2^-10 of a power of
        # two below rowmax / (7 * 224); a code by half a step, or where the scale was rounded down, the clamp
        # leaves amax - 7 * scale
        ds = np.maximum(amax / 7 / 16, 2.0 ** -10 * rowmax / (7 * 224))
        off = np.maximum(0.5 * (amax / 7 + ds), 7 * ds)
        assert (np.abs(back[:, blk] - x[:, blk]) <= off * (1 + 1e-12)).all()


def test_row_bytes_match_oracle(lib):
    n = C.c_size_t()
    for D, Dv in [(576, 512), (64, 48), (200, 136), (24, 24), (8, 8), (65536, 65528), (2048, 1032)]:
        assert lib.dsa_kv_int4_row_bytes(D, Dv, C.byref(n)) == 0
        assert n.value == O.kv_int4_layout(D, Dv)[3]
    assert dsa.dsa_kv_int4_row_bytes(576, 512) == 432
    for D, Dv in [(576, 500), (580, 512), (512, 576), (0, 0), (65544, 8), (16, 0)]:
        assert lib.dsa_kv_int4_row_bytes(D, Dv, C.byref(n)) == 2
    assert lib.dsa_kv_int4_row_bytes(576, 512, None) == 1


def test_cache_validation(lib):
    p, odd = C.c_void_p(0x10000), C.c_void_p(0x10008)
    quant, deq = lib.dsa_kv_int4_quantize, lib.dsa_kv_int4_dequantize
    assert quant(None, 576, 4, 576, 512, p, p, 8, None) == 1
    assert quant(odd, 576, 4, 576, 512, p, p, 8, None) == 1
    assert quant(p, 576, 4, 576, 512, p, odd, 8, None) == 1
    assert quant(p, 568, 4, 576, 512, p, p, 8, None) == 2      # rows that overlap
    assert quant(p, 580, 4, 576, 512, p, p, 8, None) == 2      # rows off the 16-byte boundary
    assert quant(p, 576, -1, 576, 512, p, p, 8, None) == 2
    assert quant(p, 576, 4, 576, 512, p, p, -1, None) == 2
    assert quant(p, 576, 9, 576, 512, None, p, 8, None) == 2   # more rows than the cache has, and no slots
    assert quant(p, 576, 4, 576, 508, p, p, 8, None) == 2
    assert quant(None, 576, 0, 576, 512, None, None, 0, None) == 0
    assert deq(p, 8, 576, 512, p, 4, None, None) == 1
    assert deq(odd, 8, 576, 512, p, 4, p, None) == 1
    assert deq(p, 8, 576, 512, None, 9, p, None) == 2
    assert deq(p, -1, 576, 512, p, 4, p, None) == 2
    assert deq(p, 8, 576, 512, p, -4, p, None) == 2
    assert deq(None, 0, 64, 48, None, 0, None, None) == 0


def test_attention_validation(lib):
    p, odd, f = C.c_void_p(0x10000), C.c_void_p(0x10008), C.c_float(0.07)

    def call(q=p, m=4, q_rows=None, n=4, cache=p, rows=16, slots=None, kv=0, idx=p, topk=2048, scale=f, H=128, D=576,
             Dv=512, out=p, ws=None, wsb=0):
        return lib.dsa_sparse_attn_int4kv(q, m, q_rows, n, cache, rows, slots, kv, idx, topk, None, scale, H, D, Dv,
                                          out, ws, wsb, None)

    assert call(n=0) == 0
    for k in ("q", "cache", "idx", "out"):
        assert call(**{k: None}) == 1
    for k in ("q", "cache", "out"):
        assert call(**{k: odd}) == 1
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=C.c_float(bad)) == 1
    assert call(n=5) == 2 and call(n=-1) == 2 and call(m=-1) == 2 and call(rows=-1) == 2 and call(kv=-1) == 2
    assert call(topk=0) == 2
    assert call(H=0) == 3 and call(H=129) == 3 and call(D=64, Dv=48) == 3 and call(Dv=448) == 3
    n = C.c_size_t()
    size = lib.dsa_sparse_attn_int4kv_workspace_size
    assert size(0, 128, 2048, C.byref(n)) == 0 and n.value == 0
    assert size(4, 128, 2048, None) == 1
    assert size(-1, 128, 2048, C.byref(n)) == 2 and size(4, 128, 0, C.byref(n)) == 2
    assert size(4, 129, 2048, C.byref(n)) == 3 and size(4, 0, 2048, C.byref(n)) == 3


def test_wrappers_refuse_what_is_not_on_a_gpu():
    kv, cache = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, 432, dtype=torch.uint8)
    q, idx = torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.dsa_kv_int4_quantize(kv, 512)
    with pytest.raises(ValueError):
        dsa.dsa_kv_int4_dequantize(cache, 576, 512)
    with pytest.raises(ValueError):
        dsa.dsa_sparse_attn_int4kv(q, cache, idx, 0.07, 512)


def test_sizes_past_int32_are_refused():
    """The C ABI counts rows in int32: 2^32 + 4 of them are not 4.  (Tensors without memory.)"""
    from torch._subclasses.fake_tensor import FakeTensorMode
    big = 2 ** 32 + 4
    for call in (lambda: dsa.dsa_kv_int4_row_bytes(2 ** 32 + 576, 512),
                 lambda: dsa.dsa_kv_int4_row_bytes(576, 512 - 2 ** 32),
                 lambda: dsa.dsa_sparse_attn_int4kv_workspace_size(big, 128, 2048)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()

    def t(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device="cuda")

    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    with FakeTensorMode():
        q, cache, idx = t(bf, 4, 16, 576), t(u8, 64, 432), t(i32, 4, 64)
        out = t(bf, 4, 16, 512)
        for call in (lambda: dsa.dsa_kv_int4_quantize(t(bf, big, 8), 8),
                     lambda: dsa.dsa_kv_int4_quantize(t(bf, 4, 8), 8, t(u8, big, 32)),
                     lambda: dsa.dsa_kv_int4_dequantize(t(u8, big, 32), 8, 8),
                     lambda: dsa.dsa_kv_int4_dequantize(t(u8, 64, 32), 8, 8, rows=t(i32, big)),
                     lambda: dsa.dsa_sparse_attn_int4kv(q, t(u8, big, 432), idx, 0.07, 512),
                     lambda: dsa.dsa_sparse_attn_int4kv(q, cache, idx, 0.07, 512, slots=t(i32, big)),
                     lambda: dsa.dsa_sparse_attn_int4kv(q, cache, t(i32, big, 64), 0.07, 512, q_rows=t(i32, big),
                                                        out=out),
                     lambda: dsa.dsa_sparse_attn_int4kv(q, cache, t(i32, 4, big), 0.07, 512)):
            with pytest.raises(ValueError, match="below 2\\^31"):
                call()


def test_division_of_a_call(lib):
    """Splits cover the entries, groups only up to 32 heads, and the workspace follows from the division."""
    for n, H, topk in [(0, 128, 64), (1, 1, 1), (1, 128, 2048), (8, 128, 2048), (64, 16, 2048), (300, 128, 130),
                       (200, 64, 1100), (2048, 128, 2048), (3, 37, 5003)]:
        splits, heads, first = dsa.dsa_sparse_attn_int4kv_division(n, H, topk)
        assert 1 <= splits <= 32 and splits <= -(-topk // (128 if heads else 64)) and heads in (0, 16, 32)
        assert not first or (splits == 1 and heads == 0)
        want = 4 * n if first else n * splits * H * (512 * 4 + 16) if splits > 1 else 0
        assert dsa.dsa_sparse_attn_int4kv_workspace_size(n, H, topk) == want
    f = lib.dsa_sparse_attn_int4kv_division
    assert f(4, 128, 64, None, None, None) == 0
    assert f(-1, 128, 64, None, None, None) == 2 and f(4, 128, 0, None, None, None) == 2
    assert f(4, 0, 64, None, None, None) == 3 and f(4, 129, 64, None, None, None) == 3
