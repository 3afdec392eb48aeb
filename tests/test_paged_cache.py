"""The paged latent cache on the CPU: the oracle's page tables and choices
against examples worked by hand, and the entry points' host checks (sizes,
refusals) without a GPU."""
import ctypes as C

import numpy as np
import pytest

import sparse_attention_prefill_cp_gb300 as dsa
from sparse_attention_prefill_cp_gb300 import _lib
from oracle import dsa_oracle as O


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_page_table_worked_by_hand():
    # pages of 16; the stack's top is its last valid entry
    table = [[4, -1, -1], [7, 5, -1], [-1, -1, -1]]
    held, seq = [16, 20, 0], [17, 3, 33]
    free, count = [0, 1, 2, 3, 6, 9, 9, 9, 9, 9], 5
    # request 1 releases page 5, which lies on top then; request 0 takes it, request 2 takes 6, 3, 2
    got = O.pages_update(table, held, seq, free, count, 16)
    assert got == ([[4, 5, -1], [7, -1, -1], [6, 3, 2]], [0, 1, 2, 3, 6, 5, 9, 9, 9, 9], 2)
    back = O.pages_update(got[0], seq, held, got[1], got[2], 16)
    assert back[0] == table and back[2] == count and back[1][:count] == free[:count]
    assert O.pages_slots(got[0], held, seq, 16, 40)[:2] == [5 * 16, 6 * 16]
    assert O.pages_slots(got[0], [16, 3, 31], seq, 16, 6) == [80, 3 * 16 + 15, 2 * 16, -1, -1, -1]


@pytest.mark.parametrize("held,seq,free_count", [([0], [49], 3), ([0], [-1], 3), ([-1], [4], 3), ([0], [33], 2),
                                                 ([17], [0], 3)])
def test_page_table_refusals(held, seq, free_count):
    # too long for the table, negative lengths, too few pages, a released entry that is no page
    table = [[2, -1, -1]]
    assert O.pages_update(table, held, seq, [0, 1, 3, 2], free_count, 16) is None


def test_releasing_and_taking_are_inverse():
    rng = np.random.default_rng(0)
    P, width, pool = 16, 6, 40
    lens = [int(x) for x in rng.integers(0, width * P + 1, 5)]
    table, free, count = O.pages_update([[-1] * width] * 5, [0] * 5, lens, list(range(pool)), pool, P)
    for _ in range(20):
        new = [int(x) for x in rng.integers(0, width * P + 1, 5)]
        t2, f2, c2 = O.pages_update(table, lens, new, free, count, P)
        owned = [p for row, n in zip(t2, new) for p in row[:-(-n // P)]]
        assert sorted(owned + f2[:c2]) == list(range(pool))
        back = O.pages_update(t2, new, lens, f2, c2, P)
        assert back[0] == table and back[1][:count] == free[:count] and back[2] == count
        table, free, count, lens = t2, f2, c2, new


def test_selection_worked_by_hand():
    # one head, keys 0 .. 5 along one axis: scores w * relu(q k)
    keys = np.array([[9.0], [1.0], [5.0], [5.0], [-3.0], [0.0]])
    args = (np.array([[2.0]]), np.array([1.0]), keys, list(range(6)))
    assert O.block_select(*args, 6 * 16, 16, 3) == [0, 2, 5]          # first, last, and of the tied the lower
    assert O.block_select(*args, 6 * 16, 16, 4) == [0, 2, 3, 5]
    assert O.block_select(*args, 6 * 16, 16, 4, 0, 2) == [0, 2, 4, 5]
    assert O.block_select(*args, 3 * 16 - 1, 16, 4) == [0, 1, 2, -1]  # all of them
    assert O.block_select(*args, 0, 16, 2) == [-1, -1]
    neg = (np.array([[2.0]]), np.array([-1.0]), keys, list(range(6)))
    assert O.block_select(*neg, 6 * 16, 16, 3) == [0, 4, 5]


def test_attention_over_all_pages_is_the_attention_over_rows():
    rng = np.random.default_rng(1)
    cache = rng.standard_normal((5, 16, 24))
    q = rng.standard_normal((3, 24))
    rows = cache[[4, 1, 2]].reshape(-1, 24)
    for n in (1, 16, 40):
        got = O.paged_attention(q, cache, [4, 1, 2], n, 0.3, 16)
        assert np.allclose(got, O.sparse_attention(q, rows[:n], 0.3, 16))
    got = O.paged_attention(q, cache, [4, 1, 2], 40, 0.3, 16, blocks=[0, 2, -1])
    assert np.allclose(got, O.sparse_attention(q, np.concatenate([rows[:16], rows[32:40]]), 0.3, 16))
    assert not O.paged_attention(q, cache, [4, 1, 2], 40, 0.3, 16, sink=np.ones(3), blocks=[-1]).any()


# ------------------------------------------------------------------ host checks: a status, and no launch

A = 0x10000     # an aligned address, never read


def test_update_host_checks(lib):
    ok = [A, 2, 3, A, A, 16, A, 8, A, None]

    def call(**kw):
        names = ["table", "batch", "max_pages", "held", "seq", "P", "free", "num_pages", "count", "stream"]
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.dsa_pages_update(*[a[n] for n in names])

    assert call(batch=-1) == 2 and call(max_pages=0) == 2 and call(num_pages=-1) == 2
    assert call(batch=1 << 20, max_pages=1 << 12) == 2
    assert call(P=24) == 3 and call(P=8) == 3 and call(P=256) == 3
    for name in ("table", "held", "seq", "free", "count"):
        assert call(**{name: None}) == 1, name
    assert call(batch=0) == 0


def test_slots_host_checks(lib):
    assert lib.dsa_pages_slots(A, 2, 3, None, A, 16, A, -1, None) == 2
    assert lib.dsa_pages_slots(A, -1, 3, None, A, 16, A, 4, None) == 2
    assert lib.dsa_pages_slots(A, 2, 0, None, A, 16, A, 4, None) == 2
    assert lib.dsa_pages_slots(A, 2, 3, None, A, 17, A, 4, None) == 3
    assert lib.dsa_pages_slots(A, 2, 3, None, A, 16, None, 4, None) == 1
    assert lib.dsa_pages_slots(None, 2, 3, None, A, 16, A, 4, None) == 1
    assert lib.dsa_pages_slots(A, 2, 3, None, None, 16, A, 4, None) == 1
    assert lib.dsa_pages_slots(A, 2, 3, None, A, 16, None, 0, None) == 0


def test_append_host_checks(lib):
    names = ["kv", "kv_stride", "k_idx", "slots", "n", "D", "DI", "cache", "page_stride", "row_stride", "num_pages", "P",
             "keys", "means", "stream"]
    ok = [A, 576, A, A, 4, 576, 128, A, 16 * 576, 576, 8, 16, A, A, None]

    def call(**kw):
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.dsa_pages_append(*[a[n] for n in names])

    assert call(n=-1) == 2 and call(num_pages=-1) == 2 and call(D=12) == 2 and call(kv_stride=568) == 2
    assert call(kv_stride=580) == 2 and call(row_stride=568) == 2 and call(row_stride=580) == 2
    assert call(page_stride=16 * 576 + 4) == 2 and call(num_pages=1 << 28) == 2
    assert call(P=48) == 3 and call(DI=136) == 3 and call(DI=12) == 3
    for name in ("kv", "slots", "cache", "keys", "means"):
        assert call(**{name: None}) == 1, name
    for name in ("kv", "k_idx", "cache", "keys", "means"):
        assert call(**{name: A + 8}) == 1, name
    assert call(n=0) == 0


def test_select_host_checks(lib):
    names = ["q", "w", "n", "HI", "DI", "keys", "num_pages", "P", "table", "batch", "max_pages", "lens", "req", "nsel",
             "first", "last", "out", "stream"]
    ok = [A, A, 4, 64, 128, A, 8, 64, A, 4, 10, A, None, 4, 1, 1, A, None]

    def call(**kw):
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.dsa_block_select(*[a[n] for n in names])

    assert call(n=-1) == 2 and call(n=5) == 2 and call(nsel=1) == 2 and call(nsel=0) == 2 and call(last=0) == 2
    assert call(first=-1) == 2 and call(first=4) == 2 and call(num_pages=0) == 2 and call(max_pages=0) == 2
    assert call(n=1 << 20, batch=1 << 20, nsel=1 << 12) == 2
    assert call(HI=65) == 3 and call(HI=0) == 3 and call(DI=64) == 3 and call(P=20) == 3 and call(max_pages=40000) == 3
    for name in ("q", "w", "keys", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
    assert call(q=A + 8) == 1 and call(keys=A + 8) == 1
    assert call(n=0) == 0


def test_attention_host_checks(lib):
    names = ["q", "n", "cache", "page_stride", "row_stride", "num_pages", "P", "table", "batch", "max_pages", "lens",
             "req", "blocks", "nsel", "sink", "scale", "H", "D", "Dv", "out", "ws", "ws_bytes", "stream"]
    need = dsa.dsa_paged_attn_workspace_size(4, 128, 10, 0, 64)
    ok = [A, 4, A, 64 * 576, 576, 8, 64, A, 4, 10, A, None, None, 0, None, 0.07, 128, 576, 512, A, A, need, None]

    def call(**kw):
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.dsa_paged_attn(*[a[n] for n in names])

    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(n=-1) == 2 and call(n=5) == 2 and call(num_pages=0) == 2 and call(max_pages=0) == 2 and call(nsel=-1) == 2
    assert call(row_stride=568) == 2 and call(row_stride=580) == 2 and call(page_stride=64 * 576 + 4) == 2
    assert call(max_pages=1 << 25, batch=4) == 2
    assert call(H=0) == 3 and call(H=129) == 3 and call(D=512) == 3 and call(Dv=576) == 3 and call(P=24) == 3
    for name in ("q", "cache", "table", "lens", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "cache", "out"):
        assert call(**{name: A + 8}) == 1, name
    assert call(blocks=A) == 1 and call(nsel=4) == 1     # one without the other
    assert call(ws=None) == 4 and call(ws_bytes=need - 1) == 4 and call(ws=A + 8) == 4
    assert call(n=0) == 0


def test_workspace_size(lib):
    assert dsa.dsa_paged_attn_workspace_size(0, 128, 10, 0, 64) == 0
    one = dsa.dsa_paged_attn_workspace_size(1, 16, 1, 0, 64)
    assert 0 < one <= dsa.dsa_paged_attn_workspace_size(1, 16, 1000, 0, 64)
    # it does not grow with the batch beyond the SMs
    assert dsa.dsa_paged_attn_workspace_size(4096, 128, 1000, 0, 64) == \
        dsa.dsa_paged_attn_workspace_size(100000, 128, 1000, 0, 64)
    assert lib.dsa_paged_attn_workspace_size(1, 16, 1, 0, 64, None) == 1
    n = C.c_size_t()
    assert lib.dsa_paged_attn_workspace_size(-1, 16, 1, 0, 64, C.byref(n)) == 2
    assert lib.dsa_paged_attn_workspace_size(1, 129, 1, 0, 64, C.byref(n)) == 3
    assert lib.dsa_paged_attn_workspace_size(1, 16, 1, 0, 65, C.byref(n)) == 3
    with pytest.raises(ValueError):
        dsa.dsa_paged_attn_workspace_size(1 << 31, 16, 1, 0, 64)
