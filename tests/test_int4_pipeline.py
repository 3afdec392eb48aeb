"""DSAPrefill over the 4-bit latent cache in the geometries that the bf16 path
runs: KV positions before the queries, compressed entries, the sliding window,
and the head-sharded output; in order and through slots."""
import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from sparse_attention_prefill_cp_gb300.pipeline import DSAPrefill
from workloads import IN_SEQ_SPLIT, LONG_8K, ROUND_ROBIN, TINY_INT, chunk_inputs, draw_inputs

pytestmark = pytest.mark.gpu

SMALL = TINY_INT.with_(name="int4-small", lengths=(200, 56), sink=True)
FULL = LONG_8K.with_(name="int4-full", lengths=(2200, 600), cp_size=2, sink=True, seed=33)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    dsa.load()
    yield
    dsa.dsa_poll_device_error()


def paged(kv, Dv, seed):
    """(cache in order, cache through slots, slots, the rows both stand for)."""
    cache = dsa.dsa_kv_int4_quantize(kv, Dv)
    R = cache.shape[0]
    slots = torch.randperm(R + 40, generator=torch.Generator().manual_seed(seed))[:R].to(torch.int32).cuda()
    pages = torch.empty(R + 40, cache.shape[1], dtype=torch.uint8, device="cuda")
    dsa.dsa_kv_int4_quantize(kv, Dv, pages, slots=slots)
    return cache, pages, slots, dsa.dsa_kv_int4_dequantize(cache, kv.shape[1], Dv)


def test_latent_rows_of_a_call_use_the_slots_of_that_call():
    """The rows of a cache in order, after a run over another one through slots."""
    x = {k: v.cuda() for k, v in draw_inputs(SMALL).items()}
    cache, pages, slots, rows = paged(x["kv"], SMALL.Dv, 34)
    wl = SMALL
    pipe = DSAPrefill(wl.lengths, wl.cp_size, ROUND_ROBIN, wl.H, wl.D, wl.Dv, wl.HI, wl.DI, wl.topk, wl.scale,
                      kv_int4=True)
    pipe.run(x["q"], pages, x["q_idx"], x["k_idx"], x["w"], x["sink"], kv_slots=slots)
    assert torch.equal(pipe.latent_kv(cache), rows)
    assert torch.equal(pipe.latent_kv(pages, kv_slots=slots), rows)
    with pytest.raises(ValueError):
        pipe.latent_kv(pages)


def case(kind, wl):
    """(inputs, arguments of DSAPrefill, further ones of run) of a geometry."""
    x, kw, more = draw_inputs(wl), {}, {}
    lengths = list(wl.lengths)
    if "prefix" in kind:
        kw["prefix_lens"] = [n // 2 for n in lengths]
        x, lengths, seq = chunk_inputs(x, lengths, kw["prefix_lens"])
    else:
        seq = lengths
    if "compressed" in kind:
        kw["compress_ratio"] = 4
        R = sum(n // 4 for n in seq)
        if "window" in kind:
            more["kv_ori"] = x["kv"].cuda()
        x["kv"], x["k_idx"] = x["kv"][-R:].contiguous(), x["k_idx"][-R:].contiguous()
    if "window" in kind:
        kw["window"] = 7
    return {k: v.cuda() for k, v in x.items()}, lengths, kw, more


@pytest.mark.parametrize("mode", [IN_SEQ_SPLIT, ROUND_ROBIN])
@pytest.mark.parametrize("kind", ["plain", "prefix", "compressed", "window", "prefix, window",
                                  "compressed, window", "prefix, compressed, window"])
@pytest.mark.parametrize("wl", [SMALL, FULL], ids=lambda w: w.name)
def test_geometries(wl, kind, mode):
    """Dequantised once per batch: the run over the rows that the cache stands for, bit for bit, head-sharded too."""
    x, lengths, kw, more = case(kind, wl)
    args = (lengths, wl.cp_size, mode, wl.H, wl.D, wl.Dv, wl.HI, wl.DI, wl.topk, wl.scale)
    cache, pages, slots, rows = paged(x["kv"], wl.Dv, 36)
    rest = (x["q_idx"], x["k_idx"], x["w"], x["sink"])
    plain = DSAPrefill(*args, **kw)
    want = plain.run(x["q"], rows, *rest, **more).clone()
    pipe = DSAPrefill(*args, kv_int4=True, **kw)
    assert torch.equal(pipe.run(x["q"], cache, *rest, **more), want)
    assert torch.equal(pipe.run(x["q"], pages, *rest, kv_slots=slots, **more), want)
    if "window" not in kind:
        want = plain.run_headsharded(x["q"], rows, *rest).clone()
        assert torch.equal(pipe.run_headsharded(x["q"], cache, *rest), want)
        assert torch.equal(pipe.run_headsharded(x["q"], pages, *rest, kv_slots=slots), want)


@pytest.mark.parametrize("kind", ["prefix", "compressed", "prefix, compressed"])
@pytest.mark.parametrize("fused", [False, True])
def test_geometries_read_by_the_attention(kind, fused):
    """The attention over the cache itself, against the one over the rows it stands for: both within 2^-8 of every
    weight and of the result, and their norms apart by what those roundings come to (2^-9 rms each at most)."""
    wl = FULL
    x, lengths, kw, more = case(kind, wl)
    args = (lengths, wl.cp_size, ROUND_ROBIN, wl.H, wl.D, wl.Dv, wl.HI, wl.DI, wl.topk, wl.scale)
    cache, pages, slots, rows = paged(x["kv"], wl.Dv, 37)
    rest = (x["q_idx"], x["k_idx"], x["w"], x["sink"])
    want = DSAPrefill(*args, **kw).run(x["q"], rows, *rest).clone()
    pipe = DSAPrefill(*args, kv_int4=True, kv_int4_direct=True, fused=fused, **kw)
    for kv, sl in ((cache, None), (pages, slots)):
        got = pipe.run(x["q"], kv, *rest, kv_slots=sl)
        off = (got.double() - want.double()).norm() / want.double().norm()
        assert off <= 1e-2
