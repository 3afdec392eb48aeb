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
