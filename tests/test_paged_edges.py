"""The paged latent cache at the borders of what its calls allow."""
import glob
import os

import pytest
import torch

import sparse_attention_prefill_cp_gb300 as dsa
from conftest import ROOT
from test_paged_gpu import D, gen, randn

CSRC = os.path.join(ROOT, "sparse_attention_prefill_cp_gb300", "csrc")


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
