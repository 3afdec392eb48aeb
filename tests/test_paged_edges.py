"""The paged latent cache at the borders of what its calls allow."""
import glob
import os

from conftest import ROOT

CSRC = os.path.join(ROOT, "sparse_attention_prefill_cp_gb300", "csrc")


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
