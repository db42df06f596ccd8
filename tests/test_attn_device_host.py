"""Device helpers of the attention kernels that the host can run too, in
programs built from the kernels' headers (CPU only, no GPU call)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_dense_linear_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host")
HIPCC = "/opt/rocm/bin/hipcc"


def run_program(tmp_path, name):
    exe = str(tmp_path / name)
    for cmd in ([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-Wall",
                 "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                 "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                 os.path.join(HERE, name + ".cpp"), "-o", exe], [exe]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-4000:]}\n{r.stderr[-4000:]}"
    return r.stdout


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_a_chain_reads_its_own_operands_only(tmp_path):
    assert "chain: ok" in run_program(tmp_path, "attn_chain")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_rows_of_drafts_that_may_be_read(tmp_path):
    assert "drafts: ok" in run_program(tmp_path, "attn_draft")
