"""Device helpers of the kernels over caches of 8 bits that the host can run too, in a
program built from the kernels' headers (CPU only, no GPU call)."""
import os

import pytest

from test_attn_device_host import HIPCC, run_program


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_blocks_of_keys_and_prepared_divisions(tmp_path):
    assert "seen: ok" in run_program(tmp_path, "cache_seen")
