"""Where appended rows may look things up (attn/draft.h), in a program built from the
kernels' headers (CPU only, no GPU call)."""
import os

import pytest

from test_attn_device_host import HIPCC, run_program


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_places_in_front_of_the_tables_and_of_a_sequence(tmp_path):
    assert "places: ok" in run_program(tmp_path, "cache_places")
