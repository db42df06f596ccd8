"""The host code behind include/attn.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only, no GPU call), built as
test_sanitizers.py builds the rest of the library."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, HOST_SAN, ROOT, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_attention_host_paths_under_sanitizers(tmp_path):
    flags = ["--offload-arch=gfx950", "-std=c++17", "-fPIC", "-O1", "-Xarch_device", "-O0",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC] + HOST_SAN
    sources = [os.path.join(d, f) for d in (CSRC, os.path.join(CSRC, "attn")) for f in sorted(os.listdir(d))
               if f.endswith(".hip") and f != "ceiling.hip"]

    def compile_one(src):
        obj = str(tmp_path / (os.path.relpath(src, CSRC).replace("/", "_") + ".o"))
        _run([HIPCC] + flags + ["-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources))
    main = str(tmp_path / "attn_host_args.o")
    _run([HIPCC, "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "include")] + HOST_SAN +
         ["-c", os.path.join(HERE, "attn_host_args.cpp"), "-o", main])
    exe = str(tmp_path / "attn_host_args")
    _run([HIPCC, "--offload-arch=gfx950"] + HOST_SAN + objs + [main, "-o", exe])
    assert "attention argument paths: ok" in _run([exe], env=ENV).stdout
