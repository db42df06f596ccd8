"""The structures of include/attn.h and include/cache.h as the binding sends them: packed
bytes, held against what a C compiler lays out (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from sparse_dense_linear_amd import _attn, _cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CC = shutil.which("gcc") or shutil.which("cc")

#: structure, its format, its mirror, its fields as a C program names them
PACKED = [
    ("attn_rows_t", _attn._PACK_ROWS, _attn._Rows, "data row_stride head_stride"),
    ("attn_tree_t", _attn._PACK_TREE, _attn._Tree,
     "S Tq Hq Hkv D page page_stride row_stride head_stride table_stride window sinks scale reserved"),
    ("attn_pool_t", _attn._PACK_POOL, _attn._Pool, "k v layers pages page row_bytes"),
    ("cache_scales_t", _attn._PACK_SCALES, _attn._Scales, "k v block page_stride block_stride head_stride"),
    ("cache_pool_t", _attn._PACK_CODE_POOL, _attn._CodePool,
     "pool.k pool.v pool.layers pool.pages pool.page pool.row_bytes k_scale v_scale block heads"),
    ("cache_append_t", _cache._PACK_APPEND, _cache._Append,
     "S T Hq Hkv D page pages page_stride row_stride head_stride table_stride rotated angles interleaved reserved"),
]


def numbers(fmt):
    """A value of its own for each field of a format."""
    return [i + 0.5 if code == "f" else (i << 20) + 3 for i, code in enumerate(codes(fmt), 1)]


def codes(fmt):
    out, count = [], ""
    for c in fmt.format:
        if c.isdigit():
            count += c
        else:
            out += [c] * int(count or 1)
            count = ""
    return out


@pytest.mark.skipif(CC is None, reason="needs a C compiler")
def test_packed_structures_are_those_of_the_headers(tmp_path):
    lines = ['#include <stdio.h>', '#include <string.h>', '#include "cache.h"', "int main(void)", "{"]
    for name, fmt, _, fields in PACKED:
        lines.append(f"    {{ {name} x; memset(&x, 0, sizeof x);")
        for field, code, value in zip(fields.split(), codes(fmt), numbers(fmt)):
            pointer = code == "q" and (field.split(".")[-1] in ("k", "v", "data", "k_scale", "v_scale"))
            lines.append(f"    x.{field} = {f'(void *)(intptr_t){value}' if pointer else value};")
        lines.append("    const unsigned char *b = (const unsigned char *)&x;")
        lines.append(f'    printf("{name} "); for (size_t i = 0; i < sizeof x; ++i) printf("%02x", b[i]); '
                     'printf("\\n"); }')
    lines += ["    return 0;", "}"]
    source, exe = tmp_path / "sizes.c", str(tmp_path / "sizes")
    source.write_text("\n".join(lines))
    subprocess.run([CC, "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(source), "-o", exe], check=True)
    laid_out = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True,
                                                            check=True).stdout.splitlines())
    for name, fmt, _, fields in PACKED:
        assert len(fields.split()) == len(codes(fmt)), name
        assert fmt.pack(*numbers(fmt)).hex() == laid_out[name], name


@pytest.mark.parametrize("name,fmt,mirror,fields", PACKED, ids=[p[0] for p in PACKED])
def test_packed_structures_are_their_mirrors(name, fmt, mirror, fields):
    assert fmt.size == ctypes.sizeof(mirror)
    values = numbers(fmt)
    x = mirror()
    for field, value in zip(fields.split(), values):
        at = x
        for part in field.split(".")[:-1]:
            at = getattr(at, part)
        setattr(at, field.split(".")[-1], value)
    assert bytes(x) == fmt.pack(*values)
