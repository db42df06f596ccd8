"""A paged cache that is appended to and held in 8 bits (include/cache.h) at the edges of
its definition: contexts, values and scales that calls seldom have."""
import pytest
import torch

import sparse_dense_linear_amd as sdl
from cache_ref import E4M3, INT8
from test_gpu_cache import BF16, CODES, F32, KINDS, TYPES, a_pool, bits, i32, tables

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@TYPES
@KINDS
@pytest.mark.parametrize("ctx", [-1, -3, -8, -17, -(1 << 30)])
def test_append_in_front_of_a_sequence(dtype, kind, ctx):
    """Rows at negative positions are passed over and their rotated elements are NaN; the
    rows behind them are as if they came alone."""
    new, page, block, D, rotated = 12, 16, 8, 64, 32
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(new, h, D, generator=g).to(dtype).cuda() for h in (4, 2, 2))
    cos, sin = (x.cuda() for x in tables(20, rotated))
    made = [None if x is None else x.cuda() for x in a_pool(3, page, block, 2, D, kind, dtype, g)]
    got, want = ([None if x is None else x.clone() for x in made] for _ in range(2))
    table, front = i32([[1, 2]]), min(-ctx, new)

    def call(pools, first, at):
        kw = {} if kind is None else dict(k_scale=pools[2], v_scale=pools[3])
        a = (x[first:].contiguous() for x in (k, v))
        return sdl.append_pages(*a, pools[0], pools[1], table, i32([at]), i32([0, new - first]),
                                q=q[first:].contiguous(), cos=cos, sin=sin, **kw)

    out = call(got, 0, ctx)
    if front < new:
        assert torch.equal(out[front:], call(want, front, 0))
    assert bool(out[:front, :, :rotated].isnan().all())
    assert torch.equal(out[:front, :, rotated:], q[:front, :, rotated:])
    for x, y in zip(got, want):
        assert x is None or torch.equal(bits(x), bits(y))
