"""Planning, attention over shared prefixes and rotation on the GPU where one call meets another: tiles of one CTA,
threads that call at once, a cache that goes on after it was turned. Tolerances as in test_gpu_share.py."""
import pytest
import torch

from test_gpu_cache import DEV, offsets
from test_gpu_share import Shared, attend_prefix, check_prefix, mp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,d,m,n,prefix", [
    (8, 64, 500, 2048, 40),     # 24 CTAs have a tile that sees none of its slots before one that sees some
    (16, 64, 700, 1000, 0),     # 91
    (32, 128, 640, 640, 300),
    (5, 128, 333, 4000, 64),
])
def test_fp32_tiles_behind_tiles_that_see_nothing(mp, hk, d, m, n, prefix):  # noqa: F811
    """The first tiles of a chunk see none of the pieces of its last slots. What such a piece asked for must not come
    over the next tile's rows of Q, however late it comes: Q is out of L2 in every call, and the bits are equal."""
    c = Shared(mp, "f32", hk, hk, d, 64, [n], [1], [prefix])
    cu, cu_t = offsets([m])
    q = c.randn(m, hk, d, by=1.5)
    other = torch.empty(1 << 26, device=DEV)
    first = None
    for i in range(30):
        other.fill_(float(i))
        out, lse = attend_prefix(mp, c, q, cu, cu_t, m)
        first = first if first is not None else (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    check_prefix(c, "f32", q, cu, *first)
    assert c.status.item() == 0
