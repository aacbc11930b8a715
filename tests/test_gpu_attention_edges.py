"""Attention of drafted tokens at the edges of its range: infinities without
weight, against the formula in 64 bits."""
import pytest
import torch

from decode_helpers import Drafted

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]

# (heads of a key/value head, drafted tokens): row tiles of 16, 32, 128 and 256
# rows, and two tiles of 256
SHAPES = [(2, 2), (4, 6), (4, 12), (4, 40), (2, 150)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,draft", SHAPES)
@pytest.mark.parametrize("ctx,others", [(0, 0), (61, 0), (3000, 0), (200, 150)])
def test_infinities_of_drafts_with_and_without_weight(gpu, group, draft, ctx, others, dtype):
    """An infinite v of a drafted token counts p v, as any other: infinity, or NaN
    where p underflows to 0. The first draft's score lies 1100 below the other keys'
    (p is 0 in 64 bits too), the second one's among them. In one block and cut over
    many."""
    c = Drafted(gpu, [ctx] + [200] * others, [draft] * (1 + others), group=group, dtype=dtype, seed=draft)
    c.q.fill_(1.0)
    for t, key, value in ((0, -100.0, float("inf")), (1, 0.0, float("-inf"))):
        p, o = int(c.cache.page_table[0, (ctx + t) // 16]), (ctx + t) % 16
        c.cache.k[0, p, :, o] = key
        c.cache.v[0, p, :, o, t::5] = value
    out, lse = c.run()
    c.check(out, lse)
    torch.cuda.synchronize()
    # by hand: row 0 of a sequence without committed tokens sees the first draft alone
    first = out[0, 0, 0::5]
    assert (first == float("inf")).all() if ctx == 0 else torch.isnan(first).all()
    assert (out[1, 0, 1::5] == float("-inf")).all()

