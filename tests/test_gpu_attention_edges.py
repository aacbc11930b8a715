"""Attention of drafted tokens at the edges of its range: infinities without
weight, scores beyond 2^27, many row tiles, offsets that have to be cut, against
the formula in 64 bits; waits that give up."""
import pytest
import torch

from decode_helpers import Drafted, check_attention, ints
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,draft", SHAPES)
@pytest.mark.parametrize("power", [10, 13, 14, 15])
def test_scores_far_beyond_a_million(gpu, group, draft, dtype, power):
    """q . k exact in fp32 and so far apart that the largest one takes all: the
    result is its v, or the mean of the two that share it. (Scores up to
    2^(7 + 2 power) / 8, in units of log 2 with a rounding of 2^-24 of that, which
    must not reach e^x.)"""
    ctx = 700
    c = Drafted(gpu, [ctx, 90], [draft, draft], group=group, dtype=dtype, seed=power)
    heads = torch.arange(c.q.shape[1], device=gpu)
    # (finer than powers of two: their products with the scale would be exact)
    c.q.copy_((1.0 + heads / 64.0)[None, :, None] * 2.0 ** power)
    for s in range(2):
        n = c.lens[s] + draft
        rank = torch.randperm(c.lens[s], device=gpu, generator=torch.Generator(gpu).manual_seed(s))
        rank = (rank // 2 + 1).float() / (c.lens[s] // 2 + 1)          # pairs share a score
        level = torch.cat([rank, torch.full((draft,), -1.0, device=gpu)])
        pos = torch.arange(n, device=gpu)
        pages = c.cache.page_table[s].long()[pos // 16]
        for h in range(2):
            c.cache.k[0][pages, h, pos % 16] = ((level * 60).round() / 64 * 2.0 ** power)[:, None].to(dtype)
    out, lse = c.run()
    torch.cuda.synchronize()
    for i, s in enumerate((0, 1)):
        k, v = c.rows_of(s)
        for h in range(c.q.shape[1]):
            kh, vh = k[h // group], v[h // group]
            top = kh[:, 0] == kh[:, 0].max()
            assert top[:c.lens[s]].any() and not top[c.lens[s]:].any()
            want = vh[top].mean(0)
            # the keys at the top share one probability (1 up to the rounding of the
            # offset), which is rounded to the output's type, as is the result; the
            # sums are off by 2^-22 at most
            u = torch.finfo(dtype).eps / 2
            tol = (2 * u + u * u) * want.abs() + 2.0 ** -22 * vh[top].abs().mean(0)
            got = out[c.cu_host[i]:c.cu_host[i + 1], h].double()
            assert ((got - want).abs() <= tol).all(), (s, h, (got - want).abs().max())
            x = float(c.q[0, h].double() @ kh[top][0]) * c.scale
            assert ((lse[c.cu_host[i]:c.cu_host[i + 1], h].double() - x).abs() <= abs(x) * 2.0 ** -21).all()
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)


# row tiles of 128 and of 256 rows, and the second group of 128 with few rows
@pytest.mark.parametrize("group,draft", [(4, 20), (4, 60), (4, 33), (8, 40)])
@pytest.mark.parametrize("position", [0, 1])
def test_a_wait_for_outputs_that_gives_up_is_reported(gpu, group, draft, position):
    """Products are under way when the softmax stops waiting for them: they end before
    the block gives its tensor memory back, the call ends with an error, and the
    calls behind it are right."""
    c = Drafted(gpu, [30000, 600, 9], [draft] * 3, group=group, kv_heads=1, page=32, tree="random")
    want = c.run()
    for _ in range(10):
        P.test_set_skip(P.SKIP_ATTENTION_OUTPUTS, position)
        try:
            c.run()
        finally:
            P.test_set_skip(P.SKIP_OFF)
        again = c.run()
        torch.cuda.synchronize()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
        st = D.cache_status(c.cache)
        # (a block's run may lie in one stretch: then there is no second one)
        assert st == (P.PROX_ETIMEOUT, D.CACHE_TIMEOUT) or position == 1 and st == (P.PROX_OK, 0)
    c.check(*want)


# rows of a key/value head beyond two tiles of 256: up to 64 tiles
@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("group,draft", [(3, 171), (4, 256), (8, 160), (8, 256), (64, 256)])
def test_many_row_tiles(gpu, group, draft, dim, dtype):
    c = Drafted(gpu, [70, 1000], [draft, draft - 37], group=group, kv_heads=1, dim=dim, dtype=dtype, page=64,
                tree="random", seed=group)
    c.check(*c.run())
    # one sequence alone: its tiles are cut over the blocks
    c = Drafted(gpu, [5000], [draft], group=group, kv_heads=1, dim=dim, dtype=dtype, page=128, seed=group)
    c.check(*c.run())
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)


@pytest.mark.parametrize("group,draft", [(4, 4), (2, 12), (4, 20), (4, 70)])
def test_offsets_that_are_cut_leave_the_other_rows(gpu, group, draft):
    """Rows up to the cut follow the formula; rows behind it, and the gaps between
    rows, keep what they hold."""
    c = Drafted(gpu, [30], [draft], group=group, extra_rows=5)
    heads = c.q.shape[1]

    def run(cu, max_q):
        c.cu, c.max_q = ints(cu, gpu), max_q
        c.seqs = ints([0] * (len(cu) - 1), gpu)
        wide = torch.full((draft + 5, heads + 3, 128), 3.0, dtype=c.q.dtype, device=gpu)
        lse = torch.full((draft + 5, heads), 7.0, device=gpu)
        c.run(out=wide[:, :heads], lse=lse)
        torch.cuda.synchronize()
        assert (wide[:, heads:] == 3).all()
        return wide[:, :heads], lse, D.cache_status(c.cache)[1]

    def check(out, lse, a, b, flags):
        """Rows a .. b - 1 are a chain of b - a drafted tokens, the others untouched."""
        k, v = (x[:, :30 + b - a] for x in c.rows_of(0))
        seen = torch.ones((b - a, 30 + b - a), dtype=torch.bool, device=gpu).tril(30)
        check_attention(out[a:b], lse[a:b], c.q[a:b], k, v, seen, c.scale)
        rest = torch.ones(draft + 5, dtype=torch.bool, device=gpu)
        rest[a:b] = False
        assert (out[rest] == 3).all() and (lse[rest] == 7).all()
        assert flags == D.CACHE_BAD_ARG

    for cu, first in (([0, 10 ** 6], 0),            # behind the tensor's last row
                      ([0, draft + 5], 0),          # more than max_q
                      ([-3, draft], 0),             # before its first row
                      ([2, draft, -1, 0], 2)):      # descending: no rows
        out, lse, flags = run(cu, draft)
        check(out, lse, first, draft, flags)
    for cu in ([draft, -2], [10 ** 6, 10 ** 6], [-5, -1], [-2 ** 31, -2 ** 31 + 1]):
        out, lse, flags = run(cu, draft)
        assert (out == 3).all() and (lse == 7).all() and flags == D.CACHE_BAD_ARG, cu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,draft", SHAPES)
def test_maxima_that_grow_from_tile_to_tile(gpu, group, draft, dtype):
    """Every tile of 64 keys raises a row's maximum by more than 2^8, the last one
    (drafted keys) too, in runs of many tiles: outputs are rescaled before each."""
    ctx, n = 500, 70
    c = Drafted(gpu, [ctx] * n, [draft] * n, group=group, kv_heads=4, dtype=dtype, page=64, seed=draft)
    c.q.mul_(0.05).add_(1.0)
    pos = torch.arange(ctx + draft, device=gpu)
    # a mean of pos / 100 over 128 elements: scores of 0.11 a key, 10 log2 units a tile
    for s in range(n):
        pages = c.cache.page_table[s].long()[pos // 64]
        for h in range(4):
            c.cache.k[0][pages, h, pos % 64] += (pos / 100.0)[:, None].to(dtype)
    c.check(*c.run())
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("group,draft", SHAPES)
def test_outputs_in_the_place_of_the_queries(gpu, group, draft, odd):
    for lens in ([3000, 61], [200] * 60):
        c = Drafted(gpu, lens, [draft] * len(lens), group=group, tree="random", seed=draft)
        if odd:                             # a visible infinity in v of some drafted tokens
            p, o = int(c.cache.page_table[1, lens[1] // 16]), lens[1] % 16
            c.cache.v[0, p, :, o, ::3] = float("inf")
        want, wlse = c.run()
        c.check(want, wlse)
        got, lse = c.run(out=c.q)
        torch.cuda.synchronize()
        same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
        assert got.data_ptr() == c.q.data_ptr() and same(got.contiguous(), want) and torch.equal(lse, wlse)
