"""Attention of drafted tokens over the paged cache against the formula in 64
bits. Rows of pages that no sequence has written hold NaN throughout."""
import math
import random

import pytest
import torch

from decode_helpers import Drafted, ints, tree_words
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_types_dims_pages(gpu, dim, dtype, page):
    for tree in (None, "random"):
        c = Drafted(gpu, [130, 0, 7, 64, 500], [3, 5, 1, 4, 2], dim=dim, dtype=dtype, page=page, tree=tree,
                    order=[3, 0, 4, 1, 2], seed=page)
        c.check(*c.run())
        assert D.cache_status(c.cache) == (P.PROX_OK, 0)


# rows of a key/value head around the sizes of the row tiles
@pytest.mark.parametrize("group,draft", [(1, 1), (1, 16), (1, 17), (5, 3), (4, 8), (3, 11), (8, 8), (7, 10),
                                         (8, 17), (1, 256), (16, 9), (64, 2), (4, 64), (8, 33)])
def test_rows_of_a_head(gpu, group, draft):
    c = Drafted(gpu, [90, 700], [draft, max(1, draft - 1)], group=group, tree="random", kv_heads=2, page=32)
    c.check(*c.run())


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 62, 63, 64, 65, 127, 128, 129, 255, 1000, 2049])
def test_lengths_around_tiles_and_pages(gpu, ctx):
    for page in (16, 64, 128):
        c = Drafted(gpu, [ctx], [2], page=page, seed=ctx)
        c.check(*c.run())


def test_one_token_of_many_sequences(gpu):
    rng = random.Random(2)
    n = 300                                     # more than one launch takes
    c = Drafted(gpu, [rng.randint(0, 200) for _ in range(n)], [1] * n, kv_heads=1, group=2, dim=64)
    c.check(*c.run())


def test_sequences_without_rows(gpu):
    c = Drafted(gpu, [100, 50, 0, 30], [2, 0, 0, 3], tree="random")
    c.check(*c.run())


def test_long_cache_cut_over_many_blocks(gpu):
    for draft in (1, 9, 40):
        c = Drafted(gpu, [20011], [draft], kv_heads=1, group=2, page=64, tree="random")
        c.check(*c.run())


def test_few_and_many_pieces_give_the_same(gpu):
    """A sequence alone (cut over the whole GPU) and among others (hardly cut)."""
    one = Drafted(gpu, [3001], [4], seed=5, page=16)
    out1, lse1 = one.run()
    many = Drafted(gpu, [3001] + [900] * 40, [4] * 41, seed=5, page=16)
    many.check(*many.run())
    one.check(out1, lse1)


def test_masks_that_leave_rows_empty(gpu):
    def tree(s, t, words):
        return tree_words([0 if i % 2 else 1 << i for i in range(t)], words)
    c = Drafted(gpu, [0, 0, 33], [6, 1, 4], tree=tree)
    out, lse = c.run()
    c.check(out, lse)
    assert (lse == -math.inf).any()


def test_bits_behind_the_drafts_are_ignored(gpu):
    def tree(s, t, words):
        return [[-1] * words for _ in range(t)]
    c = Drafted(gpu, [10, 70], [5, 3], tree=tree, max_q=200, words=5)
    c.check(*c.run())


def test_wide_trees_over_words_and_tiles(gpu):
    for ctx in (0, 1, 40, 63, 64, 100):
        c = Drafted(gpu, [ctx], [150], tree="random", group=1, kv_heads=1, seed=ctx)
        c.check(*c.run())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("draft,group", [(6, 2), (12, 4), (40, 4)])
def test_masked_drafts_with_odd_values(gpu, value, draft, group):
    """NaN and infinities of a drafted token reach only the rows that see it."""
    c = Drafted(gpu, [61], [draft], tree="random", group=group, seed=draft)
    sees = c.seen(0, 0)[:, 61:]
    sick = [j for j in range(draft) if int(sees[:, j].sum()) < draft][:3]
    for j in sick:
        p, o = int(c.cache.page_table[0, (61 + j) // 16]), (61 + j) % 16
        c.cache.v[0, p, :, o, 3::7] = value
    c.check(*c.run())
    # keys too: rows that do not see the last of them stay finite
    for j in sick:
        p, o = int(c.cache.page_table[0, (61 + j) // 16]), (61 + j) % 16
        c.cache.v[0, p, :, o] = 1.0
    sick = sick[-1:]
    for j in sick:
        p, o = int(c.cache.page_table[0, (61 + j) // 16]), (61 + j) % 16
        c.cache.k[0, p, :, o] = value
    out, lse = c.run()
    clean = ~sees[:, sick].any(1)
    assert clean.any() and torch.isfinite(out[clean]).all() and torch.isfinite(lse[clean]).all()
    if math.isnan(value):
        assert torch.isnan(out[~clean]).all()


def test_large_scores_and_lowest_values(gpu):
    for dtype in (torch.bfloat16, torch.float16):
        c = Drafted(gpu, [200], [3], dtype=dtype, seed=9)
        c.q.mul_(30)
        c.check(*c.run())
        c.scale = 1e-4
        c.check(*c.run())


def test_other_layers_strides_and_outputs(gpu):
    c = Drafted(gpu, [77, 130], [3, 9], layers=3, layer=2, tree="random", extra_rows=4)
    heads = c.q.shape[1]
    wide = torch.full((c.q.shape[0], heads + 3, 128), 5.0, dtype=c.q.dtype, device=gpu)
    lse = torch.full((c.q.shape[0], heads), 7.0, device=gpu)
    out, _ = c.run(out=wide[:, :heads], lse=lse)
    c.check(out, lse)
    # rows behind the last sequence, and the gaps between rows, stay
    assert (wide[12:] == 5).all() and (wide[:, heads:] == 5).all() and (lse[12:] == 7).all()


def test_padding_and_bad_entries(gpu):
    c = Drafted(gpu, [40, 40, 40], [2, 2, 2], seqs=[0, -1, 2])
    out, lse = c.run()
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)
    assert (out[2:4] == 0).all() and (lse[2:4] == -math.inf).all()
    c.seqs = ints([0, 99, 2], gpu)
    again, _ = c.run()
    assert D.cache_status(c.cache)[1] == D.CACHE_BAD_SEQ
    assert torch.equal(out, again)


def test_a_sequence_listed_twice(gpu):
    c = Drafted(gpu, [50, 3], [4, 4], seqs=[0, 0])
    c.q[4:].copy_(c.q[:4])
    out, lse = c.run()
    assert torch.equal(out[:4], out[4:]) and torch.equal(lse[:4], lse[4:])


def test_bad_state_is_reported_and_left_out(gpu):
    # a page id out of range: its keys are not seen
    for page, bad in ((16, 10**6), (64, -7)):
        c = Drafted(gpu, [300], [2], page=page)
        want = Drafted(gpu, [300], [2], page=page)
        j = 128 // page
        c.cache.page_table[0, j] = bad
        out, lse = c.run()
        assert D.cache_status(c.cache)[1] == D.CACHE_BAD_STATE
        k, v = want.rows_of(0)
        keep = torch.ones(302, dtype=torch.bool, device=gpu)
        keep[j * page:(j + 1) * page] = False
        for t in range(2):
            keep_t = keep & (torch.arange(302, device=gpu) <= 300 + t)
            x = torch.einsum("hd,hkd->hk", c.q[t].double(), k.repeat_interleave(4, 0)) * c.scale
            o = torch.softmax(x.masked_fill(~keep_t, -math.inf), 1)[:, None] @ v.repeat_interleave(4, 0)
            # rounding of probabilities and result: at most 2^-8 each, of |v| <= 6
            assert (out[t].double() - o[:, 0]).abs().max() < 2 * 6 * 2.0 ** -8
    # fewer pages held than the length and the drafts need
    c = Drafted(gpu, [30], [4])
    c.cache.held.fill_(2)
    c.run()
    assert D.cache_status(c.cache)[1] == D.CACHE_FULL
    c.cache.length.fill_(10**9)
    c.run()
    assert D.cache_status(c.cache)[1] & D.CACHE_BAD_STATE
    # offsets out of range: rows are cut, nothing behind them is touched
    c = Drafted(gpu, [30], [4])
    c.cu = ints([0, 10**6], gpu)
    out = torch.full_like(c.q, 3).contiguous()
    c.run(out=out)
    assert D.cache_status(c.cache)[1] & D.CACHE_BAD_ARG
    c.cu = ints([5, -2], gpu)
    c.run()
    assert D.cache_status(c.cache)[1] & D.CACHE_BAD_ARG


def test_offsets_past_32_bits(gpu):
    pages, kv, page, dim = 42000, 8, 64, 128
    cache = D.PagedCache(1, pages, kv, page, dim, 1, 8, torch.bfloat16, gpu)
    cache.k.zero_()
    cache.v.zero_()
    small = Drafted(gpu, [200], [3], kv_heads=kv, page=page, spare=0)
    ids = torch.tensor([41999, 5, 41990, 33333], device=gpu)
    cache.page_table[0, :4] = ids.int()
    for a, b in ((cache.k, small.cache.k), (cache.v, small.cache.v)):
        a[0, ids] = b[0, small.cache.page_table[0, :4].long()]
    cache.length.fill_(200)
    cache.held.fill_(4)
    out, lse = D.tree_attention(cache, 0, small.q, small.seqs, small.cu, 3)
    want, wlse = small.run()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_repeated_calls_give_the_same_bits(gpu):
    c = Drafted(gpu, [5000, 10, 900], [7, 1, 12], tree="random", page=64)
    first = c.run()
    for _ in range(5):
        out, lse = c.run()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_captured_pass_follows_lengths_and_tables(gpu):
    a = Drafted(gpu, [700, 220], [4, 4], tree="random", seed=1)
    b = Drafted(gpu, [300, 500], [4, 4], tree="random", seed=2)
    ws = D.attention_workspace(a.cache, 4, 8)
    out, lse = a.run(ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(out=out, lse=lse, ws=ws)
    out.zero_()
    g.replay()
    a.check(out, lse)
    # the second state's lengths, tables and rows under the same pointers
    want = b.run()
    pages, cols = b.cache.n_pages, b.cache.max_pages
    assert pages <= a.cache.n_pages and cols <= a.cache.max_pages
    a.cache.k[:, :pages] = b.cache.k
    a.cache.v[:, :pages] = b.cache.v
    a.cache.page_table[:, :cols] = b.cache.page_table
    a.cache.length.copy_(b.cache.length)
    a.cache.held.copy_(b.cache.held)
    a.q.copy_(b.q)
    a.tree.copy_(b.tree)
    g.replay()
    b.check(out, lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_two_streams_with_a_workspace_each(gpu):
    cs = [Drafted(gpu, [4000, 100], [5, 3], seed=s, page=32) for s in (1, 2)]
    want = [c.run() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [D.attention_workspace(c.cache, 5, 8) for c in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, s, ws in zip(cs, streams, wss):
            with torch.cuda.stream(s):
                got.append(c.run(ws=ws))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


# rows of a head for the kernels of 16 and 32 rows, of 128 and of 256 rows
@pytest.mark.parametrize("group,draft,position", [(4, 4, 0), (4, 4, 1), (2, 12, 2), (4, 20, 0), (4, 20, 1),
                                                  (4, 20, 4), (8, 40, 0), (8, 40, 3), (8, 40, 6)])
def test_a_load_that_never_comes_is_reported(gpu, group, draft, position):
    """The waits run out, the call ends with an error, and the next one is right."""
    c = Drafted(gpu, [30000, 600], [draft, draft], group=group, page=32, tree="random")
    P.test_set_wait(20000)
    P.test_set_skip(P.SKIP_ATTENTION, position)
    try:
        c.run()
    finally:
        P.test_set_skip(P.SKIP_OFF)
        P.test_set_wait(0)
    assert D.cache_status(c.cache) == (P.PROX_ETIMEOUT, D.CACHE_TIMEOUT)
    c.check(*c.run())
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)


# the tensor-memory kernel: one and two groups of 128 rows, a last tile of few rows
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group,draft", [(5, 8), (5, 28), (8, 37)])
def test_many_rows_of_types_dims_pages(gpu, dim, dtype, page, group, draft):
    c = Drafted(gpu, [130, 0, 7, 700], [draft, draft - 1, 1, draft // 2], dim=dim, dtype=dtype, page=page,
                group=group, tree="random", order=[3, 0, 1, 2], seed=page)
    c.check(*c.run())
    assert D.cache_status(c.cache) == (P.PROX_OK, 0)


@pytest.mark.parametrize("group,draft", [(4, 24), (4, 64), (8, 40)])
def test_runs_over_many_long_units(gpu, group, draft):
    """A block's run holds the end of one unit, whole ones, and the start of another."""
    for lens in ([9001] * 3, [4100, 9, 12000, 64, 700, 2500]):
        c = Drafted(gpu, lens, [draft] * len(lens), group=group, kv_heads=8, page=64, tree="random", seed=draft)
        c.check(*c.run())


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_another_device_than_the_current_one():
    c = Drafted(torch.device("cuda:1"), [200], [3])
    c.check(*c.run())


def test_binding_refuses_wrong_tensors(gpu):
    c = Drafted(gpu, [20], [2], tree="random")
    call = lambda **kw: D.tree_attention(c.cache, **({"layer": 0, "q": c.q, "seqs": c.seqs, "cu_q": c.cu,  # noqa: E731
                                                      "max_q": 2, "tree": c.tree} | kw))
    for bad in (dict(q=c.q.half()), dict(q=c.q[..., :64]), dict(q=c.q[0]), dict(q=c.q.cpu()),
                dict(q=c.q.transpose(0, 1)), dict(seqs=c.seqs.long()), dict(cu_q=c.cu[:1]),
                dict(tree=c.tree.int()), dict(tree=c.tree[:1]), dict(out=torch.empty(1, device=gpu)),
                dict(lse=torch.empty((2, 8), device=gpu, dtype=torch.float16))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(layer=1), dict(q=c.q[:, :7]), dict(max_q=0), dict(max_q=300), dict(scale=0.0),
                dict(ws=torch.empty(64, dtype=torch.uint8, device=gpu))):
        with pytest.raises(P.ProxError):
            call(**bad)
