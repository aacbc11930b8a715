"""Page operations on lists they have to refuse in part, on state that is out of
range, and the status word under calls on two streams."""
import random

import pytest
import torch

from decode_helpers import Drafted, ints
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

pytestmark = pytest.mark.gpu


def test_status_bits_set_while_the_word_is_read_are_kept(gpu):
    """An attention call on another stream sets a bit at some time while the word
    is read again and again: one of the reads must return it."""
    c = Drafted(gpu, [3], [1])
    c.seqs.fill_(99)
    ws = D.attention_workspace(c.cache, 1, 8)
    out, lse = c.run(ws=ws)
    assert D.cache_status(c.cache)[1] == D.CACHE_BAD_SEQ
    side, rng, lost = torch.cuda.Stream(), random.Random(1), 0
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(400):
        done = torch.cuda.Event()
        with torch.cuda.stream(side):
            torch.cuda._sleep(rng.randrange(1000, 200000))
            c.run(out=out, lse=lse, ws=ws)
            done.record()
        bits = 0
        while not done.query():
            bits |= D.cache_status(c.cache)[1]
        done.synchronize()
        bits |= D.cache_status(c.cache)[1]
        lost += bits != D.CACHE_BAD_SEQ
    assert lost == 0


def test_status_returns_and_clears_what_was_set(gpu):
    c = Drafted(gpu, [3], [1])
    for bits, st in ((0, P.PROX_OK), (D.CACHE_FULL | D.CACHE_BAD_ARG, D.PROX_EDATA),
                     (D.CACHE_TIMEOUT | D.CACHE_BAD_SEQ, P.PROX_ETIMEOUT)):
        c.cache.status.fill_(bits)
        assert D.cache_status(c.cache) == (st, bits)
        assert int(c.cache.status) == 0 and D.cache_status(c.cache) == (P.PROX_OK, 0)


def test_paths_over_unreadable_pages_are_refused(gpu):
    c = D.PagedCache(2, 20, 2, 16, 64, 4, 4, torch.bfloat16, gpu)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, device=gpu).bfloat16())
    D.cache_reserve(c, ints([0, 1, 2, 3], gpu), ints([48] * 4, gpu))
    c.length.copy_(ints([30, 30, 30, 30], gpu))
    c.page_table[0, 2] = 20                 # rows 32 .. 47 of these
    c.page_table[1, 2] = -1
    c.page_table[3, 2] = 10 ** 9
    k, v = c.k.clone(), c.v.clone()
    ok = torch.full((4,), 7, dtype=torch.uint8, device=gpu)
    # read from such a page; written to one; neither; not touched by the path
    path = ints([[2, 0, 0], [0, 1, 3], [1, 4, 9], [1, 0, 0]], gpu)
    D.cache_compact(c, ints([0, 1, 2, 3], gpu), path, ints([1, 3, 3, 1], gpu), ok)
    torch.cuda.synchronize()
    assert ok.tolist() == [0, 0, 1, 1] and c.length.tolist() == [30, 30, 33, 31]
    assert D.cache_status(c) == (D.PROX_EDATA, D.CACHE_BAD_STATE)
    for new, old in ((c.k, k), (c.v, v)):
        def row(s, pos):
            return int(c.page_table[s, pos // 16]), pos % 16
        for s, pairs in ((2, ((30, 31), (31, 34), (32, 39))), (3, ((30, 31),))):
            for to, at in pairs:
                (p, o), (q, r) = row(s, to), row(s, at)
                assert torch.equal(new[:, p, :, o], old[:, q, :, r])
                old[:, p, :, o] = old[:, q, :, r].clone() if (s, to) != (2, 31) else new[:, p, :, o]
        assert torch.equal(new, old)        # and nothing else moved


def test_reserve_refuses_too_many_columns_alone_and_too_few_pages_in_order(gpu):
    """ok[] by hand: an entry that needs more columns than the table has is refused
    alone; one that finds too few free pages, and those behind it that need any."""
    c = D.PagedCache(1, 6, 1, 16, 64, 8, 3, torch.bfloat16, gpu)

    def reserve(seqs, n_new):
        ok = torch.full((len(seqs),), 7, dtype=torch.uint8, device=gpu)
        D.cache_reserve(c, ints(seqs, gpu), ints(n_new, gpu), ok)
        torch.cuda.synchronize()
        return ok.tolist(), c.held[seqs].tolist(), D.cache_status(c)[1]

    assert reserve([0, 1, 2], [49, 1, 0]) == ([0, 1, 1], [0, 1, 0], D.CACHE_FULL)
    assert reserve([3, 4, 5, 6, 7], [48, 33, 1, 0, 16]) == ([1, 0, 0, 1, 0], [3, 0, 0, 0, 0], D.CACHE_FULL)
    # both in one call: the one that is too wide takes no page from the others' count
    assert reserve([4, 5, 6], [1000, 32, 1]) == ([0, 1, 0], [0, 2, 0], D.CACHE_FULL)
    assert int(c.n_free) == 0
