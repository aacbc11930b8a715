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


def guarded(gpu, shape, dtype, fill):
    """A tensor of `shape` inside a larger one, and the check that nothing around it
    was written."""
    n, pad = torch.Size(shape).numel(), 4096
    wide = torch.full((n + 2 * pad,), fill, dtype=dtype, device=gpu)
    # (the state's tensors start on 16 bytes, as pad elements of any type do)
    return wide[pad:pad + n].view(shape), lambda: bool((wide[:pad] == fill).all() & (wide[pad + n:] == fill).all())


def test_state_out_of_range_moves_only_what_is_in_range(gpu):
    """Page ids, lengths and counts out of range: every element of k and v outside the
    rows that can be moved stays as it was, bit for bit, and so does what lies around
    the cache's tensors."""
    pages, seqs, cols, ps = 40, 8, 12, 16
    made = [guarded(gpu, (2, pages, 2, ps, 64), torch.bfloat16, 5.0) for _ in range(2)]
    made += [guarded(gpu, s, torch.int32, -77) for s in
             ((seqs, cols), (seqs,), (seqs,), (pages,), (pages,), (1,))]
    c = D.PagedCache.from_tensors(*(t for t, _ in made))
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, device=gpu).bfloat16())
    c.page_table.zero_()
    c.length.zero_()
    c.held.zero_()
    c.ref_count.zero_()
    c.free_list.copy_(torch.arange(pages - 1, -1, -1, device=gpu))
    c.n_free.fill_(pages)
    D.cache_reserve(c, ints([0, 1], gpu), ints([40, 40], gpu))          # pages 0 1 2 and 3 4 5
    c.length.copy_(ints([40, 40, -3, 10 ** 9, 0, 0, 0, 0], gpu))
    c.page_table[0, 1] = 10 ** 6
    c.page_table[1, 2] = -5
    c.held[3] = 10 ** 8
    assert D.cache_status(c) == (P.PROX_OK, 0)

    def same(want):
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip((c.k, c.v), want)) and all(ok() for _, ok in made)

    want = [c.k.clone(), c.v.clone()]
    D.cache_fork(c, ints([0, 1, 2], gpu), ints([4, 5, 6], gpu), share=False)
    for t in want:      # 4 takes pages 6 7 8, 5 takes 9 10 11; a page without a source stays
        for to, at, rows in ((6, 0, 16), (8, 2, 8), (9, 3, 16), (10, 4, 16)):
            t[:, to, :, :rows] = t[:, at, :, :rows]
    assert same(want) and D.cache_status(c) == (D.PROX_EDATA, D.CACHE_BAD_STATE)
    assert c.page_table[4:7, :3].tolist() == [[6, 7, 8], [9, 10, 11], [0, 0, 0]]
    assert c.length.tolist() == [40, 40, -3, 10 ** 9, 40, 40, 0, 0] and int(c.n_free) == 28
    # 2 counts as empty, 3 as full to its last column
    ok = torch.full((2,), 7, dtype=torch.uint8, device=gpu)
    D.cache_reserve(c, ints([3, 2], gpu), ints([4, 4], gpu), ok)
    assert same(want) and ok.tolist() == [0, 1] and int(c.page_table[2, 0]) == 12
    assert D.cache_status(c)[1] & D.CACHE_BAD_STATE
    # rows 42 and 45 of 0 to 40 and 41; 3 has no room behind its length
    D.cache_compact(c, ints([0, 3], gpu), ints([[2, 5], [0, 1]], gpu), ints([2, 2], gpu), ok)
    for t in want:
        t[:, 2, :, 8] = t[:, 2, :, 10].clone()
        t[:, 2, :, 9] = t[:, 2, :, 13].clone()
    assert same(want) and ok.tolist() == [1, 0] and c.length.tolist()[:4] == [42, 40, -3, 10 ** 9]
    assert D.cache_status(c)[1] == D.CACHE_BAD_STATE | D.CACHE_BAD_ARG
    # a row on a page out of range, and one behind the held pages, are left out
    k = torch.randn((10, 2, 64), device=gpu).bfloat16()
    c.length[1] = 31
    D.cache_append(c, 1, ints([1, 3, 0], gpu), ints([0, 2, 3, 10], gpu), k, -k)
    for t, new in zip(want, (k, -k)):
        t[1, 4, :, 15] = new[0]                     # 1: position 31; 32 lies on page -5
        for j in range(6):                          # 0: positions 42 .. 47; 48 has no page
            t[1, 2, :, 10 + j] = new[3 + j]
    assert same(want)
    assert D.cache_status(c)[1] == D.CACHE_BAD_STATE | D.CACHE_FULL
    D.cache_free(c, ints([0, 1, 2, 3], gpu))
    assert same(want) and D.cache_status(c)[1] & D.CACHE_BAD_STATE
    free = c.free_list[:int(c.n_free)].tolist()
    assert len(set(free)) == len(free) and all(0 <= p < pages for p in free)
    assert all(int(c.ref_count[p]) == 0 for p in free) and int(c.ref_count.min()) == 0
    assert c.length.tolist() == [0, 0, 0, 0, 40, 40, 0, 0] and c.held.tolist()[:4] == [0] * 4
    # a free count and a free list out of range
    D.cache_free(c, ints([4, 5], gpu))
    c.n_free.fill_(10 ** 6)
    c.free_list[-1] = 10 ** 6
    D.cache_reserve(c, ints([7], gpu), ints([20], gpu))
    assert same(want) and D.cache_status(c)[1] & D.CACHE_BAD_STATE
    assert 0 <= int(c.n_free) <= pages
