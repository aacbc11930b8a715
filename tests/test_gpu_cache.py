"""Page operations of the paged cache against a plain model, state and rows
exactly: every list, every count, and every element of k and v."""
import random

import pytest
import torch

from decode_helpers import CacheModel, ints
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

pytestmark = pytest.mark.gpu


def make(dev, *, layers=2, pages=40, kv_heads=2, page=16, dim=64, seqs=8, cols=12, dtype=torch.bfloat16):
    c = D.PagedCache(layers, pages, kv_heads, page, dim, seqs, cols, dtype, dev)
    gen = torch.Generator(device=dev)
    gen.manual_seed(pages)
    for t in (c.k, c.v):   # any bits: rows are moved, not computed with
        t.view(torch.int16).copy_(torch.randint(-2**15, 2**15, t.shape, device=dev, generator=gen))
    return c, CacheModel(c)


class Both:
    """Runs each call on the cache and on the model."""

    def __init__(self, c, m, seed=0):
        self.c, self.m, self.dev = c, m, c.device
        self.gen = torch.Generator(device=c.device)
        self.gen.manual_seed(seed)

    def _ok(self, n):
        return torch.full((n,), 7, dtype=torch.uint8, device=self.dev)

    def reserve(self, seqs, n_new):
        ok = self._ok(len(seqs))
        D.cache_reserve(self.c, ints(seqs, self.dev), ints(n_new, self.dev), ok)
        assert self.m.reserve(seqs, n_new) == ok.tolist()

    def append(self, seqs, counts, extra=0, wide=0):
        cu = [0]
        for t in counts:
            cu.append(cu[-1] + t)
        shape = (cu[-1] + extra, self.c.n_kv_heads + wide, self.c.head_dim)
        for layer in range(self.c.n_layers):
            k, v = (torch.randn(shape, device=self.dev, generator=self.gen).to(self.c.dtype)
                    [:, :self.c.n_kv_heads] for _ in range(2))
            D.cache_append(self.c, layer, ints(seqs, self.dev), ints(cu, self.dev), k, v)
            self.m.append(layer, seqs, cu, k, v)

    def fork(self, src, dst, share=True):
        ok = self._ok(len(src))
        D.cache_fork(self.c, ints(src, self.dev), ints(dst, self.dev), share=share, ok=ok)
        assert self.m.fork(src, dst, share) == ok.tolist()

    def compact(self, seqs, path, n_path):
        ok = self._ok(len(seqs))
        D.cache_compact(self.c, ints(seqs, self.dev), ints(path, self.dev), ints(n_path, self.dev), ok)
        assert self.m.compact(seqs, path, n_path) == ok.tolist()

    def free(self, seqs):
        D.cache_free(self.c, ints(seqs, self.dev))
        self.m.free(seqs)

    def grow(self, s, n):
        """n committed tokens more."""
        self.reserve([s], [n])
        self.append([s], [n])
        while n:
            k = min(n, 256)
            self.compact([s], [list(range(k))], [k])
            n -= k

    def check(self):
        self.m.check(self.c)


@pytest.mark.parametrize("page,dim,kv,dtype", [(16, 64, 1, torch.bfloat16), (32, 128, 3, torch.float16),
                                               (64, 64, 8, torch.bfloat16), (128, 128, 2, torch.bfloat16)])
def test_a_life_of_sequences(gpu, page, dim, kv, dtype):
    b = Both(*make(gpu, page=page, dim=dim, kv_heads=kv, dtype=dtype, layers=3))
    b.check()
    b.grow(0, page * 3 + 5)
    b.grow(1, 1)
    b.grow(2, page * 2)
    b.check()
    b.fork([0, 0, 2, 1], [5, 3, 4, 6])             # shared, one with no part page
    b.check()
    b.fork([0], [7], share=False)                   # own pages
    b.check()
    b.reserve([5, 3, 7], [9, page + 1, 2])
    b.append([5, 3, 7], [9, page + 1, 2], extra=3, wide=4)
    b.check()
    b.compact([5, 3, 7], [[0, 2, 5, 8], [1, 2, page, 0], [1, 0, 0, 0]], [4, 3, 1])
    b.check()
    b.free([0, 3])
    b.check()
    b.free([5, 4, 2, 1, 6, 7])
    b.check()
    assert b.m.n_free == [b.m.n_pages]


@pytest.mark.parametrize("seed", range(6))
def test_random_calls_with_bad_entries(gpu, seed):
    rng = random.Random(seed)
    page = rng.choice((16, 32, 64))
    b = Both(*make(gpu, page=page, dim=rng.choice((64, 128)), pages=30, cols=9, kv_heads=rng.choice((1, 2, 5))), seed)
    pick = lambda n: [rng.choice((-1, 8, 8000, -7)) if rng.random() < 0.1 else rng.randrange(8)  # noqa: E731
                      for _ in range(n)]
    for step in range(40):
        n = rng.randint(1, 6)
        what = rng.choice(("reserve", "append", "fork", "fork", "compact", "compact", "free"))
        if what == "reserve":
            b.reserve(pick(n), [rng.choice((-1, 0, 1, page, 3 * page, 12 * page, rng.randint(0, 60)))
                                for _ in range(n)])
        elif what == "append":
            s = pick(n)
            b.append(s, [rng.choice((0, 1, 5, page)) for _ in s])
        elif what == "fork":
            b.fork(pick(n), pick(n), rng.random() < 0.6)
        elif what == "compact":
            m = rng.randint(1, 20)
            rows = [sorted(rng.sample(range(m + 8), m)) if rng.random() < 0.9 else [3] * m for _ in range(n)]
            b.compact(pick(n), rows, [rng.choice((m, 0, 1, m + 1 if rng.random() < 0.2 else m, -1 if
                                                  rng.random() < 0.1 else m // 2)) for _ in range(n)])
        else:
            b.free(pick(rng.randint(1, 2)))
        b.check()


def test_out_of_pages_entries_in_order(gpu):
    b = Both(*make(gpu, pages=10, seqs=8, cols=12))
    b.reserve([0, 1, 2, 3], [16 * 4, 16 * 7, 16, 0])       # 4 fit, 7 do not, nor what follows and needs any
    b.check()
    b.reserve([4], [16 * 6])
    b.reserve([5], [1])
    b.check()
    b.free([0])
    b.fork([4, 4], [6, 7], share=False)                    # nothing committed: both fit, empty
    b.check()
    b.reserve([6], [16 * 13])                              # more columns than the table has
    b.check()


def test_fork_refuses_targets_that_hold_tokens(gpu):
    b = Both(*make(gpu))
    b.grow(0, 40)
    b.grow(1, 3)
    b.fork([0, 0, 0], [1, 2, 2])
    b.check()
    b.fork([0, 1], [0, 3])
    b.check()
    b.fork([2, 4, 5], [4, 5, 6])                           # sources as they are before the call: 4 and 5 are empty
    b.check()


def test_refused_paths_leave_the_sequence(gpu):
    b = Both(*make(gpu))
    b.grow(0, 20)
    b.grow(1, 20)
    b.reserve([0, 1], [12, 12])
    for path, m in (([0, 0, 1], 3), ([2, 1, 3], 3), ([0, 1, 12], 3), ([-1, 0, 1], 3), ([0, 1, 2], 4),
                    ([0, 1, 2], -1)):
        b.compact([0], [path], [m])
        b.check()
    b.compact([0, 0, -1, 1], [[0, 3, 11]] * 4, [3, 3, 3, 0])
    b.check()


def test_long_paths_move_overlapping_rows(gpu):
    b = Both(*make(gpu, layers=2, pages=60, cols=40, page=16, dim=128))
    b.grow(0, 7)
    rng = random.Random(3)
    b.reserve([0], [300])
    b.append([0], [256])
    path = sorted(rng.sample(range(256), 200))
    b.compact([0], [path], [200])
    b.check()


def test_many_sequences_and_pages(gpu):
    """Thousands of entries and more listings than the cluster has lanes."""
    b = Both(*make(gpu, layers=1, pages=9000, kv_heads=1, seqs=4096, cols=700, page=16, dim=64))
    rng = random.Random(1)
    b.reserve(list(range(0, 3000)), [rng.randint(0, 30) for _ in range(3000)])
    b.check()
    for s, n in ((3500, 10000), (3501, 4096), (3502, 15)):
        b.reserve([s], [n])
        b.c.length[s] = n
        b.m.length[s] = n
    b.fork([3500] * 20 + [3501] * 20 + [3502], list(range(3600, 3641)))
    b.check()
    b.free([3600 + i for i in range(0, 41, 2)] + [3500, 3502])
    b.check()
    b.free(list(range(0, 3000)) + [3601 + i for i in range(0, 40, 2)] + [3501])
    b.check()
    assert b.m.n_free == [9000]


@pytest.mark.parametrize("n", [33, 255, 257, 700, 1024, 1025])
def test_entries_around_the_sizes_of_a_call(gpu, n):
    """Every call with n entries, some padding and some without tokens."""
    b = Both(*make(gpu, layers=1, pages=6 * n, kv_heads=1, seqs=2 * n + 2, cols=3, page=16, dim=64))
    rng = random.Random(n)
    seqs = list(range(n))
    rng.shuffle(seqs)
    for i in rng.sample(range(n), 3):
        seqs[i] = -1
    counts = [rng.randint(0, 5) for _ in seqs]
    b.reserve(seqs, counts)
    b.append(seqs, counts, extra=2)
    b.check()
    b.compact(seqs, [[0, 2, 4]] * n, [min(1, c) if c < 5 else 3 for c in counts])
    b.check()
    dst = [n + i for i in range(n)]
    b.fork(seqs, dst, share=False)
    b.check()
    b.free(dst)
    b.fork(seqs, dst)
    b.check()
    b.free(seqs)
    b.check()
    b.free(dst)
    b.check()
    assert b.m.n_free == [6 * n]


def test_freeing_more_listings_than_a_block_keeps(gpu):
    """4000 forks of a sequence of 2048 pages, a quarter with a page of their own."""
    n, cols, pages = 4000, 2050, 4000
    c = D.PagedCache(1, pages, 1, 16, 64, n + 1, cols, torch.bfloat16, gpu)
    D.cache_reserve(c, ints([n], gpu), ints([2048 * 16], gpu))
    c.length[n] = 2048 * 16
    seqs = torch.arange(n, dtype=torch.int32, device=gpu)
    D.cache_fork(c, torch.full_like(seqs, n), seqs)
    some = seqs[::4].contiguous()
    D.cache_reserve(c, some, torch.ones_like(some))
    torch.cuda.synchronize()
    assert D.cache_status(c) == (P.PROX_OK, 0)
    table, held = c.page_table.cpu(), c.held.cpu()
    assert held.tolist() == [2048 + (s % 4 == 0) for s in range(n)] + [2048]
    assert int(c.ref_count.max()) == n + 1
    left = int(c.n_free)
    assert left == pages - 2048 - 1000
    order = torch.cat([seqs.flip(0).cpu(), torch.tensor([n], dtype=torch.int32)])
    listed = torch.cat([table[s, :held[s]] for s in order.tolist()]).tolist()
    want = c.free_list[:left].tolist() + list(dict.fromkeys(listed))
    D.cache_free(c, order.to(gpu))
    torch.cuda.synchronize()
    assert D.cache_status(c) == (P.PROX_OK, 0)
    assert int(c.n_free) == pages and c.free_list.tolist() == want
    assert int(c.ref_count.abs().max()) == 0 and int(c.held.max()) == 0 and int(c.length.max()) == 0


def test_corrupt_state_is_reported_and_stays_in_bounds(gpu):
    c, _ = make(gpu)
    D.cache_reserve(c, ints([0, 1], gpu), ints([40, 40], gpu))
    c.length.copy_(ints([40, 40, -3, 10**9, 0, 0, 0, 0], gpu))
    c.page_table[0, 1] = 10**6
    c.page_table[1, 2] = -5
    c.held[3] = 10**8
    before = c.k.clone()
    D.cache_fork(c, ints([0, 1, 2], gpu), ints([4, 5, 6], gpu), share=False)
    st, bits = D.cache_status(c)
    assert st == D.PROX_EDATA and bits & D.CACHE_BAD_STATE
    D.cache_reserve(c, ints([3, 2], gpu), ints([4, 4], gpu))
    D.cache_compact(c, ints([0, 3], gpu), ints([[0, 1], [0, 1]], gpu), ints([2, 2], gpu))
    D.cache_free(c, ints([0, 1, 2, 3], gpu))
    torch.cuda.synchronize()
    assert D.cache_status(c)[1] & D.CACHE_BAD_STATE
    assert c.k.shape == before.shape and 0 <= int(c.n_free) <= c.n_pages
    assert D.cache_status(c) == (P.PROX_OK, 0)


def test_a_page_listed_by_two_sequences_too_often_is_not_freed_twice(gpu):
    c, _ = make(gpu)
    D.cache_reserve(c, ints([0, 1], gpu), ints([16, 16], gpu))
    c.page_table[1, 0] = c.page_table[0, 0]     # a count of 1 listed twice
    D.cache_free(c, ints([0, 1], gpu))
    st, bits = D.cache_status(c)
    assert bits & D.CACHE_BAD_STATE
    free = c.free_list[:int(c.n_free)].tolist()
    assert len(set(free)) == len(free) and int(c.ref_count.min()) >= 0


def test_offsets_past_32_bits(gpu):
    # 2.7e9 elements in each pool; the sequences live at both ends of it
    pages, kv, page, dim = 42000, 8, 64, 128
    c = D.PagedCache(1, pages, kv, page, dim, 4, 8, torch.bfloat16, gpu)
    c.k.zero_()
    c.v.zero_()
    c.free_list.copy_(torch.arange(pages, dtype=torch.int32, device=gpu))   # the last pages are taken first
    D.cache_reserve(c, ints([0], gpu), ints([150], gpu))
    k = torch.randn((150, kv, dim), device=gpu).bfloat16()
    D.cache_append(c, 0, ints([0], gpu), ints([0, 150], gpu), k, -k)
    D.cache_compact(c, ints([0], gpu), ints([list(range(1, 141))], gpu), ints([140], gpu))
    D.cache_fork(c, ints([0], gpu), ints([2], gpu), share=False)
    torch.cuda.synchronize()
    for s in (0, 2):
        rows = c.page_table[s].long()[torch.arange(140, device=gpu) // page]
        off = torch.arange(140, device=gpu) % page
        assert (rows[0] > 40000)
        assert torch.equal(c.k[0][rows, :, off], k[1:141]) and torch.equal(c.v[0][rows, :, off], -k[1:141])
    assert D.cache_status(c) == (P.PROX_OK, 0)


def test_captured_calls_replay_on_new_contents(gpu):
    b = Both(*make(gpu))
    b.grow(0, 30)
    b.grow(1, 16)
    src, dst, ok = ints([0], gpu), ints([3], gpu), torch.zeros(1, dtype=torch.uint8, device=gpu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.cache_fork(b.c, src, dst, ok=ok)
    g.replay()
    b.m.fork([0], [3], True)
    b.check()
    src.fill_(1)
    dst.fill_(5)
    g.replay()
    b.m.fork([1], [5], True)
    b.check()


def test_another_stream(gpu):
    b = Both(*make(gpu))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.grow(2, 50)
        b.fork([2], [0])
        b.free([2])
        b.check()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_another_device_than_the_current_one():
    b = Both(*make(torch.device("cuda:1")))
    b.grow(2, 50)
    b.fork([2], [0])
    b.check()


def test_binding_refuses_wrong_lists(gpu):
    c, _ = make(gpu)
    one = ints([0], gpu)
    for bad in (one.long(), one.cpu(), one.view(1, 1), torch.zeros(4, dtype=torch.int32, device=gpu)[::2]):
        with pytest.raises(ValueError):
            D.cache_reserve(c, bad, ints([0] * bad.numel(), gpu))
    with pytest.raises(ValueError):
        D.cache_reserve(c, one, ints([1, 2], gpu))
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=gpu)
    for bad in (k.half(), k[:, :1], k[..., :32], k.transpose(0, 1), k.cpu()):
        with pytest.raises(ValueError):
            D.cache_append(c, 0, one, ints([0, 2], gpu), bad, bad)
    with pytest.raises(P.ProxError):
        D.cache_append(c, 2, one, ints([0, 2], gpu), k, k)
    with pytest.raises(P.ProxError):
        D.PagedCache(1, 4, 2, 20, 64, 2, 2, torch.bfloat16, gpu)
    with pytest.raises(ValueError):
        D.PagedCache(1, 4, 2, 16, 64, 2, 2, torch.float32, gpu)
