"""Plain models of the decoding-pass operators for their tests: the cache's
page operations on host lists, attention and log probabilities in 64 bits, and
the error bounds that the kernels' roundings allow."""
import math
import random

import torch

from free_ffn_activation_b200 import decode as D

INTS = ("page_table", "length", "held", "ref_count", "free_list", "n_free")


class CacheModel:
    """The cache's calls, entry by entry, on CPU copies of its tensors."""

    def __init__(self, cache: D.PagedCache):
        self.ps, self.n_pages = cache.page_size, cache.n_pages
        self.max_seqs, self.max_pages = cache.max_seqs, cache.max_pages
        self.k, self.v = cache.k.cpu().clone(), cache.v.cpu().clone()
        for name in INTS:
            setattr(self, name, getattr(cache, name).cpu().tolist())
        self.status = 0

    def _entries(self, seqs):
        """(i, s) of entries that are neither padding, out of range nor a repetition."""
        seen = set()
        for i, s in enumerate(seqs):
            if not 0 <= s < self.max_seqs:
                self.status |= 0 if s == -1 else D.CACHE_BAD_SEQ
            elif s in seen:
                self.status |= D.CACHE_BAD_SEQ
            else:
                seen.add(s)
                yield i, s

    def _pop(self):
        self.n_free[0] -= 1
        p = self.free_list[self.n_free[0]]
        assert self.ref_count[p] == 0
        self.ref_count[p] = 1
        return p

    def _take(self, needs):
        """Entries (by index) that get their pages, of {index: pages}."""
        ok, total, free = [], 0, self.n_free[0]
        for i, need in needs.items():
            total += need
            if need == 0 or total <= free:
                ok.append(i)
            else:
                self.status |= D.CACHE_FULL
        return ok

    def reserve(self, seqs, n_new):
        needs, who = {}, {}
        for i, s in self._entries(seqs):
            want = -(-(self.length[s] + n_new[i]) // self.ps)
            if n_new[i] < 0:
                self.status |= D.CACHE_BAD_ARG
            elif want > self.max_pages:
                self.status |= D.CACHE_FULL
            else:
                needs[i], who[i] = max(0, want - self.held[s]), s
        ok = self._take(needs)
        for i in ok:
            for _ in range(needs[i]):
                self.page_table[who[i]][self.held[who[i]]] = self._pop()
                self.held[who[i]] += 1
        return [int(i in ok) for i in range(len(seqs))]

    def place(self, s, pos):
        return self.page_table[s][pos // self.ps], pos % self.ps

    def append(self, layer, seqs, cu, k_new, v_new):
        k_new, v_new = k_new.cpu(), v_new.cpu()
        seen = set()
        for i, s in enumerate(seqs):
            if cu[i + 1] == cu[i]:
                continue
            if not 0 <= s < self.max_seqs or s in seen:
                self.status |= 0 if s == -1 else D.CACHE_BAD_SEQ
                continue
            seen.add(s)
            for t in range(cu[i + 1] - cu[i]):
                pos = self.length[s] + t
                if pos >= self.held[s] * self.ps:
                    self.status |= D.CACHE_FULL
                    continue
                p, o = self.place(s, pos)
                self.k[layer, p, :, o] = k_new[cu[i] + t]
                self.v[layer, p, :, o] = v_new[cu[i] + t]

    def fork(self, src, dst, share):
        needs, who = {}, {}
        len0, held0 = list(self.length), list(self.held)
        for i, d in self._entries(dst):
            s = src[i]
            if not 0 <= s < self.max_seqs:
                self.status |= 0 if s == -1 else D.CACHE_BAD_SEQ
            elif len0[d] or held0[d]:
                self.status |= D.CACHE_BAD_ARG
            else:
                n = len0[s]
                needs[i] = int(n % self.ps > 0) if share else -(-n // self.ps)
                who[i] = (s, d)
        for s in src:   # the kernel looks at a source even where the target is left out
            if s != -1 and not 0 <= s < self.max_seqs:
                self.status |= D.CACHE_BAD_SEQ
        ok = self._take(needs)
        for i in ok:
            s, d = who[i]
            self.length[d], self.held[d] = len0[s], -(-len0[s] // self.ps)
            for j in range(self.held[d]):
                p, rows = self.page_table[s][j], min(self.ps, len0[s] - j * self.ps)
                if share and rows == self.ps:
                    self.ref_count[p] += 1
                else:
                    to = self._pop()
                    self.k[:, to, :, :rows] = self.k[:, p, :, :rows]
                    self.v[:, to, :, :rows] = self.v[:, p, :, :rows]
                    p = to
                self.page_table[d][j] = p
        return [int(i in ok) for i in range(len(dst))]

    def compact(self, seqs, path, n_path):
        ok = [0] * len(seqs)
        for i, s in self._entries(seqs):
            m, room = n_path[i], self.held[s] * self.ps - self.length[s]
            p = path[i][:m] if 0 <= m <= len(path[i]) else None
            if p is None or any(not 0 <= x < room for x in p) or any(a >= b for a, b in zip(p, p[1:])):
                self.status |= D.CACHE_BAD_ARG
                continue
            for j, x in enumerate(p):
                (a, ao), (b, bo) = self.place(s, self.length[s] + x), self.place(s, self.length[s] + j)
                self.k[:, b, :, bo] = self.k[:, a, :, ao].clone()
                self.v[:, b, :, bo] = self.v[:, a, :, ao].clone()
            self.length[s] += m
            ok[i] = 1
        return ok

    def free(self, seqs):
        gone = []
        for _, s in self._entries(seqs):
            for p in self.page_table[s][:self.held[s]]:
                self.ref_count[p] -= 1
                gone.append(p)
            self.length[s] = self.held[s] = 0
        for p in dict.fromkeys(gone):
            if self.ref_count[p] == 0:
                self.free_list[self.n_free[0]] = p
                self.n_free[0] += 1

    def check(self, cache: D.PagedCache, rows=True):
        torch.cuda.synchronize()
        for name in INTS:
            assert getattr(cache, name).cpu().tolist() == getattr(self, name), name
        if rows:
            same = lambda a, b: torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))  # noqa: E731
            assert same(cache.k, self.k) and same(cache.v, self.v)
        assert D.cache_status(cache)[1] == self.status
        self.status = 0


def ints(v, dev, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=dev)


def random_tree(rng, t, words):
    """Ancestor-or-self bits of a random tree, int64 [t][words]."""
    rows = []
    for i in range(t):
        up = rng.randint(-1, i - 1)
        rows.append((rows[up] if up >= 0 else 0) | 1 << i)
    return tree_words(rows, words)


def tree_words(rows, words):
    cut = [[r >> 64 * w & (1 << 64) - 1 for w in range(words)] for r in rows]
    return [[w - (1 << 64) if w >> 63 else w for w in r] for r in cut]


class Drafted:
    """A cache with committed and drafted rows and the queries of a pass."""

    def __init__(self, dev, lens, drafts, *, kv_heads=2, group=4, dim=128, page=16,
                 dtype=torch.bfloat16, tree=None, seed=0, layers=1, layer=0, spare=2, order=None,
                 fill=float("nan"), extra_rows=0, max_q=None, words=None, seqs=None):
        rng = random.Random(seed)
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        n = len(lens)
        cols = max([-(-(l + t) // page) for l, t in zip(lens, drafts)] + [1])
        pages = sum(-(-(l + t) // page) for l, t in zip(lens, drafts)) + spare
        self.cache = c = D.PagedCache(layers, pages, kv_heads, page, dim, n, cols, dtype, dev)
        # what no sequence has written must not matter
        c.k.fill_(fill)
        c.v.fill_(fill)
        ids = list(range(pages))
        rng.shuffle(ids)
        table = torch.zeros(n, cols, dtype=torch.int32)
        self.layer, self.lens, self.drafts, self.group = layer, lens, drafts, group
        at = 0
        for s, (l, t) in enumerate(zip(lens, drafts)):
            k = -(-(l + t) // page)
            table[s, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
            at += k
            pos = torch.arange(l + t, device=dev)
            rows = table[s].to(dev).long()[pos // page] if l + t else pos
            for pool in (c.k, c.v):
                new = torch.randn((l + t, kv_heads, dim), device=dev, generator=gen).to(dtype)
                pool[layer][rows, :, pos % page] = new
        c.page_table.copy_(table)
        c.length.copy_(torch.tensor(lens, dtype=torch.int32))
        c.held.copy_(torch.tensor([-(-(l + t) // page) for l, t in zip(lens, drafts)],
                                  dtype=torch.int32))
        self.order = list(range(n)) if order is None else order
        self.seqs = ints(self.order if seqs is None else seqs, dev)
        self.cu_host = [0]
        for s in self.order:
            self.cu_host.append(self.cu_host[-1] + drafts[s])
        self.cu = ints(self.cu_host, dev)
        rows = self.cu_host[-1] + extra_rows
        heads = kv_heads * group
        wide = torch.randn((rows, heads + 2 * kv_heads, dim), device=dev, generator=gen).to(dtype)
        self.q = wide[:, :heads]
        self.max_q = max_q or max(drafts + [1])
        self.words = words or -(-self.max_q // 64)
        self.tree = None
        if tree is not None:
            per = [random_tree(rng, drafts[s], self.words) if tree == "random" else tree(s, drafts[s], self.words)
                   for s in self.order]
            self.tree = ints([r for p in per for r in p] + [[0] * self.words] * extra_rows, dev, torch.int64)
            self.tree = self.tree.view(rows, self.words)
        self.scale = dim ** -0.5

    def rows_of(self, s):
        """k, v of sequence s's tokens, [heads][tokens][dim] in fp64."""
        c, n = self.cache, self.lens[s] + self.drafts[s]
        pos = torch.arange(n, device=c.device)
        page = c.page_table[s].long()[pos // c.page_size]
        return tuple(p[self.layer][page, :, pos % c.page_size].double().transpose(0, 1)
                     for p in (c.k, c.v))

    def seen(self, i, s):
        l, t = self.lens[s], self.drafts[s]
        m = torch.ones((t, l + t), dtype=torch.bool, device=self.cache.device)
        if self.tree is None:
            return m.tril(l)
        bit = torch.arange(t, device=m.device)
        w = self.tree[self.cu_host[i]:self.cu_host[i + 1]]
        m[:, l:] = (w[:, bit // 64] >> (bit % 64)) & 1 == 1
        return m

    def run(self, **kw):
        return D.tree_attention(self.cache, self.layer, self.q, self.seqs, self.cu, self.max_q,
                                tree=self.tree, scale=self.scale, **kw)

    def check(self, out, lse):
        torch.cuda.synchronize()
        for i, s in enumerate(self.order):
            r = slice(self.cu_host[i], self.cu_host[i + 1])
            if r.start < r.stop:
                check_attention(out[r], lse[r], self.q[r], *self.rows_of(s), self.seen(i, s), self.scale,
                                f"sequence {s}")


def check_attention(out, lse, q, k, v, seen, scale, what=""):
    """Compares one sequence's rows (q [rows][heads][dim], k and v
    [kv_heads][tokens][dim] in fp64, seen [rows][tokens]) with the formula in
    64 bits, within what the roundings allow.

    u: rounding of a value to the output's type (half a step), which the
    probabilities meet once and the result once. A score is a sum of `dim`
    fp32 products (each step off by at most 2^-23 of the sum of their
    magnitudes); e^x adds 2^-21, the sum over n keys n 2^-23. fp16
    probabilities below its normal range are off by up to 2^-25."""
    dim, n = k.shape[2], k.shape[1]
    u = torch.finfo(out.dtype).eps / 2
    group = q.shape[1] // k.shape[0]
    empty = ~seen.any(1)
    for h in range(q.shape[1]):
        kh, vh, qh = k[h // group], v[h // group], q[:, h].double()
        assert not (seen & (~torch.isfinite(kh)).any(1)).any(), "the model takes finite keys where they are seen"
        kz, vz = torch.nan_to_num(kh, 0, 0, 0), torch.nan_to_num(vh, 0, 0, 0)
        x = (qh @ kz.T * scale).masked_fill(~seen, -math.inf)
        z = torch.logsumexp(x, 1)
        p = torch.where(seen, (x - torch.where(z == -math.inf, 0.0, z)[:, None]).exp(), 0.0)
        o, a = p @ vz, p @ vz.abs()
        for j in (~torch.isfinite(vh)).any(1).nonzero()[:, 0].tolist():
            rows = seen[:, j]
            o[rows] += p[rows, j:j + 1] * torch.where(torch.isfinite(vh[j]), 0.0, vh[j])
        size = qh.abs() @ kz.T.abs() * scale
        dp = (dim + 8) * 2.0 ** -23 * (size * seen).amax(1, keepdim=True) + 2.0 ** -21
        tol = a * (u + 2 * dp + n * 2.0 ** -23) * (1 + u) + u * o.abs() + 1e-30
        if out.dtype == torch.float16:
            tol = tol + n * 2.0 ** -25 * vz.abs().max() * 2 + 2.0 ** -25
        got = out[:, h].double()
        odd = ~torch.isfinite(o)
        assert torch.equal(torch.isnan(got), torch.isnan(o)), f"NaN: {what} head {h}"
        assert torch.equal(got[odd & ~torch.isnan(o)], o[odd & ~torch.isnan(o)])
        bad = ((got - o).abs() > tol) & ~odd
        assert not bad.any(), f"{what} head {h}: off by {(got - o)[bad].abs().max()}, allowed {tol[bad].min()}"
        gz = lse[:, h].double()
        assert (gz[empty] == -math.inf).all() and (got[empty] == 0).all()
        lt = dp[:, 0] + n * 2.0 ** -23 + 2.0 ** -21 * z.abs().clamp(min=1)
        assert (((gz - z).abs() <= lt) | empty).all(), f"lse: {what} head {h}"


def check_logprobs(logits, tokens, top_k, got):
    """Compares with the definition in 64 bits. With z the log2-scaled distance
    to the maximum, e^z is off by 2^-21 + |z| 2^-23 (two roundings of z), a
    thread's sum of t terms by t 2^-24 more; the result's own rounding 2^-24."""
    x = logits.double()
    rows, vocab = x.shape
    m = x.amax(1, keepdim=True)
    none = (m == -math.inf)[:, 0]
    z = torch.where(x == -math.inf, -math.inf, x - torch.where(m == -math.inf, 0.0, m))
    e = z.exp()
    s0 = e.sum(1)
    ez = (e * torch.where(e > 0, z.abs(), 0.0)).sum(1) / s0      # mean distance
    ds = 2.0 ** -21 + 2.0 ** -23 * 1.5 * ez + (vocab / 256 + 64) * 2.0 ** -24
    ent = s0.log() + ez
    ent = torch.where(none, 0.0, ent)
    bad = torch.isnan(s0) & ~none
    logp = torch.where(none[:, None], -math.inf, z - s0.log()[:, None])
    # the result's type is fp32, and rounding to nearest takes a magnitude of
    # 2^128 - 2^103 (the largest number and half a step) or more to infinity: the
    # type's lowest value under its largest one is -6.8e38
    logp = torch.where(logp <= -(2.0 ** 128 - 2.0 ** 103), -math.inf, logp)

    def close(got, want, tol, what):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), what
        ok = (got == want) | ((got - want).abs() <= tol) | torch.isnan(want)
        assert ok.all(), f"{what}: {got[~ok][:4].tolist()} for {want[~ok][:4].tolist()}"

    close(got.entropy, torch.where(bad, math.nan, ent),
          torch.nan_to_num(ds * (1 + 2.1 * ez) + 2.0 ** -23 * ent, 0, 0, 0), "entropy")
    if tokens is not None and tokens.shape[1]:
        t = tokens.long()
        inside = (t >= 0) & (t < vocab)
        want = logp.gather(1, t.clamp(0, vocab - 1))
        want = torch.where(inside & ~bad[:, None], want, math.nan)
        close(got.logp, want, torch.nan_to_num(ds[:, None] + 2.0 ** -23 * want.abs(), 1e30, 0, 0), "logp")
    if top_k:
        # NaN first, then descending, equal ones by index
        key = torch.where(torch.isnan(x), math.inf, x)
        nan_first = torch.sort((~torch.isnan(x)).to(torch.int8), dim=1, stable=True).indices
        by = torch.sort(key.gather(1, nan_first), dim=1, descending=True, stable=True).indices
        at = nan_first.gather(1, by)[:, :top_k]
        assert torch.equal(got.top_ids.long(), at), "top_ids"
        want = torch.where(bad[:, None], math.nan, logp.gather(1, at))
        close(got.top_logp, want, torch.nan_to_num(ds[:, None] + 2.0 ** -23 * want.abs(), 1e30, 0, 0), "top_logp")
