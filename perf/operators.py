"""The operators of a decoding pass over drafted tokens, in plain torch.

What stands next to the sparse feed-forward layer when a model decodes with
passes of one to a few dozen tokens: attention of a tree (or chain) of drafted
tokens over a paged key/value cache, the page operations of that cache, and the
log probabilities that decide which drafted tokens are kept.

``listed`` names the cases, ``prepare`` makes a case's inputs, ``run`` makes one
pass: with ``own`` false in elementary torch operations in 32 bits, with ``own``
true through this repository's entry points. ``exact`` gives the same results
from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(name, n, draft, ctx, kv_heads, group, head_dim, page, dtype="bf16", tree=True):
    return {"name": name, "kind": "attend", "n": n, "draft_min": draft[0], "draft_max": draft[1],
            "ctx_min": ctx[0], "ctx_max": ctx[1], "kv_heads": kv_heads, "group": group,
            "head_dim": head_dim, "page": page, "dtype": dtype, "tree": tree}


def _cache(name, kind, n, copies, ctx, layers, kv_heads, head_dim, page, draft=0, share=True,
           dtype="bf16"):
    return {"name": name, "kind": kind, "n": n, "copies": copies, "ctx_min": ctx[0],
            "ctx_max": ctx[1], "layers": layers, "kv_heads": kv_heads, "head_dim": head_dim,
            "page": page, "draft": draft, "share": share, "dtype": dtype}


def _score(name, rows, vocab, dtype, n_tok, top_k, pad=0):
    return {"name": name, "kind": "score", "rows": rows, "vocab": vocab, "dtype": dtype,
            "n_tok": n_tok, "top_k": top_k, "pad": pad}


def listed():
    return [
        # one sequence, one token: the latency of an ordinary decoding pass
        _attend("attend one token", 1, (1, 1), (1021, 1021), 8, 4, 128, 16, tree=False),
        # one sequence, a pass of eight drafted tokens (the widest pass of the
        # feed-forward layer) behind a prompt of middling length
        _attend("attend pass of 8", 1, (8, 8), (16383, 16383), 8, 4, 128, 64),
        # a batch of short chats of uneven lengths, drafts of uneven sizes,
        # narrow heads, an odd group, small pages, fp16
        _attend("attend ragged batch", 24, (1, 11), (0, 6000), 4, 7, 64, 16, dtype="fp16"),
        # one sequence, a large tree behind a long prompt
        _attend("attend large tree", 1, (64, 64), (32749, 32749), 8, 4, 128, 64),
        # a serving batch: many long prompts, a tree on each
        _attend("attend large batch", 16, (40, 64), (8000, 32000), 8, 4, 128, 64),
        # beams: four children of each of a few short sequences, given back
        _cache("fork beams", "fork", 2, 4, (300, 700), 4, 8, 128, 16),
        # many branches of long shared prompts: nearly all of it is bookkeeping
        _cache("fork long prompts", "fork", 8, 4, (20000, 60000), 1, 8, 128, 16),
        # whole copies of long sequences, all layers: bandwidth
        _cache("copy long sequences", "fork", 4, 1, (9000, 17000), 8, 8, 128, 64, share=False),
        # a speculative step on a branch: fork, reserve, append a tree's rows
        # in every layer, keep the accepted path, free the branch
        _cache("branch and keep", "branch", 8, 2, (900, 5000), 12, 8, 128, 64, draft=32),
        # the next token of one sequence
        _score("score one row", 1, 32000, "bf16", 1, 0),
        # verification of the drafts of a batch, with alternatives
        _score("score drafts", 64, 151936, "bf16", 1, 20),
        # a prompt's tokens scored in fp32, an odd vocabulary in padded rows
        _score("score prompt", 4000, 128257, "fp32", 1, 5, pad=63),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "fork", "branch", "score", "score"))
    if kind == "attend":
        kv, group, dim = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8)), rng.choice((64, 128))
        hi = _log(rng, 16, 32000)
        draft = _log(rng, 1, 64)
        # as much as the largest listed case reads and computes, at most
        n = _log(rng, 1, max(1, min(32, 16 * 20000 * 8 * 128 // ((hi + 64) * kv * dim),
                                    16 * 20000 * 8 * 4 * 52 // ((hi + 64) * kv * group * draft))))
        return {k: v for k, v in _attend(
            "", n, (rng.choice((1, draft)), draft), (rng.choice((0, hi // 3, hi)), hi), kv, group,
            dim, rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "fp16")),
            rng.random() < 0.75).items() if k != "name"}
    if kind in ("fork", "branch"):
        page = rng.choice((16, 32, 64, 128))
        kv, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
        hi = _log(rng, 40, 16000)
        layers, n = _log(rng, 1, 8), _log(rng, 1, 4)
        share = kind == "branch" or rng.random() < 0.6
        copies = _log(rng, 1, 6) if share else 1
        return {k: v for k, v in _cache(
            "", kind, n, copies, (max(1, hi // rng.choice((1, 2, 5))), hi), layers, kv, dim, page,
            draft=_log(rng, 2, 64) if kind == "branch" else 0, share=share,
            dtype=rng.choice(("bf16", "fp16"))).items() if k != "name"}
    vocab = _log(rng, 1000, 160000)
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    rows = _log(rng, 1, max(1, min(4000, 4000 * 128000 * 2 // (vocab * BYTES[dtype]))))
    return {k: v for k, v in _score("", rows, vocab, dtype, rng.choice((1, 1, 3)),
                                    rng.choice((0, 1, 5, 20, 40)),
                                    rng.choice((0, 0, 5, 64))).items() if k != "name"}


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------

def _ragged(count, lo, hi, salt):
    """`count` whole numbers of [lo, hi], the same ones each time; one is hi."""
    r = random.Random(salt * 1000003 + count * 8191 + lo * 31 + hi)
    v = [r.randint(lo, hi) for _ in range(count)]
    v[r.randrange(count)] = hi
    return v


def _attend_sizes(c):
    return (_ragged(c["n"], c["ctx_min"], c["ctx_max"], 1),
            _ragged(c["n"], c["draft_min"], c["draft_max"], 2))


def _path_sizes(c):
    """Accepted drafted tokens of each branch."""
    return _ragged(c["n"] * c["copies"], 1, max(1, min(c["draft"], 8)), 3)


def work(case):
    c, e = case, BYTES[case["dtype"]]
    if c["kind"] == "attend":
        lens, drafts = _attend_sizes(c)
        kv_row = 2 * c["kv_heads"] * c["head_dim"] * e
        heads = c["kv_heads"] * c["group"]
        rows = sum(drafts)
        keys = sum(l + t for l, t in zip(lens, drafts))
        pairs = sum(t * l + t * (t + 1) // 2 for l, t in zip(lens, drafts))
        return {"bytes": keys * kv_row + 2 * rows * heads * c["head_dim"] * e + rows * heads * 4
                + sum(-(-(l + t) // c["page"]) * 4 for l, t in zip(lens, drafts)),
                "flops": 4 * pairs * heads * c["head_dim"]}
    if c["kind"] == "score":
        return {"bytes": c["rows"] * (c["vocab"] * e + c["n_tok"] * 8 + 4 + c["top_k"] * 8),
                "flops": 6 * c["rows"] * c["vocab"]}
    lens = [l for l in _ragged(c["n"], c["ctx_min"], c["ctx_max"], 1) for _ in range(c["copies"])]
    row = 2 * c["layers"] * c["kv_heads"] * c["head_dim"] * e
    moved = sum(l % c["page"] if c["share"] else l for l in lens)
    pages = sum(-(-l // c["page"]) for l in lens)
    ints = pages * 4 * (4 if c["share"] else 6)     # tables read and written, counts up and down
    if c["kind"] == "branch":
        moved += len(lens) * c["draft"] + sum(_path_sizes(c))
    return {"bytes": 2 * moved * row + ints, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tree(rng, t, words):
    """Rows of ancestor-or-self bits of a random tree over t drafted tokens."""
    rows = []
    for i in range(t):
        up = rng.randint(-1, i - 1) if rng.random() < 0.5 else i - 1
        rows.append((rows[up] if up >= 0 else 0) | 1 << i)
    out = []
    for r in rows:
        ws = [r >> (64 * w) & (1 << 64) - 1 for w in range(words)]
        out.append([w - (1 << 64) if w >> 63 else w for w in ws])
    return out


def _randn(shape, dtype, gen):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    if c["kind"] == "score":
        return _prepare_score(c, gen)
    if c["kind"] == "attend":
        return _prepare_attend(c, gen, rng)
    return _prepare_cache(c, gen, rng)


def _pool(c, layers, lens, rng, gen, slots, spare):
    """A cache that holds sequences of `lens` tokens in its first slots, on
    pages in no order, and `spare` free pages."""
    dt, ps = DTYPES[c["dtype"]], c["page"]
    need = [-(-l // ps) for l in lens]
    n_pages = sum(need) + spare
    shape = (layers, n_pages, c["kv_heads"], ps, c["head_dim"])
    ids = list(range(n_pages))
    rng.shuffle(ids)
    cols = max(need + [1]) + spare // max(1, slots - len(lens)) + 2 if slots > len(lens) else max(need + [1])
    table = torch.zeros(slots, cols, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    ref = torch.zeros(n_pages, dtype=torch.int32)
    ref[ids[:at]] = 1
    rest = ids[at:] + [0] * at
    zeros = [0] * (slots - len(lens))
    return {"k": _randn(shape, dt, gen), "v": _randn(shape, dt, gen), "page_table": table.cuda(),
            "length": _ints(lens + zeros), "held": _ints(need + zeros), "ref_count": ref.cuda(),
            "free_list": _ints(rest), "n_free": _ints([n_pages - at])}


POOL = ("k", "v", "page_table", "length", "held", "ref_count", "free_list", "n_free")


def _own_cache(s):
    from free_ffn_activation_b200 import decode
    return decode.PagedCache.from_tensors(**{k: s[k] for k in POOL})


def _prepare_attend(c, gen, rng):
    lens, drafts = _attend_sizes(c)
    heads = c["kv_heads"] * c["group"]
    # the drafted rows are in the cache behind the committed ones
    s = _pool(c, 1, [l + t for l, t in zip(lens, drafts)], rng, gen, c["n"], 0)
    s["length"] = _ints(lens)
    rows, words = sum(drafts), -(-max(drafts) // 64)
    # queries are a view of the fused projection's output
    qkv = _randn((rows, heads + 2 * c["kv_heads"], c["head_dim"]), DTYPES[c["dtype"]], gen)
    order = list(range(c["n"]))
    rng.shuffle(order)
    cu = [0]
    for b in order:
        cu.append(cu[-1] + drafts[b])
    s |= {"case": c, "q": qkv[:, :heads], "seqs": _ints(order), "cu": _ints(cu), "max_q": max(drafts),
          "longest": max(l + t for l, t in zip(lens, drafts)), "tree": None,
          "scale": c["head_dim"] ** -0.5, "lens": lens, "drafts": drafts, "order": order}
    if c["tree"]:
        s["tree"] = _ints([r for b in order for r in _tree(rng, drafts[b], words)], torch.int64)
    if own:
        from free_ffn_activation_b200 import decode
        s["cache"] = _own_cache(s)
        s["ws"] = decode.attention_workspace(s["cache"], s["max_q"], heads)
    return s


def _prepare_cache(c, gen, rng):
    n, copies, ps, draft = c["n"], c["copies"], c["page"], c["draft"]
    lens = _ragged(n, c["ctx_min"], c["ctx_max"], 1)
    kids = [l for l in lens for _ in range(copies)]
    fresh = [(1 if l % ps else 0) if c["share"] else -(-l // ps) for l in kids]
    more = [-(-(l + draft) // ps) - -(-l // ps) for l in kids]
    s = _pool(c, c["layers"], lens, rng, gen, n + len(kids), sum(fresh) + sum(more) + 3)
    src = [i for i in range(n) for _ in range(copies)]
    dst = list(range(n, n + len(kids)))
    rng.shuffle(dst)
    s |= {"case": c, "src": _ints(src), "dst": _ints(dst), "lens": lens, "kids": kids, "src_host": src,
          "dst_host": dst, "fresh": fresh, "more": more}
    if c["kind"] == "branch":
        kept = _path_sizes(c)
        path = [sorted(rng.sample(range(draft), k)) + [0] * (max(kept) - k) for k in kept]
        new = (c["layers"], len(kids) * draft, c["kv_heads"], c["head_dim"])
        s |= {"n_new": _ints([draft] * len(kids)), "cu": _ints([draft * i for i in range(len(kids) + 1)]),
              "k_new": _randn(new, DTYPES[c["dtype"]], gen), "v_new": _randn(new, DTYPES[c["dtype"]], gen),
              "path": _ints(path), "n_path": _ints(kept), "path_host": path, "kept": kept}
    if own:
        s["cache"] = _own_cache(s)
    else:
        s |= _lists(s)
    return s


def _lists(s):
    """Which (entry, place) pairs the plain form of the page operations works
    on: a host that knows the lengths knows them."""
    c = s["case"]
    ps = c["page"]
    flat = lambda counts: (torch.tensor([i for i, k in enumerate(counts) for _ in range(k)], device="cuda", dtype=torch.long),
                           torch.tensor([j for k in counts for j in range(k)], device="cuda", dtype=torch.long))
    held = [-(-l // ps) for l in s["kids"]]
    got = {"shared": flat([l // ps for l in s["kids"]] if c["share"] else [0] * len(held)),
           "held_list": flat([h + m for h, m in zip(held, s["more"])]), "fresh_list": flat(s["fresh"]),
           "more_list": flat(s["more"])}
    i, j = got["fresh_list"]
    first = torch.tensor([l // ps if c["share"] else 0 for l in s["kids"]], device="cuda", dtype=torch.long)
    got["fresh_col"] = j + first[i]
    lens = torch.tensor(s["kids"], device="cuda", dtype=torch.long)
    got["fresh_rows"] = (lens[i] - got["fresh_col"] * ps).clamp(max=ps)
    if c["kind"] == "branch":
        got["drafted"] = flat([c["draft"]] * len(held))
        got["path_list"] = flat(s["kept"])
    return got


def _prepare_score(c, gen):
    wide = _randn((c["rows"], c["vocab"] + c["pad"]), torch.float32, gen).mul_(2.5)
    logits = wide[:, :c["vocab"]]
    # a few likely tokens, as a model gives them
    at = torch.randint(0, c["vocab"], (c["rows"], 4), device="cuda", generator=gen)
    logits.scatter_add_(1, at, torch.rand((c["rows"], 4), device="cuda", generator=gen) * 12)
    tokens = torch.randint(0, c["vocab"], (c["rows"], c["n_tok"]), device="cuda", generator=gen)
    tokens[:, :1] = at[:, :1]
    return {"case": c, "logits": wide.to(DTYPES[c["dtype"]])[:, :c["vocab"]], "tokens": tokens.int()}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"attend": _own_attend, "score": _own_score}.get(kind, _own_pages)(state)
    return {"attend": _plain_attend, "score": _plain_score}.get(kind, _plain_pages)(state)


def _own_attend(s):
    from free_ffn_activation_b200 import decode
    out, lse = decode.tree_attention(s["cache"], 0, s["q"], s["seqs"], s["cu"], s["max_q"],
                                     tree=s["tree"], scale=s["scale"], ws=s["ws"])
    return {"out": out, "lse": lse}


def _own_score(s):
    from free_ffn_activation_b200 import decode
    r = decode.logprobs(s["logits"], s["tokens"], top_k=s["case"]["top_k"])
    return _score_out(s, r.logp, r.entropy, r.top_ids, r.top_logp)


def _own_pages(s):
    from free_ffn_activation_b200 import decode
    c, cache = s["case"], s["cache"]
    decode.cache_fork(cache, s["src"], s["dst"], share=c["share"])
    if c["kind"] == "branch":
        decode.cache_reserve(cache, s["dst"], s["n_new"])
        for layer in range(c["layers"]):
            decode.cache_append(cache, layer, s["dst"], s["cu"], s["k_new"][layer], s["v_new"][layer])
        decode.cache_compact(cache, s["dst"], s["path"], s["n_path"])
    decode.cache_free(cache, s["dst"])
    return {k: s[k] for k in POOL}


def _score_out(s, logp, entropy, ids, top):
    return {"logp": logp, "entropy": entropy} | ({"top_ids": ids, "top_logp": top} if s["case"]["top_k"] else {})


def _plain_score(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    z = x - m
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    norm = total.log()
    entropy = norm[:, 0] - (e * torch.where(e > 0, z, 0.0)).sum(-1) / total[:, 0]
    logp = z.gather(1, s["tokens"].long()) - norm
    k = s["case"]["top_k"]
    if not k:
        return _score_out(s, logp, entropy, None, None)
    # equal values stay in the order of their places
    top, at = torch.sort(z, dim=-1, descending=True, stable=True)
    return _score_out(s, logp, entropy, at[:, :k].int(), top[:, :k] - norm)


def _plain_attend(s):
    c = s["case"]
    kv, group, dim, ps = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    seqs, cu, t_max = s["seqs"].long(), s["cu"].long(), s["max_q"]
    n, dev = seqs.numel(), s["q"].device
    length, count = s["length"][seqs].long(), cu[1:] - cu[:-1]
    pos = torch.arange(s["longest"], device=dev)
    there = pos < (length + count)[:, None]
    page = torch.where(there, s["page_table"][seqs][:, pos // ps].long(), 0)
    k = s["k"][0][page, :, pos % ps].float().permute(0, 2, 1, 3)        # [n, kv, longest, dim]
    v = s["v"][0][page, :, pos % ps].float().permute(0, 2, 1, 3)
    t = torch.arange(t_max, device=dev)
    row = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)            # [n, t_max]
    q = s["q"][row].float().view(n, t_max, kv, group, dim).permute(0, 2, 1, 3, 4)
    j = pos - length[:, None]                                           # drafted index of a key
    if s["tree"] is None:
        seen = j[:, None] <= t[:, None]
    else:
        jc = j.clamp(0, s["tree"].shape[1] * 64 - 1)[:, None].expand(n, t_max, -1)
        seen = (s["tree"][row].gather(2, jc // 64) >> (jc % 64) & 1).bool() | (j < 0)[:, None]
    seen = (seen & there[:, None])[:, None, :, None]                    # [n, 1, t_max, 1, longest]
    x = q.reshape(n, kv, t_max * group, dim) @ k.transpose(2, 3)
    x = (x * s["scale"]).view(n, kv, t_max, group, -1).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - torch.where(m == -math.inf, 0.0, m)).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(n, kv, t_max * group, -1) @ v).view(n, kv, t_max, group, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(n, t_max, kv * group, dim)
    lse = (m + total.log())[..., 0].permute(0, 2, 1, 3).reshape(n, t_max, kv * group)
    r = torch.arange(s["q"].shape[0], device=dev)
    b = torch.bucketize(r, cu[1:], right=True)
    at = r - cu[b]
    return {"out": o[b, at].to(s["q"].dtype), "lse": lse[b, at]}


def _plain_pages(s):
    c = s["case"]
    ps, src, dst = c["page"], s["src"].long(), s["dst"].long()
    k, v, table, length, held = s["k"], s["v"], s["page_table"], s["length"], s["held"]
    ref, free, n_free = s["ref_count"], s["free_list"], s["n_free"]

    # fork: whole pages are shared (or copied), the part of a page behind them is copied
    length[dst] = length[src]
    held[dst] = (length[src] + ps - 1) // ps
    i, j = s["shared"]
    page = table[src[i], j]
    table[dst[i], j] = page
    ref.index_add_(0, page, torch.ones_like(page))
    i, j = s["fresh_list"][0], s["fresh_col"]
    old, new = table[src[i], j].long(), _pop(free, n_free, i.numel())
    table[dst[i], j] = new.int()
    ref[new] = 1
    part = (torch.arange(ps, device=k.device) < s["fresh_rows"][:, None])[None, :, None, :, None]
    k[:, new] = torch.where(part, k[:, old], k[:, new])
    v[:, new] = torch.where(part, v[:, old], v[:, new])

    if c["kind"] == "branch":
        # reserve pages for the drafted rows
        i, j = s["more_list"]
        new = _pop(free, n_free, i.numel())
        table[dst[i], held[dst[i]].long() + j] = new.int()
        ref[new] = 1
        held[dst] = torch.maximum(held[dst], (length[dst] + s["n_new"] + ps - 1) // ps)
        # append them
        i, j = s["drafted"]
        at = length[dst[i]].long() + j
        page = table[dst[i], at // ps].long()
        k[:, page, :, at % ps] = s["k_new"].transpose(0, 1)
        v[:, page, :, at % ps] = s["v_new"].transpose(0, 1)
        # keep the accepted path
        i, j = s["path_list"]
        base = length[dst[i]].long()
        a, b = base + s["path"][i, j], base + j
        pa, pb = table[dst[i], a // ps].long(), table[dst[i], b // ps].long()
        k[:, pb, :, b % ps] = k[:, pa, :, a % ps]
        v[:, pb, :, b % ps] = v[:, pa, :, a % ps]
        length[dst] += s["n_path"]

    # free: a page that nobody holds any more goes back, in the order of its first listing
    i, j = s["held_list"]
    page = table[dst[i], j].long()
    ref.index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))
    order = torch.arange(page.numel(), device=page.device)
    first = torch.full_like(ref, page.numel(), dtype=torch.long).scatter_reduce_(0, page, order, "amin")
    gone = (ref[page] == 0) & (first[page] == order)
    rank = torch.cumsum(gone, 0) - 1
    # (pages that stay are written to the place behind the list's end)
    wide = torch.cat([free, free[:1]])
    wide[torch.where(gone, n_free + rank, free.numel())] = page.int()
    free.copy_(wide[:-1])
    n_free += gone.sum()
    length[dst] = 0
    held[dst] = 0
    return {key: s[key] for key in POOL}


def _pop(free, n_free, count):
    got = free[n_free.long() - 1 - torch.arange(count, device=free.device)].long()
    n_free -= count
    return got


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "score": _exact_score}.get(case["kind"], _exact_pages)(s)


def _exact_score(s):
    k, parts = s["case"]["top_k"], []
    for x, tokens in zip(s["logits"].split(256), s["tokens"].split(256)):
        logp = torch.log_softmax(x.double(), -1)
        entropy = -torch.special.xlogy(logp.exp(), logp.exp()).sum(-1)
        top = logp.topk(k, -1).values if k else None
        parts.append((logp.gather(1, tokens.long()), entropy, top))
    logp, entropy = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    return _score_out(s, logp, entropy, None, torch.cat([p[2] for p in parts]) if k else None)


def _exact_attend(s):
    c = s["case"]
    ps, dim, group = c["page"], c["head_dim"], c["group"]
    cu = s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, b in enumerate(s["order"]):
        l, t = s["lens"][b], s["drafts"][b]
        pages = s["page_table"][b, :-(-(l + t) // ps)].long()
        rows = slice(cu[i], cu[i + 1])
        seen = torch.ones(t, l + t, dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen = seen.tril(l)
        else:
            bit = torch.arange(t, device="cuda")
            seen[:, l:] = (s["tree"][rows][:, bit // 64] >> (bit % 64)) & 1 == 1
        for h in range(c["kv_heads"]):
            key = s["k"][0, pages, h].reshape(-1, dim)[:l + t].double()
            val = s["v"][0, pages, h].reshape(-1, dim)[:l + t].double()
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][rows, g].double() @ key.T * s["scale"]).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                p = torch.where(z[:, None] > -math.inf, (x - z[:, None]).exp(), 0.0)
                out[rows, g] = p @ val
                lse[rows, g] = z
    return {"out": out, "lse": lse}


def _exact_pages(s):
    c, ps = s["case"], s["case"]["page"]
    k, v = s["k"].clone(), s["v"].clone()
    table, length, held = s["page_table"].tolist(), s["length"].tolist(), s["held"].tolist()
    ref, n_free = s["ref_count"].tolist(), s["n_free"].item()
    free = s["free_list"].tolist()

    def new_page():
        nonlocal n_free
        n_free -= 1
        ref[free[n_free]] = 1
        return free[n_free]

    for a, b in zip(s["src_host"], s["dst_host"]):
        length[b], held[b] = length[a], -(-length[a] // ps)
        for j in range(held[b]):
            page, rows = table[a][j], min(ps, length[a] - j * ps)
            if c["share"] and rows == ps:
                ref[page] += 1
            else:
                to = new_page()
                k[:, to, :, :rows], v[:, to, :, :rows] = k[:, page, :, :rows], v[:, page, :, :rows]
                page = to
            table[b][j] = page
    if c["kind"] == "branch":
        for b in s["dst_host"]:
            while held[b] * ps < length[b] + c["draft"]:
                table[b][held[b]] = new_page()
                held[b] += 1
        for i, b in enumerate(s["dst_host"]):
            at = torch.arange(length[b], length[b] + c["draft"], device="cuda")
            page = torch.tensor(table[b], device="cuda")[at // ps]
            new = slice(i * c["draft"], (i + 1) * c["draft"])
            k[:, page, :, at % ps] = s["k_new"][:, new].transpose(0, 1)
            v[:, page, :, at % ps] = s["v_new"][:, new].transpose(0, 1)
            for to, frm in enumerate(s["path_host"][i][:s["kept"][i]]):
                (x, y), (p, q) = divmod(length[b] + frm, ps), divmod(length[b] + to, ps)
                k[:, table[b][p], :, q] = k[:, table[b][x], :, y].clone()
                v[:, table[b][p], :, q] = v[:, table[b][x], :, y].clone()
            length[b] += s["kept"][i]
    gone = []
    for b in s["dst_host"]:
        for page in table[b][:held[b]]:
            ref[page] -= 1
            gone.append(page)
        length[b] = held[b] = 0
    for page in dict.fromkeys(gone):
        if ref[page] == 0:
            free[n_free] = page
            n_free += 1
    return {"k": k.double(), "v": v.double(), "page_table": _ints(table), "length": _ints(length),
            "held": _ints(held), "ref_count": _ints(ref), "free_list": _ints(free), "n_free": _ints([n_free])}
