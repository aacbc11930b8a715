"""Decoding with drafted trees: the page operations, tree attention and log
probabilities together with the sparse FFN block, several steps long, each
operator checked on the inputs it met and the cache against the rows that the
accepted tokens had."""
import random

import numpy as np
import pytest
import torch

from decode_helpers import check_attention, check_logprobs, ints, random_tree
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P
from free_ffn_activation_b200 import synth as S

pytestmark = pytest.mark.gpu

D_MODEL, D_FF, HEADS, KV, DIM, VOCAB, LAYERS = 256, 768, 4, 2, 64, 1003, 2


class Model:
    def __init__(self, dev):
        gen = torch.Generator(device=dev)
        gen.manual_seed(3)
        rand = lambda *s: (torch.randn(s, device=dev, generator=gen) * 0.06).bfloat16()  # noqa: E731
        self.embed, self.head = rand(VOCAB, D_MODEL).float() * 20, rand(VOCAB, D_MODEL)
        self.qkv = [rand((HEADS + 2 * KV) * DIM, D_MODEL) for _ in range(LAYERS)]
        self.out = [rand(D_MODEL, HEADS * DIM) for _ in range(LAYERS)]
        self.ffn, self.tau = [], []
        for ell in range(LAYERS):
            L = S.make_layer(S.LayerSpec(D_MODEL, D_FF, sigma=0.05, seed=ell))
            self.ffn.append(P.ProxLayer.from_weights(L["w_up_cm"], L["w_gate_cm"], L["w_down"], device=dev))
            x = P.as_bf16(S.make_tokens(64, D_MODEL, seed=ell, stream="x_cal"), dev)
            self.tau.append(P.calibrate(self.ffn[ell], x, 0.5, 0.4))


def check_pass(cache, rows, seqs, cu, bits, model, tokens, tree):
    """One pass over drafted tokens; returns their k, v rows per layer and the
    log probabilities' result."""
    dev = cache.device
    h = model.embed[tokens]
    new = []
    seqs_d, cu_d = ints(seqs, dev), ints(cu, dev)
    for ell in range(LAYERS):
        qkv = (P.rmsnorm_bf16(h) @ model.qkv[ell].T).view(-1, HEADS + 2 * KV, DIM)
        q, k, v = qkv.split((HEADS, KV, KV), 1)
        D.cache_append(cache, ell, seqs_d, cu_d, k, v)
        out, lse = D.tree_attention(cache, ell, q, seqs_d, cu_d, max(b - a for a, b in zip(cu, cu[1:])), tree=tree)
        torch.cuda.synchronize()
        for i, s in enumerate(seqs):
            r = slice(cu[i], cu[i + 1])
            old_k, old_v = rows[s][ell]
            kk, vv = (torch.cat([a, b[r]]).double().transpose(0, 1) for a, b in ((old_k, k), (old_v, v)))
            t = r.stop - r.start
            seen = torch.ones((t, old_k.shape[0] + t), dtype=torch.bool, device=dev)
            seen[:, old_k.shape[0]:] = bits[i] if bits is not None else torch.ones((t, t), dtype=torch.bool).tril()
            check_attention(out[r], lse[r], q[r], kk, vv, seen, DIM ** -0.5, f"layer {ell} sequence {s}")
        new.append((k, v))
        h = h + (out.reshape(-1, HEADS * DIM) @ model.out[ell].T).float()
        h, _, f = P.ffn_block(model.ffn[ell], h, *model.tau[ell])
        assert torch.isfinite(h).all() and 0 < float(f.mask_s.float().mean()) < 1
    logits = P.rmsnorm_bf16(h) @ model.head.T
    got = D.logprobs(logits, tokens.int().unsqueeze(1), top_k=4)
    torch.cuda.synchronize()
    check_logprobs(logits, tokens.int().unsqueeze(1), 4, got)
    return new, got


def keep(rows, s, new, cu, i, path):
    """The accepted rows of entry i join what sequence s is known to hold."""
    at = torch.tensor([cu[i] + p for p in path], device=new[0][0].device, dtype=torch.long)
    rows[s] = [(torch.cat([a, k[at]]), torch.cat([b, v[at]])) for (a, b), (k, v) in zip(rows[s], new)]


@pytest.mark.parametrize("page", [16, 64])
def test_steps_of_drafting_and_branching(gpu, page):
    rng = random.Random(page)
    model = Model(gpu)
    cache = D.PagedCache(LAYERS, 60, KV, page, DIM, 8, 20, torch.bfloat16, gpu)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    none = lambda: [(torch.zeros((0, KV, DIM), dtype=torch.bfloat16, device=gpu),) * 2 for _ in range(LAYERS)]  # noqa: E731
    rows = {s: none() for s in range(8)}
    # two prompts, a chain each
    lens = [21, 6]
    cu, seqs = [0, 21, 27], [0, 1]
    toks = torch.tensor([rng.randrange(VOCAB) for _ in range(27)], device=gpu)
    D.cache_reserve(cache, ints(seqs, gpu), ints(lens, gpu))
    new, _ = check_pass(cache, rows, seqs, cu, None, model, toks, None)
    path = [list(range(lens[i])) + [0] * (21 - lens[i]) for i in range(2)]
    D.cache_compact(cache, ints(seqs, gpu), ints(path, gpu), ints(lens, gpu))
    for i, s in enumerate(seqs):
        keep(rows, s, new, cu, i, list(range(lens[i])))
    live = [0, 1]
    for step in range(6):
        if step == 2:                       # branches of the first, and a whole copy of the second
            D.cache_fork(cache, ints([0, 0], gpu), ints([4, 2], gpu))
            D.cache_fork(cache, ints([1], gpu), ints([7], gpu), share=False)
            rows[4], rows[2], rows[7] = list(rows[0]), list(rows[0]), list(rows[1])
            live = [0, 1, 4, 2, 7]
        if step == 4:                       # a parent goes, its children stay
            D.cache_free(cache, ints([0, 7], gpu))
            rows[0], rows[7] = none(), none()
            live = [1, 4, 2]
        rng.shuffle(live)
        t = [rng.randint(1, 8) for _ in live]
        cu = [0]
        for x in t:
            cu.append(cu[-1] + x)
        toks = torch.tensor([rng.randrange(VOCAB) for _ in range(cu[-1])], device=gpu)
        trees = [random_tree(rng, x, 1) for x in t]
        tree = ints([r for w in trees for r in w], gpu, torch.int64)
        bits = [torch.tensor([[r[0] >> j & 1 for j in range(x)] for r in w], dtype=torch.bool, device=gpu)
                for w, x in zip(trees, t)]
        ok = torch.zeros(len(live), dtype=torch.uint8, device=gpu)
        D.cache_reserve(cache, ints(live, gpu), ints(t, gpu), ok)
        assert ok.all()
        new, got = check_pass(cache, rows, live, cu, bits, model, toks, tree)
        # the path to the drafted token the model finds likeliest
        path, count = [], []
        for i, x in enumerate(t):
            best = int(got.logp[cu[i]:cu[i + 1], 0].argmax())
            p = [j for j in range(x) if trees[i][best][0] >> j & 1]
            count.append(len(p))
            path.append(p + [0] * (8 - len(p)))
            keep(rows, live[i], new, cu, i, p)
        D.cache_compact(cache, ints(live, gpu), ints(path, gpu), ints(count, gpu))
        torch.cuda.synchronize()
        assert cache.length[live].tolist() == [rows[s][0][0].shape[0] for s in live]
        # shared pages too hold what each sequence accepted
        for s in live:
            n = rows[s][0][0].shape[0]
            pos = torch.arange(n, device=gpu)
            at = cache.page_table[s].long()[pos // page]
            for ell in range(LAYERS):
                assert torch.equal(cache.k[ell][at, :, pos % page], rows[s][ell][0])
                assert torch.equal(cache.v[ell][at, :, pos % page], rows[s][ell][1])
    D.cache_free(cache, ints(live + [-1], gpu))
    assert D.cache_status(cache) == (P.PROX_OK, 0)
    assert int(cache.n_free) == 60 and sorted(cache.free_list.tolist()) == list(range(60))
    assert np.all(cache.ref_count.cpu().numpy() == 0)
