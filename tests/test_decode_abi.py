"""Argument checks of the decoding-pass calls, on the host (no GPU)."""
import ctypes as C
import os
import re

import pytest
import torch

from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B = 1 << 20


def fake(**over):
    f = dict(n_layers=2, n_pages=64, page_size=16, n_kv_heads=4, head_dim=128, dtype=0, max_seqs=8,
             max_pages=16, **{n: B * (i + 1) for i, n in enumerate(
                 ("k", "v", "page_table", "length", "held", "ref_count", "free_list", "n_free", "status"))})
    f.update(over)
    return D._Cache(**f)


BAD_CACHES = [dict(n_layers=0), dict(n_layers=4097), dict(n_pages=0), dict(page_size=48),
              dict(page_size=256), dict(page_size=0), dict(n_kv_heads=0), dict(head_dim=96),
              dict(dtype=2), dict(dtype=-1), dict(max_seqs=0), dict(max_seqs=4097),
              dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(n_pages=1 << 25),
              dict(max_seqs=4096, max_pages=1 << 18), dict(k=None), dict(v=B + 8),
              dict(page_table=None), dict(status=None), dict(n_free=B + 4)]


def calls(c):
    L = D._lib()
    r = C.byref(c)
    return {
        "init": lambda: L.prox_cache_init(r, None),
        "reserve": lambda: L.prox_cache_reserve(r, 2, B, B, None, None),
        "append": lambda: L.prox_cache_append(r, 0, 2, B, B, 3, B, 512, B, 512, None),
        "fork": lambda: L.prox_cache_fork(r, 2, B, B, 1, None, B, 1 << 20, None),
        "compact": lambda: L.prox_cache_compact(r, 2, B, B, 4, B, None, None),
        "free": lambda: L.prox_cache_free(r, 2, B, None),
        "status": lambda: L.prox_cache_status(r, None, None),
        "attention": lambda: attend(c),
    }


@pytest.mark.parametrize("over", BAD_CACHES, ids=lambda o: "-".join(f"{k}={v}" for k, v in o.items()))
def test_bad_caches_are_refused_by_every_call(over):
    for name, call in calls(fake(**over)).items():
        assert call() == P.PROX_EINVAL, name
    if not any(k in over for k in ("k", "v", "page_table", "status", "n_free")):
        assert D._lib().prox_cache_workspace_bytes(C.byref(fake(**over))) == 0


def test_workspace_size():
    assert D._lib().prox_cache_workspace_bytes(C.byref(fake())) >= 64 * 16
    assert D._lib().prox_cache_workspace_bytes(None) == 0


def test_page_calls_check_counts_and_pointers():
    L, c = D._lib(), fake()
    r = C.byref(c)
    for n in (-1, 9):   # more entries than sequences
        assert L.prox_cache_reserve(r, n, B, B, None, None) == P.PROX_EINVAL
        assert L.prox_cache_fork(r, n, B, B, 1, None, B, 1 << 20, None) == P.PROX_EINVAL
        assert L.prox_cache_compact(r, n, B, B, 4, B, None, None) == P.PROX_EINVAL
        assert L.prox_cache_free(r, n, B, None) == P.PROX_EINVAL
        assert L.prox_cache_append(r, 0, n, B, B, 3, B, 512, B, 512, None) == P.PROX_EINVAL
    # nothing to do, nothing launched
    assert L.prox_cache_reserve(r, 0, None, None, None, None) == P.PROX_OK
    assert L.prox_cache_fork(r, 0, None, None, 0, None, None, 0, None) == P.PROX_OK
    assert L.prox_cache_compact(r, 0, None, None, 4, None, None, None) == P.PROX_OK
    assert L.prox_cache_free(r, 0, None, None) == P.PROX_OK
    assert L.prox_cache_append(r, 0, 0, None, None, 3, None, 512, None, 512, None) == P.PROX_OK
    assert L.prox_cache_append(r, 0, 2, None, None, 0, None, 512, None, 512, None) == P.PROX_OK
    for bad in (None, B + 2):
        assert L.prox_cache_reserve(r, 2, bad, B, None, None) == P.PROX_EINVAL
        assert L.prox_cache_reserve(r, 2, B, bad, None, None) == P.PROX_EINVAL
        assert L.prox_cache_fork(r, 2, bad, B, 1, None, B, 1 << 20, None) == P.PROX_EINVAL
        assert L.prox_cache_fork(r, 2, B, bad, 1, None, B, 1 << 20, None) == P.PROX_EINVAL
        assert L.prox_cache_fork(r, 2, B, B, 1, None, bad, 1 << 20, None) == P.PROX_EINVAL
        assert L.prox_cache_compact(r, 2, B, bad, 4, B, None, None) == P.PROX_EINVAL
        assert L.prox_cache_compact(r, 2, B, B, 4, bad, None, None) == P.PROX_EINVAL
        assert L.prox_cache_free(r, 2, bad, None) == P.PROX_EINVAL
        assert L.prox_cache_append(r, 0, 2, B, bad, 3, B, 512, B, 512, None) == P.PROX_EINVAL
        assert L.prox_cache_append(r, 0, 2, B, B, 3, bad, 512, B, 512, None) == P.PROX_EINVAL
        assert L.prox_cache_append(r, 0, 2, B, B, 3, B, 512, bad, 512, None) == P.PROX_EINVAL
    for share in (-1, 2):
        assert L.prox_cache_fork(r, 2, B, B, share, None, B, 1 << 20, None) == P.PROX_EINVAL
    assert L.prox_cache_fork(r, 2, B, B, 1, None, B, 64 * 16, None) == P.PROX_ENOMEM
    for m in (0, -1, 257):
        assert L.prox_cache_compact(r, 2, B, B, m, B, None, None) == P.PROX_EINVAL
    for layer, stride in ((-1, 512), (2, 512), (0, 508), (0, 511), (0, 504), (0, -512)):
        assert L.prox_cache_append(r, layer, 2, B, B, 3, B, stride, B, 512, None) == P.PROX_EINVAL
        assert L.prox_cache_append(r, layer, 2, B, B, 3, B, 512, B, stride, None) == P.PROX_EINVAL \
            or stride == 512


def attend(c, layer=0, n=2, seqs=B, cu=B, rows=5, max_q=4, heads=16, q=B, q_stride=2048, tree=B,
           words=1, scale=0.1, out=B, out_stride=2048, lse=B, ws=B, ws_bytes=1 << 40):
    return D._lib().prox_tree_attention(C.byref(c), layer, n, seqs, cu, rows, max_q, heads, q, q_stride,
                                        tree, words, scale, out, out_stride, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over", [
    dict(layer=-1), dict(layer=2), dict(n=-1), dict(n=65537), dict(rows=-1), dict(max_q=0),
    dict(max_q=257), dict(heads=0), dict(heads=6), dict(heads=4 * 65), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(words=0),
    dict(max_q=65, words=1), dict(seqs=None), dict(cu=None), dict(q=None), dict(out=None),
    dict(ws=None), dict(q=B + 8), dict(out=B + 8), dict(ws=B + 8), dict(tree=B + 4), dict(lse=B + 2),
    dict(q_stride=2047), dict(q_stride=2040), dict(out_stride=2044), dict(out_stride=0)],
    ids=lambda o: "-".join(f"{k}={v}" for k, v in o.items()))
def test_attention_arguments(over):
    assert attend(fake(), **over) == P.PROX_EINVAL


def test_scales_whose_log2_form_overflows():
    assert attend(fake(), scale=2.4e38) == P.PROX_EINVAL
    assert attend(fake(), scale=2.3e38, n=0) == P.PROX_OK


def test_attention_of_nothing_is_ok():
    assert attend(fake(), n=0, seqs=None, q=None, out=None, ws=None) == P.PROX_OK
    assert attend(fake(), rows=0, seqs=None, q=None, out=None, ws=None) == P.PROX_OK


def score(rows=3, vocab=100, dtype=0, x=B, stride=100, tokens=B, n_tok=1, k=5, logp=B, ent=B, ids=B,
          top=B):
    return D._lib().prox_logprobs(rows, vocab, dtype, x, stride, tokens, n_tok, k, logp, ent, ids, top, None)


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(dtype=3), dict(dtype=-1), dict(x=None),
    dict(x=B + 1), dict(dtype=2, x=B + 2), dict(stride=99), dict(stride=-100), dict(n_tok=-1),
    dict(n_tok=1025), dict(k=-1), dict(k=65), dict(vocab=4, stride=4, k=5), dict(tokens=None),
    dict(logp=None), dict(ids=None), dict(top=None), dict(ent=B + 2), dict(tokens=B + 1)],
    ids=lambda o: "-".join(f"{k}={v}" for k, v in o.items()))
def test_logprobs_arguments(over):
    assert score(**over) == P.PROX_EINVAL


def test_logprobs_of_nothing_is_ok():
    assert score(rows=0, x=None) == P.PROX_OK


def test_headers_and_binding_list_the_same_calls():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "prox_decode.h")).read(), flags=re.S)
    assert set(re.findall(r"\b(prox_\w+)\s*\(", src)) == set(D.ABI_FUNCTIONS)
    assert "range" in P.status_str(D.PROX_EDATA)


def test_binding_checks_tensors():
    x = torch.zeros(3, 10)
    with pytest.raises(ValueError):
        D.logprobs(x)                                    # not on a GPU
    k = torch.zeros(1, 2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.PagedCache.from_tensors(k, k, torch.zeros(2, 2, dtype=torch.int32), i, i, i, i, i[:1])
    with pytest.raises(ValueError):
        D.PagedCache.from_tensors(k.float(), k, torch.zeros(2, 2, dtype=torch.int32), i, i, i, i, i[:1])
    with pytest.raises(ValueError):
        D.PagedCache.from_tensors(k[0], k, torch.zeros(2, 2, dtype=torch.int32), i, i, i, i, i[:1])
