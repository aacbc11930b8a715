"""Binding of the decoding-pass calls of libprox (``include/prox_decode.h``):
a paged key/value cache with its page operations, attention of drafted tokens
over it, and token log probabilities. What stands next to the sparse FFN of
``prox`` in a pass of one to a few dozen tokens.

Argument marshalling only, as in ``prox``: every step runs in the CUDA kernels
behind the C ABI, calls are enqueued on the current torch stream of the
tensors' device, and argument errors raise before anything is launched. Whole
numbers that live on the device are checked by the kernels; ``cache_status``
reads what they found.
"""
from __future__ import annotations

import ctypes as C
import functools
from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import prox as P
from .prox import PROX_EINVAL, PROX_OK, ProxError

PROX_EDATA = 6

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # PROX_BF16, PROX_FP16, PROX_FP32

# bits of the cache's status word
CACHE_BAD_SEQ, CACHE_FULL, CACHE_BAD_STATE, CACHE_BAD_ARG, CACHE_TIMEOUT = 1, 2, 4, 8, 16

MAX_DRAFT = 256      # drafted tokens of one sequence in tree_attention
MAX_TOP = 64         # alternatives of logprobs

ABI_FUNCTIONS = (
    "prox_cache_init", "prox_cache_workspace_bytes", "prox_cache_reserve", "prox_cache_append",
    "prox_cache_fork", "prox_cache_compact", "prox_cache_free", "prox_cache_status",
    "prox_attention_workspace_bytes", "prox_tree_attention", "prox_logprobs",
)


class _Cache(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_layers", "n_pages", "page_size", "n_kv_heads", "head_dim",
                                       "dtype", "max_seqs", "max_pages")] + \
               [(n, C.c_void_p) for n in ("k", "v", "page_table", "length", "held", "ref_count",
                                          "free_list", "n_free", "status")]


@functools.cache
def _lib() -> C.CDLL:
    L = P.lib()
    vp, i, l, f, sz, cp = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t, C.POINTER(_Cache)
    L.prox_cache_init.argtypes = [cp, vp]
    L.prox_cache_workspace_bytes.argtypes = [cp]
    L.prox_cache_reserve.argtypes = [cp, i, vp, vp, vp, vp]
    L.prox_cache_append.argtypes = [cp, i, i, vp, vp, i, vp, l, vp, l, vp]
    L.prox_cache_fork.argtypes = [cp, i, vp, vp, i, vp, vp, sz, vp]
    L.prox_cache_compact.argtypes = [cp, i, vp, vp, i, vp, vp, vp]
    L.prox_cache_free.argtypes = [cp, i, vp, vp]
    L.prox_cache_status.argtypes = [cp, vp, C.POINTER(C.c_uint32)]
    L.prox_attention_workspace_bytes.argtypes = [cp, i, i]
    L.prox_tree_attention.argtypes = [cp, i, i, vp, vp, i, i, i, vp, l, vp, i, f, vp, l, vp, vp, sz,
                                      vp]
    L.prox_logprobs.argtypes = [i, i, i, vp, l, vp, i, i, vp, vp, vp, vp, vp]
    for name in ABI_FUNCTIONS:
        getattr(L, name).restype = sz if name.endswith("workspace_bytes") else C.c_int
    return L


_NONE = nullcontext()


def _on(dev: torch.device):
    """The context in which a call for tensors of `dev` is launched."""
    return _NONE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(dev: torch.device) -> int:
    """The current stream's handle (without building a torch.cuda.Stream)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _ints(t: torch.Tensor, shape: tuple, dev: torch.device, name: str, dtype=torch.int32) -> int:
    """Pointer of a contiguous device list, checked."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, heads: int, dim: int, dtype, dev: torch.device, name: str) -> tuple:
    """(pointer, row stride) of [rows][heads][dim] whose rows are contiguous."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[1] != heads or shape[2] != dim or \
            t.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor [rows][{heads}][{dim}] on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    s = t.stride()
    if s[2] != 1 or (s[1] != dim and heads > 1):
        raise ValueError(f"{name}: a row's heads must be contiguous, got strides {s}")
    return t.data_ptr(), s[0] if shape[0] > 1 else heads * dim


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

class PagedCache:
    """A paged key/value cache: its device tensors, in libprox's layouts.

    k, v bf16 or fp16 [n_layers][n_pages][n_kv_heads][page_size][head_dim];
    page_table int32 [max_seqs][max_pages]; length, held int32 [max_seqs];
    ref_count, free_list int32 [n_pages]; n_free int32 [1]. The tensors stay
    those the cache was made with; their contents are the cache's state."""

    def __init__(self, n_layers: int, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int,
                 max_seqs: int, max_pages: int, dtype=torch.bfloat16, device="cuda"):
        """An empty cache; k and v are not initialised."""
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        i32 = functools.partial(torch.zeros, dtype=torch.int32, device=dev)
        self._adopt(torch.empty(shape, dtype=dtype, device=dev),
                    torch.empty(shape, dtype=dtype, device=dev), i32((max_seqs, max_pages)),
                    i32(max_seqs), i32(max_seqs), i32(n_pages), i32(n_pages), i32(1))
        with _on(dev):
            P._check(_lib().prox_cache_init(self._ref, _stream(dev)), "prox_cache_init")

    @classmethod
    def from_tensors(cls, k, v, page_table, length, held, ref_count, free_list, n_free) -> "PagedCache":
        """A cache over tensors that hold its state already."""
        self = cls.__new__(cls)
        self._adopt(k, v, page_table, length, held, ref_count, free_list, n_free)
        return self

    def _adopt(self, k, v, page_table, length, held, ref_count, free_list, n_free):
        if k.dim() != 5 or page_table.dim() != 2:
            raise ValueError("k must be [n_layers][n_pages][n_kv_heads][page_size][head_dim], "
                             "page_table [max_seqs][max_pages]")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"k must be bfloat16 or float16, got {k.dtype}")
        layers, pages, heads, size, dim = k.shape
        seqs, cols = page_table.shape
        P._need(k, k.dtype, k.shape, "k")
        dev = k.device
        _ints(v, k.shape, dev, "v", k.dtype)
        for name, t, shape in (("page_table", page_table, (seqs, cols)), ("length", length, (seqs,)),
                               ("held", held, (seqs,)), ("ref_count", ref_count, (pages,)),
                               ("free_list", free_list, (pages,)), ("n_free", n_free, (1,))):
            _ints(t, shape, dev, name)
        self.k, self.v, self.page_table, self.length, self.held = k, v, page_table, length, held
        self.ref_count, self.free_list, self.n_free = ref_count, free_list, n_free
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.max_seqs, self.max_pages, self.dtype, self.device = seqs, cols, k.dtype, dev
        self._struct = _Cache(layers, pages, size, heads, dim, DTYPES[k.dtype], seqs, cols,
                              *(t.data_ptr() for t in (k, v, page_table, length, held, ref_count,
                                                       free_list, n_free, self.status)))
        self._ref = C.byref(self._struct)
        n = int(_lib().prox_cache_workspace_bytes(self._ref))
        if n == 0:
            raise ProxError(PROX_EINVAL, "prox_cache_workspace_bytes")
        self._ws = torch.empty(n, dtype=torch.uint8, device=dev)


def cache_reserve(cache: PagedCache, seqs: torch.Tensor, n_new: torch.Tensor,
                  ok: torch.Tensor | None = None) -> None:
    """prox_cache_reserve: pages for n_new[i] tokens behind the committed ones
    of sequence seqs[i] (int32 [n] each); ok uint8 [n] tells which got them (too few
    free pages refuse an entry and those behind it, too many columns it alone)."""
    n, dev = seqs.numel(), cache.device
    a = (n, _ints(seqs, (n,), dev, "seqs"), _ints(n_new, (n,), dev, "n_new"),
         None if ok is None else _ints(ok, (n,), dev, "ok", torch.uint8))
    with _on(dev):
        P._check(_lib().prox_cache_reserve(cache._ref, *a, _stream(dev)), "prox_cache_reserve")


def cache_append(cache: PagedCache, layer: int, seqs: torch.Tensor, cu_new: torch.Tensor,
                 k_new: torch.Tensor, v_new: torch.Tensor) -> None:
    """prox_cache_append: rows cu_new[i] .. cu_new[i+1] - 1 of k_new and v_new
    [rows][n_kv_heads][head_dim] behind the committed tokens of seqs[i], in one
    layer, on pages that cache_reserve has given the sequence."""
    n, dev = seqs.numel(), cache.device
    kp, ks = _rows(k_new, cache.n_kv_heads, cache.head_dim, cache.dtype, dev, "k_new")
    vp, vs = _rows(v_new, cache.n_kv_heads, cache.head_dim, cache.dtype, dev, "v_new")
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    a = (layer, n, _ints(seqs, (n,), dev, "seqs"), _ints(cu_new, (n + 1,), dev, "cu_new"),
         k_new.shape[0], kp, ks, vp, vs)
    with _on(dev):
        P._check(_lib().prox_cache_append(cache._ref, *a, _stream(dev)), "prox_cache_append")


def cache_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, *, share: bool = True,
               ok: torch.Tensor | None = None) -> None:
    """prox_cache_fork: empty sequences dst[i] become copies of src[i], sharing
    whole pages (share) or on pages of their own."""
    n, dev = src.numel(), cache.device
    a = (n, _ints(src, (n,), dev, "src"), _ints(dst, (n,), dev, "dst"), int(bool(share)),
         None if ok is None else _ints(ok, (n,), dev, "ok", torch.uint8), cache._ws.data_ptr(),
         cache._ws.numel())
    with _on(dev):
        P._check(_lib().prox_cache_fork(cache._ref, *a, _stream(dev)), "prox_cache_fork")


def cache_compact(cache: PagedCache, seqs: torch.Tensor, path: torch.Tensor, n_path: torch.Tensor,
                  ok: torch.Tensor | None = None) -> None:
    """prox_cache_compact: the drafted rows path[i][: n_path[i]] (ascending)
    become committed tokens of seqs[i]; path int32 [n][max_path]; ok uint8 [n] tells
    which paths were taken, each as a whole or not at all."""
    n, dev = seqs.numel(), cache.device
    if path.dim() != 2:
        raise ValueError("path must be [n][max_path]")
    a = (n, _ints(seqs, (n,), dev, "seqs"), _ints(path, (n, path.shape[1]), dev, "path"),
         path.shape[1], _ints(n_path, (n,), dev, "n_path"),
         None if ok is None else _ints(ok, (n,), dev, "ok", torch.uint8))
    with _on(dev):
        P._check(_lib().prox_cache_compact(cache._ref, *a, _stream(dev)), "prox_cache_compact")


def cache_free(cache: PagedCache, seqs: torch.Tensor) -> None:
    """prox_cache_free: gives back the pages of the listed sequences."""
    n, dev = seqs.numel(), cache.device
    p = _ints(seqs, (n,), dev, "seqs")
    with _on(dev):
        P._check(_lib().prox_cache_free(cache._ref, n, p, _stream(dev)), "prox_cache_free")


def cache_status(cache: PagedCache) -> tuple[int, int]:
    """(status, CACHE_* bits) of the cache's status word; clears the bits returned."""
    flags = C.c_uint32()
    with _on(cache.device):
        st = _lib().prox_cache_status(cache._ref, _stream(cache.device), C.byref(flags))
    return st, flags.value


# ---------------------------------------------------------------------------
# attention of drafted tokens
# ---------------------------------------------------------------------------

def attention_workspace(cache: PagedCache, max_q: int, n_heads: int) -> torch.Tensor:
    """Workspace of tree_attention for up to max_q rows a sequence and n_heads
    heads, any number of sequences; calls that overlap need one each."""
    with _on(cache.device):
        size = int(_lib().prox_attention_workspace_bytes(cache._ref, n_heads, max_q))
    if size == 0:
        raise ProxError(PROX_EINVAL, "prox_attention_workspace_bytes")
    return torch.empty(size, dtype=torch.uint8, device=cache.device)


def tree_attention(cache: PagedCache, layer: int, q: torch.Tensor, seqs: torch.Tensor,
                   cu_q: torch.Tensor, max_q: int, *, tree: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """prox_tree_attention: (out, lse) of drafted tokens q [rows][n_heads][head_dim]
    (rows cu_q[i] .. cu_q[i+1] - 1 belong to sequence seqs[i]) over one layer of
    the cache. tree int64 [rows][words] has the bits of the drafted tokens each
    row sees; None is a chain. scale defaults to head_dim ** -0.5. Rows behind
    the last sequence are left as they are in out and lse. out may be q."""
    # (outputs made here are not checked, and made from sizes given one by one: the
    # shortest calls take less time on the GPU than on the host)
    dev, dim = cache.device, cache.head_dim
    n, shape = seqs.numel(), q.shape
    heads = shape[1] if len(shape) == 3 else 0
    qp, qs = _rows(q, heads, dim, cache.dtype, dev, "q")
    rows = shape[0]
    if out is None:
        out = torch.empty(rows, heads, dim, dtype=cache.dtype, device=dev)
        op, os_ = out.data_ptr(), heads * dim
    elif out.shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out.shape)}")
    else:
        op, os_ = _rows(out, heads, dim, cache.dtype, dev, "out")
    if lse is None:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _ints(lse, (rows, heads), dev, "lse", torch.float32)
    if ws is None:
        ws = attention_workspace(cache, max_q, heads)
    size = ws.numel()
    words = 0
    if tree is not None:
        words = tree.shape[1] if tree.dim() == 2 else -1
        tree = _ints(tree, (rows, words), dev, "tree", torch.int64)
    a = (layer, n, _ints(seqs, (n,), dev, "seqs"), _ints(cu_q, (n + 1,), dev, "cu_q"), rows, max_q,
         heads, qp, qs, tree, words, dim ** -0.5 if scale is None else float(scale), op, os_, lp,
         _ints(ws, (size,), dev, "ws", torch.uint8), size)
    with _on(dev):
        P._check(_lib().prox_tree_attention(cache._ref, *a, _stream(dev)), "prox_tree_attention")
    return out, lse


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------

@dataclass
class LogprobsOut:
    logp: torch.Tensor | None         # fp32 [rows][n_tok]
    entropy: torch.Tensor             # fp32 [rows]
    top_ids: torch.Tensor | None      # int32 [rows][top_k]
    top_logp: torch.Tensor | None     # fp32 [rows][top_k]


def logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, *,
             top_k: int = 0) -> LogprobsOut:
    """prox_logprobs: log probabilities of tokens int32 [rows][n_tok] (or [rows])
    under softmax of logits [rows][vocab] (bf16, fp16 or fp32; rows may be
    strided), the rows' entropy, and their top_k alternatives."""
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dim() != 2 or logits.dtype not in DTYPES or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a bf16, fp16 or fp32 tensor [rows][vocab] with contiguous "
                         f"rows, got {logits.dtype} {tuple(logits.shape)} strides {logits.stride()}")
    rows, vocab = logits.shape
    dev = logits.device
    n_tok = 0
    if tokens is not None:
        if tokens.dim() == 1:
            tokens = tokens.unsqueeze(1)
        n_tok = tokens.shape[1] if tokens.dim() == 2 else -1
        tp = _ints(tokens, (rows, n_tok), dev, "tokens")
    f32, k = torch.float32, top_k > 0
    out = LogprobsOut(torch.empty(rows, n_tok, dtype=f32, device=dev) if n_tok else None,
                      torch.empty(rows, dtype=f32, device=dev),
                      torch.empty(rows, top_k, dtype=torch.int32, device=dev) if k else None,
                      torch.empty(rows, top_k, dtype=f32, device=dev) if k else None)
    a = (rows, vocab, DTYPES[logits.dtype], logits.data_ptr(),
         logits.stride(0) if rows > 1 else vocab, tp if n_tok else None, n_tok, top_k,
         P._ptr(out.logp), out.entropy.data_ptr(), P._ptr(out.top_ids), P._ptr(out.top_logp))
    with _on(dev):
        P._check(_lib().prox_logprobs(*a, _stream(dev)), "prox_logprobs")
    return out


__all__ = ["PagedCache", "cache_reserve", "cache_append", "cache_fork", "cache_compact",
           "cache_free", "cache_status", "attention_workspace", "tree_attention", "LogprobsOut",
           "logprobs", "CACHE_BAD_SEQ", "CACHE_FULL", "CACHE_BAD_STATE", "CACHE_BAD_ARG",
           "CACHE_TIMEOUT", "MAX_DRAFT", "MAX_TOP"]
