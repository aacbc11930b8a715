"""Token log probabilities, entropy and top alternatives against the
definition in 64 bits."""
import math

import pytest
import torch

from decode_helpers import check_logprobs
from free_ffn_activation_b200 import decode as D
from free_ffn_activation_b200 import prox as P

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def logits(dev, rows, vocab, dtype, seed=0, spread=3.0, pad=0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return (torch.randn((rows, vocab + pad), device=dev, generator=gen) * spread).to(dtype)[:, :vocab]


def run(x, n_tok=2, top_k=0, seed=0):
    gen = torch.Generator(device=x.device)
    gen.manual_seed(seed)
    t = torch.randint(0, x.shape[1], (x.shape[0], n_tok), device=x.device, generator=gen).int()
    got = D.logprobs(x, t, top_k=min(top_k, x.shape[1]))
    torch.cuda.synchronize()
    check_logprobs(x, t, min(top_k, x.shape[1]), got)
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 64, 255, 1000, 4095, 4097, 16384, 32000, 50257])
def test_vocabularies(gpu, dtype, vocab):
    for rows in (1, 5):
        run(logits(gpu, rows, vocab, dtype, vocab), top_k=20)


@pytest.mark.parametrize("rows", [1, 2, 9, 37, 74, 75, 148, 149, 600])
def test_rows_per_cluster(gpu, rows):
    run(logits(gpu, rows, 32064, torch.bfloat16, rows), top_k=5)
    run(logits(gpu, rows, 5003, torch.float32, rows), top_k=0)


@pytest.mark.parametrize("top_k", [0, 1, 2, 16, 17, 20, 33, 63, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_alternatives(gpu, top_k, dtype):
    run(logits(gpu, 3, 40001, dtype, top_k), top_k=top_k)
    run(logits(gpu, 300, 3001, dtype, top_k), top_k=top_k)


# CTAs of 256 threads for many rows or short ones, of 512 for few long ones
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1300, 40001), (40, 40001), (3, 150001), (1300, 700)])
def test_rows_of_every_kind_in_wide_and_narrow_blocks(gpu, rows, vocab, dtype):
    x = logits(gpu, rows, vocab, dtype, vocab, pad=5)
    up = torch.linspace(-9, 9, vocab, device=gpu).to(dtype)
    x[0] = up                       # more candidates than there is room for
    x[1] = up.flip(0)
    x[2] = 1.5                      # equal values
    run(x, top_k=64)
    run(x, top_k=1)
    x[0, :vocab // 2] = -math.inf
    x[1] = -math.inf
    x[2, 7] = math.inf if dtype is torch.float32 else torch.finfo(dtype).max
    x[-1, vocab // 3:] = torch.finfo(dtype).min
    run(x, top_k=20)
    run(x, n_tok=700, top_k=0)


def test_equal_values_go_by_index(gpu):
    for vocab in (100, 5000, 60000):
        x = torch.zeros((2, vocab), device=gpu, dtype=torch.bfloat16)
        x[1] = torch.arange(vocab, device=gpu) % 3           # thousands of equal maxima
        x[0, 1::2] = -0.0                                    # equal to 0
        run(x, top_k=64)


def test_row_ends_of_equal_values_are_not_lost(gpu):
    """The elements before the first and behind the last whole vector count
    even when every element of the row is a candidate."""
    for dtype in TYPES:
        x = torch.ones((3000, 9001), device=gpu, dtype=dtype)
        for _ in range(5):
            got = D.logprobs(x, top_k=9)
            assert (got.top_ids == torch.arange(9, device=gpu)).all()
        x[:, -3:] = 2.0
        got = D.logprobs(x, top_k=5)
        assert (got.top_ids == torch.tensor([8998, 8999, 9000, 0, 1], device=gpu)).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_orders_that_fill_the_candidates(gpu, dtype):
    """Ascending rows make every element a candidate when it is met."""
    up = torch.arange(30000, device=gpu, dtype=torch.float32)
    x = torch.stack([up / 3000, -up / 3000, (up * 7919 % 30000) / 1000]).to(dtype)
    run(x, top_k=64)


@pytest.mark.parametrize("dtype", TYPES)
def test_masks_and_lowest_values(gpu, dtype):
    low = torch.finfo(dtype).min
    x = logits(gpu, 9, 3001, dtype)
    x[0, 5:] = -math.inf
    x[1, 5:] = low
    x[2] = -math.inf                 # nothing left
    x[3] = low                       # all equal: uniform
    x[4, :] = -math.inf
    x[4, 3000] = 2.0                 # one left
    x[5, :3000] = -math.inf
    x[6, 0] = torch.finfo(dtype).max
    x[7, ::2] = -math.inf
    for top_k in (0, 8):
        got = run(x, top_k=top_k)
        assert (got.logp[2] == -math.inf).all() and got.entropy[2] == 0
        assert abs(float(got.entropy[3]) - math.log(3001)) < 1e-5
        assert got.entropy[4] == 0


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_infinity(gpu, value, dtype):
    for vocab in (3001, 40000):
        x = logits(gpu, 4, vocab, dtype)
        x[1, vocab // 2] = value
        x[2, :7] = value
        for top_k in (0, 10):
            got = run(x, top_k=top_k)
            assert torch.isnan(got.entropy[1:3]).all() and torch.isfinite(got.entropy[[0, 3]]).all()


def test_far_apart_values(gpu):
    for spread in (1e-3, 1.0, 30.0, 1e4, 1e37):
        run(logits(gpu, 4, 20000, torch.float32, spread=spread), top_k=4)


def test_row_starts_of_any_alignment(gpu):
    for dtype in TYPES:
        wide = logits(gpu, 6, 9000, dtype)
        for off in range(9):
            run(wide[:, off:off + 8191 - off], top_k=6, n_tok=3)
        run(wide[1:4:2, 3:], top_k=6)
        run(wide[:1, 1:], top_k=6)


def test_tokens(gpu):
    x = logits(gpu, 3, 1000, torch.bfloat16)
    t = torch.tensor([[0, 999, -1, 1000], [5, 5, 2**31 - 1, -2**31], [999, 0, 1, 2]], device=gpu, dtype=torch.int32)
    got = D.logprobs(x, t, top_k=3)
    torch.cuda.synchronize()
    check_logprobs(x, t, 3, got)
    many = torch.randint(0, 1000, (3, 1024), device=gpu).int()
    check_logprobs(x, many, 0, D.logprobs(x, many))
    none = D.logprobs(x)
    assert none.logp is None and none.top_ids is None and torch.equal(none.entropy, got.entropy)
    flat = D.logprobs(x, t[:, 0].contiguous())
    assert torch.equal(flat.logp, got.logp[:, :1])
    assert D.logprobs(x[:0], t[:0]).entropy.shape == (0,)


def test_offsets_past_32_bits(gpu):
    rows, vocab = 36000, 65001           # 2.3e9 elements
    x = torch.empty((rows, vocab), dtype=torch.bfloat16, device=gpu)
    x.fill_(1.0)
    x[-1] = logits(gpu, 1, vocab, torch.bfloat16)[0]
    t = torch.full((rows, 1), 3, dtype=torch.int32, device=gpu)
    got = D.logprobs(x, t, top_k=2)
    torch.cuda.synchronize()
    last = D.LogprobsOut(got.logp[-1:], got.entropy[-1:], got.top_ids[-1:], got.top_logp[-1:])
    check_logprobs(x[-1:], t[-1:], 2, last)
    assert (got.logp[:-1] + math.log(vocab)).abs().max() < 1e-5
    assert (got.top_ids[:-1] == torch.tensor([0, 1], device=gpu)).all()


def test_same_bits_every_time_and_in_a_graph(gpu):
    x = logits(gpu, 20, 50000, torch.bfloat16)
    t = torch.zeros((20, 1), dtype=torch.int32, device=gpu)
    a = D.logprobs(x, t, top_k=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = D.logprobs(x, t, top_k=10)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = D.logprobs(x, t, top_k=10)
    g.replay()
    torch.cuda.synchronize()
    for o in (b, c):
        assert all(torch.equal(getattr(a, f), getattr(o, f)) for f in ("logp", "entropy", "top_ids", "top_logp"))
    x.copy_(logits(gpu, 20, 50000, torch.bfloat16, seed=4))
    g.replay()
    torch.cuda.synchronize()
    check_logprobs(x, t, 10, c)


def test_binding_refuses_wrong_tensors(gpu):
    x = logits(gpu, 3, 100, torch.float32)
    t = torch.zeros((3, 1), dtype=torch.int32, device=gpu)
    for bad in (x.double(), x[0], x.t(), x[:, ::2]):
        with pytest.raises(ValueError):
            D.logprobs(bad)
    for bad in (t.long(), t[:2], t.cpu(), t.view(1, 3)):
        with pytest.raises(ValueError):
            D.logprobs(x, bad)
    for k in (-1, 65, 101):
        with pytest.raises(P.ProxError):
            D.logprobs(x, t, top_k=k)
