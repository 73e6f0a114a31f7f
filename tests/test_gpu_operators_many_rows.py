"""More rows than one launch can hold: 2^32 threads or more in a grid wrap, and only the
remainder would run, without an error."""

import pytest
import torch

import matrix_optimizers_sharded_amd as mo
from gpu_util import say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def release(gpu):
    yield
    torch.cuda.empty_cache()


def test_lookup(gpu):
    n = (1 << 26) + 77
    say(f"embedding_lookup of {n} rows")
    tokens = (torch.arange(n, dtype=torch.int32, device=gpu) % 1009) - 1
    table = torch.arange(1, 1008, device=gpu, dtype=F32)[:, None].contiguous()
    out = torch.full((n, 1), -1.0, device=gpu)
    mo.embedding_lookup(table, tokens, out=out)
    # token -1 and token 1007 (outside the table) give zeros
    assert torch.equal(out[:, 0], torch.where(tokens < 1007, tokens + 1, 0).to(F32))


def test_distill(gpu):
    n, half = (1 << 26) + 77, 1 << 25
    say(f"distill of {n} rows")
    gen = torch.Generator(device=gpu)
    gen.manual_seed(1)
    x = torch.randn(n, 2, generator=gen, device=gpu, dtype=F32).to(BF16)
    ids = (torch.arange(n, dtype=torch.int32, device=gpu) % 3)[:, None].contiguous()
    t, rg = torch.zeros(n, 1, device=gpu), torch.ones(n, device=gpu)
    loss, lse, grad = mo.distill_forward_backward(x, ids, t, rg)
    back = mo.distill_backward(x, lse, ids, t, rg)
    for lo in range(0, n, half):
        r = slice(lo, min(n, lo + half))
        want = mo.distill_forward_backward(x[r], ids[r], t[r], rg[r])
        for got, w in zip((loss, lse, grad), want):
            assert torch.equal(got[r], w)
        assert torch.equal(back[r], mo.distill_backward(x[r], want[1], ids[r], t[r], rg[r]))


def test_embedding_gradient(gpu):
    """Tokens in an order that visits every id alike: the gradient counts the visits."""
    vocab, extra = 1 << 26, 4096 + 77
    n = (1 << 30) + extra
    say(f"embedding_grad of {n} rows")
    tokens = torch.empty(n, dtype=torch.int32, device=gpu)
    for lo in range(0, n, 1 << 28):
        i = torch.arange(lo, min(n, lo + (1 << 28)), device=gpu)
        tokens[lo:lo + (1 << 28)] = ((i * 40503 + 7) % vocab).to(torch.int32)
    del i
    grad = mo.embedding_grad(torch.ones(n, 1, dtype=BF16, device=gpu), tokens, vocab, grad_dtype=F32)
    want = torch.full((vocab,), float(1 << 4), device=gpu)      # 40503 is odd: whole rounds of all ids
    want[tokens[n - extra:].long()] += 1
    assert torch.equal(grad[:, 0], want)


def test_expert_product(gpu):
    n = (1 << 30) + 77
    say(f"expert_matmul of {n} rows")
    x = torch.empty(n, 1, dtype=BF16, device=gpu)
    x[:, 0] = torch.arange(256, device=gpu).to(BF16).repeat((n + 255) // 256)[:n]
    w = torch.tensor([2.0, -1.0], device=gpu).to(BF16).view(2, 1, 1)
    off = torch.tensor([3, 1 << 29, n - 5], dtype=torch.int32, device=gpu)
    y = mo.expert_matmul(x, w, off)
    assert not y[:3].any() and not y[n - 5:].any()
    assert torch.equal(y[3:1 << 29], x[3:1 << 29] * 2)
    assert torch.equal(y[1 << 29:n - 5], -x[1 << 29:n - 5])
