"""A workspace that grows while a graph that uses it lives, and on another stream."""

import pytest
import torch

import matrix_optimizers_sharded_amd as mo
from test_gpu_operators import generator

pytestmark = pytest.mark.gpu


def test_a_larger_call_after_a_capture_leaves_the_graph_its_buffer(gpu):
    gen = generator(gpu, 41)
    n, vocab, dim = 9000, 3001, 72
    ws = mo.Workspace(gpu)
    tokens = torch.randint(0, vocab, (n,), generator=gen, device=gpu)
    g = torch.randn(n, dim, generator=gen, device=gpu)
    step = lambda: mo.embedding_grad(g, tokens, vocab, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    nbytes = ws.buf.numel()
    big = torch.randint(0, vocab, (8 * n,), generator=gen, device=gpu)
    mo.embedding_grad(torch.randn(8 * n, dim, generator=gen, device=gpu), big, vocab, workspace=ws)
    assert ws.buf.numel() > nbytes
    # whoever allocates the same size now must not get the graph's buffer
    others = [torch.full((nbytes,), 7, dtype=torch.uint8, device=gpu) for _ in range(4)]
    for r in range(3):
        tokens.copy_(torch.randint(0, vocab, (n,), generator=gen, device=gpu))
        want = mo.embedding_grad(g, tokens, vocab)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want), f"replay {r}"
        assert all(bool((o == 7).all()) for o in others), f"replay {r}"


def test_a_larger_call_on_another_stream(gpu):
    gen = generator(gpu, 43)
    vocab, dim = 3001, 72
    ws = mo.Workspace(gpu)
    calls = []
    for n in (9000, 50000, 200000):
        tokens = torch.randint(0, vocab, (n,), generator=gen, device=gpu)
        calls.append((torch.randn(n, dim, generator=gen, device=gpu), tokens))
    want = [mo.embedding_grad(g, t, vocab) for g, t in calls]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for (g, t), w in zip(calls, want):
        for stream in (main, side):
            side.wait_stream(main)
            main.wait_stream(side)
            with torch.cuda.stream(stream):
                got = mo.embedding_grad(g, t, vocab, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(got, w)
