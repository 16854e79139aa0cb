"""Calls of the orthogonalised update that differ in eps and scale alone, as those of a
schedule do: one form, no other form lost, each call with its own."""
import threading

import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import layers
from helpers import say
from test_orthogonalize_gpu import gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [(40, 60), (128, 256), (300, 200)], ids=lambda s: "x".join(map(str, s)))
def test_a_schedule_of_scales(size):
    say("orthogonalize schedule", size)
    g = torch.randn(size, generator=gen(1), device="cuda")
    one = dg.orthogonalize(g)
    kept = set(layers._FORMS)
    for i in range(layers._MAX_FORMS + 10):
        out = dg.orthogonalize(g, scale=2.0 ** -(i % 50))
        if i < 50:
            assert torch.equal(out, one * 2.0 ** -i)
    assert set(layers._FORMS) == kept
    # |g| is about sqrt(M N): eps of |g| halves X
    assert not torch.equal(dg.orthogonalize(g, eps=float(g.norm())), one)
    assert torch.equal(dg.orthogonalize(g, eps=1e-7), one)
    assert bool((torch.signbit(dg.orthogonalize(g, scale=-0.0)) != torch.signbit(dg.orthogonalize(g, scale=0.0))).all())


def test_eps_and_scale_are_checked_in_every_call():
    g = torch.randn(300, 200, generator=gen(2), device="cuda")
    one = dg.orthogonalize(g)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(scale=1e-37), dict(scale=1e300)):
        with pytest.raises(dg.GemmError):
            dg.orthogonalize(g, **bad)
    assert torch.equal(dg.orthogonalize(g), one)


def test_threads_with_scales_of_their_own():
    g = torch.randn(300, 200, generator=gen(3), device="cuda")
    one = dg.orthogonalize(g)
    torch.cuda.synchronize()
    wrong = []

    def work(scale):
        stream = torch.cuda.Stream()
        for _ in range(100):
            out = dg.orthogonalize(g, scale=scale, stream=stream)
            stream.synchronize()
            if not torch.equal(out, one * scale):
                wrong.append(scale)
    threads = [threading.Thread(target=work, args=(2.0 ** i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_captured_calls_keep_their_scale():
    g = torch.randn(128, 256, generator=gen(4), device="cuda")
    dg.orthogonalize(g)
    graphs, outs = [], []
    for scale in (0.5, 4.0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dg.orthogonalize(g, scale=scale))
        graphs.append(graph)
    for seed in range(3):
        g.copy_(torch.randn(128, 256, generator=gen(10 + seed), device="cuda"))
        want = dg.orthogonalize(g, scale=-1.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want * -0.5) and torch.equal(outs[1], want * -4.0)
