"""Calls of the 8-bit layers from several threads at once, of forms known and new, each on
a stream of its own."""
import threading

import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from test_i8_gpu import codes, gen, need_gpu, powers, product, quantized  # noqa: F401

pytestmark = pytest.mark.gpu


def test_threads():
    g = gen(12)
    cases = []
    for i in range(4):
        M, N, K = 1 + 40 * i, 24 + 8 * i, 80 + 16 * i
        x, w, sx, sw = codes(g, M, K), codes(g, N, K), powers(g, M), powers(g, N)
        cases.append((x, w, sx, sw, (product(x, w.t()) * sx.double()[:, None] * sw.double()).float(),
                      torch.randn(M, K, generator=g, device="cuda")))
    wanted = [quantized(c[5]) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        x, w, sx, sw, want, v = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for turn in range(200):
                rows = 1 + turn % x.shape[0]      # forms come and go
                y = dg.linear_i8(x[:rows], sx[:rows], w.t(), sw, out_dtype=torch.float32)
                q, s = dg.quantize_i8(v)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(y, want[:rows]) and torch.equal(q, wanted[i][0]) and torch.equal(s, wanted[i][1])):
                    wrong.append((i, turn))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
