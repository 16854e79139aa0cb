"""Results of the orthogonalised update between each other's rows, in place and not."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from test_orthogonalize_gpu import DTYPES, gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


# heads, rows, columns of a head: in one launch, in strips, in three products a step
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [(6, 50, 40), (8, 128, 256), (12, 300, 130), (3, 256, 20)],
                         ids=lambda s: "x".join(map(str, s)))
def test_heads_of_one_weight(size, dtype):
    heads, d, width = size
    say("orthogonalize heads", size, dtype)
    w = torch.randn(d, heads * width, generator=gen(d), device="cuda").to(DTYPES[dtype])
    for whole in (w, w.t().contiguous().t(), torch.cat((w, w[:, :5]), 1)[:, :-5]):
        view = whole.view(d, heads, width) if whole.is_contiguous() else whole.unflatten(1, (heads, width))
        stack = view.transpose(0, 1)
        want = torch.stack([dg.orthogonalize(h.contiguous()) for h in stack])
        out = torch.full((d + 2, heads * width), 7.0, device="cuda", dtype=DTYPES[dtype])
        dg.orthogonalize(stack, out=out[1:-1].view(d, heads, width).transpose(0, 1))
        assert torch.equal(out[1:-1].view(d, heads, width).transpose(0, 1), want)
        assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
        for _ in range(2):   # a call of this form again
            again = whole.clone(memory_format=torch.preserve_format)
            place = again.unflatten(1, (heads, width)).transpose(0, 1)
            assert dg.orthogonalize(place, out=place) is place
            assert torch.equal(place, want)


def test_results_that_share_elements_are_refused():
    g = torch.randn(4, 20, 30, device="cuda")
    flat = torch.full((5000,), 7.0, device="cuda")
    for strides in ((599, 30, 1), (0, 30, 1), (29, 120, 1), (15, 60, 1), (1, 30, 1)):
        with pytest.raises(ValueError, match="overlap"):
            dg.orthogonalize(g, out=flat.as_strided((4, 20, 30), strides))
    assert bool((flat == 7).all())
