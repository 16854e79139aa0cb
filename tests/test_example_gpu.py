"""The feed-forward example runs and its results are those of 64-bit torch
operations up to the roundings of its steps."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("features,inner,tokens", [(264, 520, 300), (100, 230, 17)])
def test_feed_forward_example(features, inner, tokens):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # along any path from x to a result fewer than eight values are rounded to
    # bfloat16, each off by at most 2^-8 of itself
    assert example.main([f"--features={features}", f"--inner={inner}", f"--tokens={tokens}"]) < 8 * 2.0 ** -8
