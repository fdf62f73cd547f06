"""The serving example runs the paged operators together: chunked prompts equal to the contiguous
forward (both round their output to bf16, half a step each, and their weights), decode with weight
tracking, eviction at the limit."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_serving_example():
    from local_linear_attention_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, lengths = example.serve()
    assert worst <= 4 * 2.0 ** -8
    # 700 + 1 passes the limit of 512 at the first step (384 left, 39 more); 90 and 300 never do
    assert lengths == [384 + 39, 90 + 40, 300 + 40]
