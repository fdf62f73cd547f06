"""The operators of drafting and branching together, as a server uses them: the example's drafted decoding gives the
tokens of the plain one, in fewer passes, and leaves no page behind."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(prompt_tokens=16, samples=1, page=16, count=30, seed=1),
                                dict(prompt_tokens=3, samples=4, page=32, seed=2)])
def test_drafting_example(kw):
    from local_linear_attention_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("paged_drafting", os.path.join(ROOT, "examples", "paged_drafting.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    tokens, again, passes, held = example.serve(**kw)
    assert tokens == again and held == 0
    assert passes < len(tokens[0])  # most drafts hold the next token
