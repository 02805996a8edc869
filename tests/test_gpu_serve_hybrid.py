"""The example of a served hybrid: prompt and decode agree, forked rows go on
like their parents, and a compaction changes nothing."""
import os
import sys

import pytest
import torch

import gated_delta_rule_41_gb300 as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_served_hybrid(cache):
    import serve_hybrid

    g = torch.Generator().manual_seed(3)
    prompt = torch.randint(0, 1000, (130,), generator=g).tolist()
    whole = serve_hybrid.Hybrid(cache=cache)
    want = whole.prompts([4], [prompt])[0]
    m = serve_hybrid.Hybrid(cache=cache)
    m.prompts([2, 0], [prompt[:-1], prompt[:50]])
    m.fork([2], [9])
    ids = torch.full((m.rows,), prompt[-1], device="cuda")
    logits = m.step(ids)
    # two orders of the same sums in bf16, eight layers deep; a wrong row or page
    # gives logits that are not related
    for row in (2, 9):
        assert torch.nn.functional.cosine_similarity(logits[row], want, dim=0) > 0.995
    assert torch.equal(logits[2], logits[9])
    kda.check()
    # release a row and compact: the others go on as without it
    twin = serve_hybrid.Hybrid(cache=cache)
    twin.prompts([2, 0], [prompt[:-1], prompt[:50]])
    twin.fork([2], [9])
    twin.step(ids)
    m.release([0])
    a, b = m.step(ids), twin.step(ids)
    assert torch.equal(a[2], b[2]) and torch.equal(a[9], b[9])
    held = int((m.refs > 0).sum())
    assert (m.refs[:held] > 0).all() and m.lens.tolist()[0] == 0
    kda.check()


def test_example_runs():
    import serve_hybrid

    serve_hybrid.main(["--steps", "4"])
    serve_hybrid.main(["--steps", "4", "--cache", "e4m3"])
