"""The decode loop of examples/decode_step.py: a shared prompt gives what private copies of it give."""
import importlib.util
import os

import pytest

from conftest import ROOT
from serve_ref import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_shared_and_private_prompts_agree(example):
    t = torch()
    model = example.Model()
    prompt = t.randint(0, 4099, (77,), generator=t.Generator().manual_seed(3)).cuda()
    shared, logits, lp = example.generate(model, prompt, sequences=5, steps=4)
    again, _, lp2 = example.generate(model, prompt, sequences=5, steps=4)
    assert t.equal(shared, again) and t.equal(lp, lp2)  # the same numbers draw the same tokens
    assert t.all((shared >= 0) & (shared < 4099)) and t.all(lp < 0)
    private, plogits, _ = example.generate(model, prompt, sequences=5, steps=4, private=True)
    # The prompt's logits: the same products in other tiles, bf16 roundings on the way.
    assert (logits - plogits).norm() <= 0.05 * logits.norm()
    # The first token comes from those logits; the draw is the same number.
    assert t.equal(shared[:, 0], private[:, 0])
