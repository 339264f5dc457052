"""score() of examples/decode_step.py writes only the pages that it is given, and refuses texts that do not fit."""
import pytest

from serve_ref import torch
from test_gpu_dense_step import example, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mx", [False, True])
def test_scoring_between_decode_steps_leaves_their_pages(example, mx):
    t = torch()
    model = example.Model(mx=mx)
    text = t.randint(0, 4099, (45,), generator=t.Generator().manual_seed(3)).cuda()
    alone = example.score(model, text, top=4)
    example.generate(model, text, sequences=3, steps=2)
    caches = [c for layer in model.layers for c in (layer.cache.k, layer.cache.v)]
    before = [c.clone() for c in caches]
    s = example.score(model, text, top=4, pages=[400, 17, 399])
    assert all(t.equal(s[k], alone[k]) for k in s)
    kept = t.ones(model.pages, dtype=t.bool, device="cuda")
    kept[t.tensor([400, 17, 399]).cuda()] = False
    for c, b in zip(caches, before):
        assert t.equal(c[kept], b[kept]) and not t.equal(c, b)


def test_texts_that_do_not_fit_are_refused(example):
    t = torch()
    model = example.Model(layers=1, pages=4, positions=60)
    text = t.arange(70, device="cuda")
    for bad, pages in ((text[:0], None), (text[:1], None), (text[:65], None), (text[:61], None), (text[:17], [1]),
                       (text[:17], [1, 1]), (text[:17], [1, 4]), (text[:17], [-1, 2])):
        with pytest.raises(ValueError):
            example.score(model, bad, pages=pages)
    assert example.score(model, text[:60])["rank"].shape == (59,)
    assert example.score(model, text[:17], pages=[3, 0, 1])["rank"].shape == (16,)
    assert int(model.status.item()) == 0
