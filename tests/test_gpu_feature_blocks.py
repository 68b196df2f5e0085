"""The example that runs the lookup, the row groups, the norms, the products and the gates together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def blocks(htl):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import feature_blocks
    return feature_blocks


def test_trains_and_serves(blocks):
    gen = torch.Generator(device="cuda").manual_seed(0)
    tables, samples = 5, 600
    keys = torch.randint(0, 40, (samples, tables), device="cuda", generator=gen) | (torch.arange(tables, device="cuda") << 48)
    labels = (keys[:, 0] % 2 == 0).float()
    model = blocks.FeatureBlocks(tables, 64, capacity_log2=12)
    before = model.score(keys)
    first, logits = model.step(keys, labels)
    # keeping activations in 8 bits changes nothing in the forward pass
    assert torch.equal(logits, before)
    for _ in range(60):
        loss, _ = model.step(keys, labels)
    # half the samples each way: what a model that learnt nothing keeps is log 2 = 0.69 and above
    assert torch.isfinite(loss) and float(loss) < 0.35 < float(first)
    right = ((model.score(keys) > 0) == (labels > 0)).float().mean()
    assert float(right) > 0.9
    # one request
    assert torch.allclose(model.score(keys[:1]), model.score(keys)[:1], rtol=1e-4, atol=1e-4)


def test_same_step_twice_gives_the_same_bits(blocks):
    gen = torch.Generator(device="cuda").manual_seed(1)
    keys = torch.randint(0, 300, (1000, 7), device="cuda", generator=gen) | (torch.arange(7, device="cuda") << 48)
    labels = (keys[:, 1] % 2 == 0).float()
    a, b = (blocks.FeatureBlocks(7, 40, capacity_log2=14) for _ in range(2))
    (_, la), (_, lb) = a.step(keys, labels), b.step(keys, labels)
    assert torch.equal(la, lb)
    # the plan, norms, products and their gradients do not depend on the order of workgroups
    for p, q in zip(a.before + a.after + [a.wz, a.wu], b.before + b.after + [b.wz, b.wu]):
        assert torch.equal(p, q) and torch.isfinite(p).all()
