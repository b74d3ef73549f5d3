"""The residual blocks' operators where their numbers or their callers come to an end: choices that
one list of the router holds alone."""

import pytest
import torch

from test_gpu_block_ops import DEV, _built, check_route  # noqa: F401
from test_gpu_model_ops import gen

pytestmark = pytest.mark.gpu


# ---- the router's choice ---------------------------------------------------------------

def lanes(experts):
    """Lanes that share a token's logits: each has every so many-th run of eight."""
    return next(n for most, n in ((8, 1), (16, 2), (32, 4), (64, 8), (128, 8), (256, 16),
                                  (1024, 32)) if experts <= most)


@pytest.mark.parametrize("experts", [64, 72, 128, 129, 160, 256, 300, 384, 512, 520, 1024])
@pytest.mark.parametrize("spread", ["ulp", "same", "wide"])
def test_the_largest_logits_with_one_lane(experts, spread):
    """The nine (or more) largest logits of a token lie with one lane; the eighth and the ninth are
    one step of FP32 apart, either way round, or equal, or far apart."""
    g = gen(experts)
    tokens, width = 96, lanes(experts)
    logits = -4.0 - torch.rand(tokens, experts, device=DEV, generator=g)
    for t in range(tokens):
        part = t % width
        mine = [e for e in range(experts) if e // 8 % width == part]
        order = torch.randperm(len(mine), generator=torch.Generator().manual_seed(t)).tolist()
        mine = [mine[i] for i in order][:9 + t % 3]
        if t % 4 == 0:  # the first run of the lane and the first expert of the next
            mine = sorted(e for e in range(experts) if e // 8 % width == part)[:9]
        for place, e in enumerate(mine):
            logits[t, e] = 9.0 - place if place < 7 else 1.0
        if len(mine) > 8:
            step = {"ulp": 2.0 ** -23, "same": 0.0, "wide": 0.25}[spread]
            logits[t, mine[7 + t // 4 % 2]] += step
    check_route(logits, 8)
    check_route(logits, 7)
