"""The expert operators at the edges of their definition: infinite ties, scores far below a
row's largest, saturated scores, rows that are no numbers, and results that must not depend on
the tokens beside them.

Tolerances as in test_gpu_experts.py."""
import math

import numpy as np
import pytest
import torch

import predictor_gated_channel_b200 as sfn
from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build
from test_gpu_experts import DEV, expert_weights, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfn_build.build()
    _capi.lib()


# ---------------------------------------------------------- experts' products
@pytest.mark.parametrize("T,E,k,d,f", [(300, 4, 2, 4096, 1792), (1500, 3, 2, 272, 208),
                                       (40, 16, 4, 400, 240), (700, 5, 2, 144, 4096)])
def test_experts_token_by_itself(T, E, k, d, f):
    """A token's bits are the same alone, among a few (streams) and among many
    (tiles, pairs): what follows the exact integer sums is the same arithmetic."""
    W = expert_weights(T, E, f, d)
    x = rand(T, T, d).to(torch.bfloat16).to(DEV)
    g = torch.Generator().manual_seed(T)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    experts[2, 0] = -1
    weights = torch.rand((T, k), generator=g).to(DEV)
    experts = experts.to(DEV)
    y = sfn.experts_i8_forward(x, experts, weights, **W)
    for first, n in ((0, 1), (1, 5), (T - 1, 1), (T // 2, 32 // k), (3, 37)):
        rows = slice(first, first + n)
        part = sfn.experts_i8_forward(x[rows].contiguous(), experts[rows].contiguous(),
                                      weights[rows].contiguous(), **W)
        assert torch.equal(part, y[rows]), (first, n)
