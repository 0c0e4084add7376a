"""token_logprobs over logits of large magnitude, as masks of finite numbers and unscaled scores have them, against the
definition in 64 bits. Tolerances as in test_logprobs_gpu.py."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_logprobs_gpu import compare

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("V", [40000, 152064])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", [-1e8, -1e10, -1e12, -1e30])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_masks_of_finite_numbers(V, dtype, mask, scale):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.full((6, V), mask, device="cuda")
    few = torch.randperm(V // 3, generator=g, device="cuda")[:40]
    x[1, V - 1 - few] = torch.randn(40, generator=g, device="cuda") * 3          # allowed in the last third alone
    x[2, few] = torch.randn(40, generator=g, device="cuda") * 3                  # in the first
    x[3, V // 2] = 2.5                                                           # one
    x[4] = torch.randn(V, generator=g, device="cuda") * 3
    x[4, ::5] = mask
    x[5, ::2] = -INF                                                             # two kinds of mask
    x = x.to(dtype)
    for t in (0, V - 1 - int(few[0]), V // 2):
        tt = torch.full((6,), t, dtype=torch.int32, device="cuda")
        for ws in (None, mbw.token_logprobs_workspace()):
            compare(x, tt, 32, scale, ws)


@pytest.mark.parametrize("V", [300, 40000, 152064])
@pytest.mark.parametrize("big", [2.0 ** 20, 5e7, 2e8, 1e10, -5e7, -2e8, -1e10, 1e20])
def test_logits_near_a_large_number(V, big):
    """The numbers next to one, ties among them, and minus infinities."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    at = torch.tensor(big, dtype=torch.float32).view(torch.int32).item()
    near = torch.randint(-6, 7, (4, V), generator=g, device="cuda") + at
    x = near.to(torch.int32).view(torch.float32).clone()
    x[1, ::3] = -INF
    x[2] = x[2, :1]
    x[3, :V // 2] = big - abs(big) * 0.5
    t = torch.tensor([0, 1, V - 1, V // 2], dtype=torch.int32, device="cuda")
    for ws in (None, mbw.token_logprobs_workspace()):
        compare(x, t, 20, 1.0, ws)
        compare(x.bfloat16(), t, 20, 1.0, ws)


@pytest.mark.parametrize("V", [3, 2000, 40000, 152064])
@pytest.mark.parametrize("far", [1e2, 1e3, -1e4, 1e5, -1e6, 1e7, -5e7, 3e8])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logits_spread_around_a_far_number(V, far, scale):
    """The reference moves many times on the way: rising rows, and rows in no order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V + 1)
    x = torch.randn(24, V, generator=g, device="cuda") * 3 + far
    x[:8] = x[:8].sort(-1).values
    t = torch.randint(V, (24,), generator=g, device="cuda").int()
    for ws in (None, mbw.token_logprobs_workspace()):
        compare(x, t, 5, scale, ws)
