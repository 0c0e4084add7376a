"""kv4_append of values at and beyond the ends of fp16: what fits is held, and a group with a value that does not reads as
NaN, in whatever place and of either sign, in K and in V."""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import new_cache, ulp_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("other", [0.0, -65280.0, 65280.0])
def test_values_at_the_ends_of_fp16(d, group, other):
    """The largest bf16 value within fp16 is 65280, the next one 65536."""
    values = [65280.0, -65280.0, 65536.0, -65536.0, 1e5, 5e5, -1e5, 982000.0, 3e38]
    x = torch.full((len(values), 1, d), other, device="cuda")
    x[torch.arange(len(values)), 0, torch.arange(len(values)) % group] = torch.tensor(values, device="cuda")
    x = x.bfloat16()
    cache = new_cache(1, 16, 1, d, group)
    slots = torch.arange(len(values), device="cuda")
    mbw.kv4_append(cache, x, x, slots)
    n, s, m = ref.quantize(x, group)
    want = n * s + m
    for got in mbw.kv4_gather(cache, slots):
        got = ref.f64(got)
        assert got[2:, :, :group].isnan().all() and not got[:2].isnan().any() and not got[:, :, group:].isnan().any()
        fit = want[:2]
        assert ((got[:2] - fit).abs() <= ulp_bf16(fit) * (1 + 2.0 ** -10)).all()
        assert ((got[2:, :, group:] - other).abs() <= abs(other) * 2.0 ** -8).all()
