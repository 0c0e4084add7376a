"""Flags that have no truth value are refused alike by the compiled and by the Python functions, with nothing launched."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_fast_calls_gpu import python_only, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["interleaved", "return_lse"])
def test_flags_without_a_truth_value(monkeypatch, which):
    cache, q, k, v, slots, pos, cs = setup()
    table, ctx = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([9], dtype=torch.int32, device="cuda")
    flag = torch.ones(2)

    def call():
        if which == "interleaved":
            return mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=cs, interleaved=flag)
        return mbw.kv4_attention(cache, q, table, ctx, return_lse=flag)

    said = []
    for f in (call, lambda: python_only(monkeypatch, call)):
        n = mbw.launch_count()
        with pytest.raises(RuntimeError) as e:
            f()
        said.append((e.type, str(e.value)))
        assert mbw.launch_count() == n
    assert said[0] == said[1] and not isinstance(e.value, mbw.MbwError)
