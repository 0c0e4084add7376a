"""The package's names are its binding's, whenever they are looked at."""
import memory_bound_weight_gb300 as mbw
from memory_bound_weight_gb300 import _binding as B


def test_a_function_replaced_in_the_binding_is_seen(monkeypatch):
    for name in ("gemv_bf16", "kv4_attention", "check_device_error"):
        assert getattr(mbw, name) is getattr(B, name)
        other = object()
        with monkeypatch.context() as m:
            m.setattr(B, name, other)
            assert getattr(mbw, name) is other
        assert getattr(mbw, name) is getattr(B, name)
