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


def test_one_that_is_deleted_or_set_in_the_package_itself(monkeypatch):
    keep = mbw.gemv_bf16
    with monkeypatch.context() as m:
        m.delattr(B, "gemv_bf16")
        assert not hasattr(mbw, "gemv_bf16")
    assert mbw.gemv_bf16 is keep
    mine = object()
    monkeypatch.setattr(mbw, "gemv_bf16", mine)  # the package's own stays when the binding's changes
    with monkeypatch.context() as m:
        m.setattr(B, "gemv_bf16", object())
        assert mbw.gemv_bf16 is mine
