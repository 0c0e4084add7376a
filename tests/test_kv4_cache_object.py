"""A Kv4Cache stays what it was made over: no call hands the library an address or sizes that are not its tensor's."""
import copy

import pytest

torch = pytest.importorskip("torch")

import memory_bound_weight_gb300 as mbw  # noqa: E402
from test_kv4_host import calls, host, host_cache  # noqa: E402,F401


def every_call(c, make):
    i32, i64 = torch.int32, torch.int64
    k, q = make(5, 2, 128), make(5, 4, 128)
    return [lambda: mbw.kv4_append(c, k, k, make(5, dtype=i64)), lambda: mbw.kv4_gather(c, make(5, dtype=i64)),
            lambda: mbw.kv4_attention(c, q, make(5, 3, dtype=i32), make(5, dtype=i32))]


@pytest.mark.parametrize("name", ["pages", "kv_heads", "head_dim", "page_size", "group", "other"])
def test_its_attributes_cannot_be_set(calls, name):  # noqa: F811
    c = host_cache()
    with pytest.raises(AttributeError):
        setattr(c, name, host(9, c.pages.shape[1], dtype=torch.uint8) if name == "pages" else 4)
    with pytest.raises(AttributeError):
        delattr(c, name)
    assert c.pages.shape[0] == 3 and (c.kv_heads, c.head_dim, c.page_size, c.group) == (2, 128, 16, 64)
    for call in every_call(c, host):
        call()
    assert len(calls) == 3


@pytest.mark.parametrize("change", ["another", "larger", "smaller"])
def test_pages_that_moved_are_refused(calls, change):  # noqa: F811
    c = host_cache()
    n = c.pages.shape[1]
    keep = c.pages.untyped_storage()  # so that the allocator does not give the same memory again
    if change == "another":
        c.pages.data = torch.zeros(3, n, dtype=torch.uint8)
    elif change == "larger":
        c.pages.resize_(3000, n)
    else:
        c.pages.resize_(2, n)
    for call in every_call(c, host):
        with pytest.raises(ValueError, match="pages were moved or resized"):
            call()
    assert calls == [] and keep is not None


def test_a_copy_is_refused_not_made_over_another_caches_struct(calls):  # noqa: F811
    with pytest.raises(Exception):
        copy.copy(host_cache())


@pytest.mark.gpu
def test_pages_that_moved_are_refused_by_the_compiled_calls():
    def make(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    n = mbw.kv4_page_bytes(16, 2, 128)
    for change in ("another", "larger", "smaller"):
        c = mbw.Kv4Cache(make(3, n, dtype=torch.uint8), 2, 128)
        for call in every_call(c, make):
            call()
        keep = c.pages.untyped_storage()
        if change == "another":
            c.pages.data = make(3, n, dtype=torch.uint8)
        else:
            c.pages.resize_(3000 if change == "larger" else 2, n)
        launches = mbw.launch_count()
        for call in every_call(c, make):
            with pytest.raises(ValueError, match="pages were moved or resized"):
                call()
        assert mbw.launch_count() == launches and keep is not None
