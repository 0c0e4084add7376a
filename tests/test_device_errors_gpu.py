"""mbw_check_device_error names everything that kernels flagged since the last call, and clears it."""
import itertools

import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


def bad_slot():
    x = normal(gen(99), 1, 1, 64)
    mbw.kv4_append(new_cache(1, 16, 1, 64, 32), x, x, torch.tensor([16], device="cuda"))


def attend(nq, hq):
    cache = new_cache(1, 16, 1, 64, 32, fill=0)
    mbw.kv4_attention(cache, normal(gen(99), nq, hq, 64), torch.tensor([[1]], dtype=torch.int32, device="cuda"),
                      torch.tensor([16], dtype=torch.int32, device="cuda"))


def bad_target():
    mbw.token_logprobs(torch.zeros(1, 10, device="cuda"), torch.tensor([10], dtype=torch.int32, device="cuda"))


FLAGS = {"a cache slot or position": bad_slot, "a page id": lambda: attend(1, 1), "a target token id": bad_target,
         "a bounded wait": lambda: mbw.selftest_wait_expiry(64)}


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_all_that_was_flagged_is_named_once(n):
    for words in itertools.combinations(FLAGS, n):
        for w in words:
            FLAGS[w]()
        with pytest.raises(mbw.MbwError) as e:
            mbw.check_device_error()
        assert e.value.status == (7 if "a bounded wait" in words else 8)
        for w in FLAGS:
            assert (w in str(e.value)) == (w in words), (words, str(e.value))
        mbw.check_device_error()


def test_the_chunk_kernels_flag_is_named_too():
    attend(512, 4)  # 2048 query rows
    bad_slot()
    with pytest.raises(mbw.MbwError, match="a cache slot or position.*; a page id"):
        mbw.check_device_error()
    mbw.check_device_error()
