"""The paged cache's status word: nothing that was recorded is lost."""
import pytest
import torch

import paged_ref as ref
from block_causal_attention_b200 import PagedCache, _abi
from test_gpu_paged import BF, gen, rand

pytestmark = pytest.mark.gpu


def test_kinds_of_error_are_reported_one_after_the_other():
    """A wait that ran out, and a written token without a page, before the word is read."""
    g = gen(31)
    cache = PagedCache(4, 2, 48, 4, test_force_timeout=True)
    table = ref.i32([[0, 1]])
    cache.attend(rand((1, 4, 48), BF, g), table, ref.i32([0, 1]), ref.i32([0]), ref.i32([200]))
    k = rand((3, 2, 48), BF, g)
    cache.write(k, k, table, ref.i32([0, 3]), ref.i32([256]))
    assert cache.status() == _abi.BCA_ERR_DEVICE_TIMEOUT
    assert cache.status() == _abi.BCA_ERR_BAD_PAGE
    assert cache.status() == _abi.BCA_OK


def test_a_new_cache_says_ok_on_any_stream_and_errors_of_other_streams_are_seen():
    g = gen(32)
    side = torch.cuda.Stream()
    k = rand((3, 2, 48), BF, g)
    table, off, at = ref.i32([[0, 1]]), ref.i32([0, 3]), ref.i32([256])
    torch.cuda.synchronize()
    for _ in range(5):
        cache = PagedCache(4, 2, 48, 4)
        assert cache.status(side) == _abi.BCA_OK
        cache.write(k, k, table, off, at, stream=side)
        side.synchronize()
        assert cache.status() == _abi.BCA_ERR_BAD_PAGE
        assert cache.status(side) == _abi.BCA_OK
