"""The workspace of paged attention: a call may need more than a larger one (its tiles go by the rows
of an average slice), so there is a size that no call of the cache passes."""
import itertools

import pytest

from block_causal_attention_b200 import PagedCache, _abi


@pytest.mark.parametrize("hq,hkv,d", [(128, 8, 48), (6, 2, 24), (4, 4, 32), (400, 1, 48)])
def test_no_call_needs_more_than_the_most(hq, hkv, d):
    cache = PagedCache(hq, hkv, d, 10, host_only=True)
    most = cache.max_workspace_bytes()
    sizes = [1, 2, 3, 5, 8, 16, 17, 31, 64, 65, 100, 257, 1000, 1025, 10 ** 5, 2 ** 31 - 1]
    need = {(n, s, w): cache.workspace_bytes(n, s, w)
            for n, s, w in itertools.product(sizes, sizes, (0, 1, 96, 97, 400, 2 ** 24 - 1))}
    assert max(need.values()) == most                        # reached, and nowhere passed
    assert any(need[n, s, w] < need[n, t, w] for n, s, w in need for t in sizes if t < s)


def test_the_most_of_no_cache():
    assert _abi.lib().bca_paged_max_workspace_bytes(None) == 0
