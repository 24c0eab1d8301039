"""The tests' forms of the paged cache for whole pools against those written
token by token (CPU)."""
import numpy as np
import pytest

import _paged as P


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_quantization_hqmq_b200 import build
    build.build()


@pytest.mark.parametrize("S,page,cap", [(8, 16, 0), (32, 32, 5), (48, 16, 400), (1, 64, 30), (11, 16, 20)])
def test_values_of_whole_pools(S, page, cap):
    import _paged_fast as F
    rng = np.random.default_rng(S)
    for pool in (P.empty_pool(rng, 3, 2, page, S, cap), F.filled_pool(rng, 3, 2, page, S, cap)):
        got = F.values(pool)
        want, ok = P.dense(pool, [2, 0, 1], 3 * page)
        assert ok.all()
        np.testing.assert_array_equal(F.dense(got, [2, 0, 1], 3 * page), want)
    b = pool["words"].shape[3]
    idx = rng.integers(0, 1 << b, (7, 32))
    np.testing.assert_array_equal(F.pack_all(idx, b), np.array([P.pack_words(i, b) for i in idx], np.uint32))
    np.testing.assert_array_equal(F.unpack_all(F.pack_all(idx, b), b), idx)
