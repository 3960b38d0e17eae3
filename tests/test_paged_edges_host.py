"""Refusals and no-ops at the ends of the paged operators' arguments, without a GPU (as in test_paged_host.py)."""
import pytest

import dense_gemm_transformer_gb300 as dg
from tests.test_paged_host import H, INVALID, MISALIGNED, P, _cache


@pytest.fixture(scope="module")
def lib():
    return dg.load(build_if_missing=True)


def test_grow_checks_its_pools(lib):
    for change, pool, status in [(dict(pool_count=9), (P, 2, 1 << 20, 8192), INVALID),
                                 (dict(page_bytes=-16), (P, 2, 1 << 20, 8192), INVALID),
                                 (dict(page_bytes=8), (P, 2, 1 << 20, 8192), MISALIGNED),
                                 ({}, (P + 8, 2, 1 << 20, 8192), MISALIGNED), ({}, (P, 2, 1 << 20, 8), MISALIGNED),
                                 ({}, (0, 2, 1 << 20, 8192), INVALID)]:
        assert lib.gemm_cache_grow(H, _cache(pool, **change), 1, P, P, 1, P, P, P, None) == status
