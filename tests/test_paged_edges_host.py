"""Refusals and no-ops at the ends of the paged operators' arguments, without a GPU (as in test_paged_host.py)."""
import pytest
import torch

import dense_gemm_transformer_gb300 as dg
from dense_gemm_transformer_gb300 import paged
from tests.test_paged_host import ATTENTION, H, INVALID, MISALIGNED, OK, P, ROTARY, _cache, _pack


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


def _tensor_of(device, shape, dtype):
    """A tensor said to be on a CUDA device, over an address that nothing reads."""
    count = 1
    stride = []
    for n in reversed(shape):
        stride.insert(0, count)
        count *= n
    storage = torch._C._construct_storage_from_data_pointer(P, torch.device(device), count * dtype.itemsize)
    meta = {"dtype": dtype, "storage_offset": 0, "size": torch.Size(shape), "stride": tuple(stride),
            "device": torch.device(device), "storage": storage}
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(meta, storage)


def test_tensors_of_another_device_are_refused(lib):
    """Before the library is called: its handle there is None."""
    ops = paged.PagedOps()
    ops._lib, ops._h = lib, None
    device = "cuda:7"
    x = _tensor_of(device, (4, 2, 64), torch.bfloat16)
    pages = _tensor_of(device, (3, 16, 2, 64), torch.bfloat16)
    table, lens = _tensor_of(device, (4, 3), torch.int32), _tensor_of(device, (4,), torch.int32)
    refs, slots = _tensor_of(device, (3,), torch.int32), _tensor_of(device, (4,), torch.int64)
    with pytest.raises(ValueError, match="current device"):
        ops.rotary(x, None, slots, slots, q_out=x)
    with pytest.raises(ValueError, match="current device"):
        ops.rotary(x, None, slots, slots, q_out=x, stream=0x1000)
    with pytest.raises(ValueError, match="current device"):
        ops.rotary_append(x, x, x, None, slots, pages, pages, q_out=x)
    with pytest.raises(ValueError, match="current device"):
        ops.paged_attention(x, pages, pages, table, lens, out=x)
    with pytest.raises(ValueError, match="current device"):
        ops.cache_grow(table, lens, refs, 16, lens, lens, 4)
    with pytest.raises(ValueError, match="current device"):
        ops.cache_shrink(table, lens, refs, 16, lens)
    with pytest.raises(ValueError, match="current device"):
        ops.cache_fork((pages,), table, lens, refs, 16, lens, lens)
    with pytest.raises(ValueError, match="current device"):
        ops.cache_compact((pages,), table, refs)
    with pytest.raises(ValueError, match="current device"):
        ops.cache_copy((pages,), refs, refs)


def test_nothing_to_append_is_no_error(lib):
    """Tensors without elements have no address."""
    none = dict(tokens=0, q=0, k=0, v=0, q_out=0, positions=0, slots=0)
    assert lib.gemm_rotary(H, _pack("gemm_rotary_t", {**ROTARY, **none}), None) == OK
    assert lib.gemm_rotary(H, _pack("gemm_rotary_t", {**ROTARY, **none, "head_dim": 127}), None) == INVALID
    assert lib.gemm_rotary(H, _pack("gemm_rotary_t", {**ROTARY, **none, "num_pages": -1}), None) == INVALID


def test_attention_over_its_queries_is_refused(lib):
    assert ATTENTION["out"] == ATTENTION["q"]
    assert lib.gemm_paged_attention(H, _pack("gemm_paged_attention_t", ATTENTION), None) == INVALID
    assert lib.gemm_paged_attention(H, _pack("gemm_paged_attention_t", {**ATTENTION, "k_slot": 260}), None) == MISALIGNED
