"""What PagedCache refuses by looking at tensors alone (fake CUDA tensors: no GPU, no data)."""
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from learned_kv_cache_gb300 import paged
from learned_kv_cache_gb300.paged import PagedCache


@pytest.fixture(autouse=True)
def fake():
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")                         # a fake tensor's data pointer is 0
        yield


def pool(*shape, dtype=torch.float16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def ints(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="cuda")


def cache(k, v=None):
    return PagedCache(k, k if v is None else v, ints(4, 8), ints(4), ints(k.shape[0]), ints((k.shape[0] + 31) // 32))


def test_broadcast_pools_are_refused():
    """A stride of 0 stands for the dense one in the descriptor: the pages of a pool that has one each 1024
    elements would be looked for behind the end of a pool that repeats a page."""
    one = pool(1, 16, 64)
    for bad in (one.expand(100, 16, 64), pool(100, 1, 64).expand(100, 16, 64), pool(100, 2, 1, 64)[:, 0].expand(100, 16, 64),
                pool(1, 1, 64).expand(100, 16, 64)):
        assert 0 in bad.stride()
        with pytest.raises(ValueError, match="broadcast"):
            cache(bad)


def test_strided_pools_are_taken():
    """Interleaved K and V, padded tokens, one-page pools whatever their page stride says."""
    kv = pool(100, 2, 16, 64)
    c = cache(kv[:, 0], kv[:, 1])
    assert (c._desc.page_stride, c._desc.token_stride) == (2048, 64)
    c = cache(pool(100, 16, 128)[:, :, :64])
    assert (c._desc.page_stride, c._desc.token_stride) == (2048, 128)
    c = cache(pool(1, 16, 64).expand(1, 16, 64))
    assert (c._desc.page_stride, c._desc.token_stride) == (0, 64)


def test_a_stream_of_another_device_is_refused():
    """It used to be dropped: the call ran on the current stream of the cache's device."""
    c = cache(pool(100, 16, 64))
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    z, q = pool(4, 1, 64), pool(2, 4, 64)
    for call in (lambda: paged.kvp_paged_init(c, stream=other), lambda: paged.kvp_paged_append(c, z, z, stream=other),
                 lambda: paged.kvp_paged_fork(c, ints(4), stream=other), lambda: paged.kvp_paged_free(c, stream=other),
                 lambda: paged.kvp_paged_compact(c, ints(4, 1), ints(4), stream=other),
                 lambda: paged.kvp_paged_decode_attn(q, c, stream=other)):
        with pytest.raises(ValueError, match="stream must be on cuda:0, got cuda:1"):
            call()
