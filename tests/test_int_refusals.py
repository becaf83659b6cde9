"""Refusals on the CPU of calls whose operands do not hold what the kernels would read or write: nothing here
reaches a device, each call fails a check before any launch."""
import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3", "int8", "int4"])
def test_swap_refuses_host_pools_that_do_not_hold_the_blocks(pk, kv):
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype=kv)
    nbytes = pk.block_bytes(d)
    device = torch.zeros(4, nbytes, dtype=torch.uint8)
    host = lambda n=3, b=nbytes: torch.zeros(n, b, dtype=torch.uint8)
    swap = lambda k, v: pk.swap_blocks(device, device, d, k, v, i32(1, 2), pk.SWAP_OUT)
    for k, v in ((host(b=nbytes - 16), host()), (host(), host(b=nbytes - 16)), (host(), host(2))):
        with pytest.raises(ValueError, match="must hold 3 blocks"):
            swap(k, v)
    if kv == "int8":  # one byte an element leaves no room for the rows' scales and zeros
        with pytest.raises(ValueError, match="must hold 3 blocks"):
            swap(*(torch.zeros(3, 2, 16, 64, dtype=torch.uint8) for _ in range(2)))
    with pytest.raises(ValueError, match="pinned"):  # the right size gets as far as the next check
        swap(host(), host())
