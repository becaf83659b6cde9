"""NaN, infinities and ranges past binary32 in what integer-coded pools are given: a row that its codes cannot
express reads back as NaN and touches no other row; a NaN score or value gives NaN in the heads that it reaches,
however the sequence is split, and nowhere else."""
import numpy as np
import pytest
import torch

import quant_util as qu
from parity_util import TOL, max_error

pytestmark = pytest.mark.gpu

KVS = ["int8", "int4"]


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    pagedkv.lib()
    yield pagedkv


@pytest.fixture(autouse=True)
def clean(pk):
    pk.get_device_error()
    yield
    torch.cuda.synchronize()


def spoil(x):
    """Rows of x [T, H, D] that no codes express; returns their numbers."""
    nan, inf = float("nan"), float("inf")
    D = x.shape[-1]
    x[1, :, 0] = nan
    x[3, :, D - 1] = nan
    x[4, :, 6] = nan
    x[7] = nan
    x[8, :, 9] = inf
    x[10, :, 10] = -inf
    x[11, :, 2], x[11, :, 3] = inf, -inf
    x[13] = inf  # constant, and still no finite range
    bad = [1, 3, 4, 7, 8, 10, 11, 13]
    if x.dtype == torch.bfloat16:
        x[14, :, 1], x[14, :, 2] = -3e38, 3e38  # finite, but hi - lo is not
        bad.append(14)
    return bad


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_that_no_codes_express(pk, kv, D, Hkv, dtype):
    rng = np.random.default_rng(D)
    T, NB, bits = 40, 4, qu.BITS[kv]
    k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, D))).to(qu.TORCH[dtype]) for _ in range(2))
    bad = spoil(k)
    spoil(v)
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv)
    fill = rng.integers(0, 256, (2, NB, Hkv, pk.block_bytes(desc) // Hkv), dtype=np.uint8)
    want, rb = fill.copy(), D * bits // 8
    params = np.zeros(fill.shape, bool)  # bytes of the spoiled rows' scales and zeros
    for t, slot in enumerate(slots):
        b, o = slot // 16, slot % 16
        for h in range(Hkv):
            for z, x in ((0, k), (1, v)):
                if t in bad:
                    want[z, b, h, qu.places(D, bits, bool(z))[o]] = 0
                    params[z, b, h, 16 * rb + 8 * o:16 * rb + 8 * o + 8] = True
                else:
                    qu.write_row(want[z], D, bits, bool(z), b, h, o, x[t, h].float().numpy())
    pools = [torch.from_numpy(f.copy()).cuda() for f in fill]
    pk.paged_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), *pools, desc)
    got = np.stack([p.cpu().numpy() for p in pools])
    assert np.array_equal(got[~params], want[~params])
    assert np.all(np.isnan(got[params].view(np.float32)))
    ko, vo = (torch.zeros(T, Hkv, D, dtype=qu.TORCH[dtype], device="cuda") for _ in range(2))
    pk.paged_kv_read(torch.from_numpy(slots).cuda(), *pools, desc, ko, vo)
    for o in (ko, vo):
        nan = torch.isnan(o).cpu().numpy()
        assert np.all(nan[bad]) and not nan[np.setdiff1d(np.arange(T), bad)].any()
    assert pk.get_device_error() == 0
