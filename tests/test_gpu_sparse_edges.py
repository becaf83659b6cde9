"""Block selection and sparse decode where sums leave binary32, and on the long loops that short cases do not reach."""
import numpy as np
import pytest
import torch

import quant_util as qu

pytestmark = pytest.mark.gpu


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


def dev32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def select(pk, q, bounds, tables, lens, n, sink, recent, Hkv, bounds_dev=None):
    S, Hq, D = q.shape
    desc = pk.CacheDesc(num_blocks=bounds.shape[0], num_kv_heads=Hkv, head_size=D,
                        kv_dtype="bf16" if q.dtype == torch.bfloat16 else "f16")
    ws = torch.full((pk.select_blocks_workspace_bytes(S, Hkv, max(lens)),), 255, dtype=torch.uint8, device="cuda")
    sel = torch.full((S, Hkv, n), -9, dtype=torch.int32, device="cuda")
    pk.select_blocks(q.cuda(), bounds.cuda() if bounds_dev is None else bounds_dev, desc, dev32(tables), dev32(lens),
                     max(lens), sel, ws, sink_blocks=sink, recent_blocks=recent)
    assert pk.get_device_error() == 0
    return sel.cpu().numpy()


@pytest.mark.parametrize("first", [-1.0, 1.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [5, 40])
def test_sums_that_leave_binary32_on_the_way_to_a_finite_score(pk, first, D, n):
    """A few blocks' scores start with a quarter of the channels at +-2^124 and the next quarter takes them back:
    binary32 sums end in an infinity or NaN where the true score is the row's highest.  |q|_1 max |bound| is 2^130
    or 2^131, and no score is infinite."""
    rng = np.random.default_rng(n + D)
    lens, Hkv, G = [16 * 300, 16 * 90 - 5], 2, 4
    NB, tables = qu.make_tables(rng, lens)
    q = torch.full((2, Hkv * G, D), 2.0 ** 60, dtype=torch.bfloat16)
    hi = rng.uniform(1, 2, (NB, Hkv, D)) * 2.0 ** 53
    c = D // 4
    for s, js in ((0, [3, 77, 150, 299]), (1, [11, 12])):
        for i, j in enumerate(js):
            b = tables[s, j]
            hi[b, :, :c], hi[b, :, c:2 * c] = first * 2.0 ** 64, -first * 2.0 ** 64
            hi[b, :, 2 * c:] = 2.0 ** (57 + i)  # true scores 2^(117 + i) D / 2, above 2^(114) D
    bounds = torch.from_numpy(np.stack([np.full_like(hi, -2.0 ** 64), hi], 2)).to(torch.bfloat16)
    want = qu.ref_select(q, bounds.double().numpy(), tables, lens, n, 1, 1, Hkv)
    assert {3, 77, 150}.issubset(want[0, 0]) and {11, 12}.issubset(want[1, 1])
    assert np.array_equal(select(pk, q, bounds, tables, lens, n, 1, 1, Hkv), want)
