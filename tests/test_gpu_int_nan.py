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


LENS = [500, 33, 17]


def attend(pk, pools, kd, vd, q, tables, way, part):
    S, Hq, D = q.shape
    t, l = torch.from_numpy(tables).cuda(), torch.tensor(LENS, dtype=torch.int32).cuda()
    out = torch.full((S, Hq, D), 7.0, device="cuda").to(q.dtype)
    n = tables.shape[1]
    buf = lambda b: torch.full((max(16, b),), 255, dtype=torch.uint8, device="cuda")
    if way == "dense":
        pk.paged_attention_decode(q.cuda(), kd, vd, pools.desc, t, l, max(LENS), D ** -0.5, out, partition_tokens=16 * part,
                                  workspace=buf(pk.decode_workspace_bytes(S, Hq, D, max(LENS), 16 * part)))
    else:
        sel = np.stack([np.where(np.arange(n) < (L + 15) // 16, np.arange(n), -1) for L in LENS])
        sel = torch.from_numpy(np.repeat(sel[:, None], pools.Hkv, 1).astype(np.int32)).cuda()
        pk.paged_attention_decode_sparse(q.cuda(), kd, vd, pools.desc, t, l, sel, D ** -0.5, out, partition_blocks=part,
                                         workspace=buf(pk.decode_sparse_workspace_bytes(S, Hq, D, n, part)))
    assert pk.get_device_error() == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("part", [1, 2, 4, 8, 32])  # 32, 16, 8, 4 partitions and one: every form of the merge
@pytest.mark.parametrize("way", ["dense", "sparse"])
@pytest.mark.parametrize("what", ["query", "key", "value", "all_keys"])
@pytest.mark.parametrize("D,G", [(128, 1), (64, 4), (128, 8)])
@pytest.mark.parametrize("kv", KVS)
def test_nan_reaches_its_heads_and_no_others(pk, kv, D, G, what, way, part):
    rng = np.random.default_rng(part + D)
    Hkv = 2
    NB, tables = qu.make_tables(rng, LENS)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = qu.queries(rng, 3, Hkv * G, D, "bf16")
    ref = qu.ref_dense(q, pools, tables, LENS, D ** -0.5)
    kd, vd = pools.dev()
    pools.spoil_tail(tables, LENS, kd, vd)
    hit = np.zeros((3, Hkv * G), bool)
    if what == "query":
        q[0, G, 3] = q[2, 0, D - 1] = float("nan")
        hit[0, G] = hit[2, 0] = True
    else:
        rb = D * qu.BITS[kv] // 8
        pool = vd if what == "value" else kd
        nan = torch.full((8,), 255, dtype=torch.uint8, device="cuda")  # scale and zero NaN
        for s, t in ((0, 18), (0, 499), (1, 32)) if what != "all_keys" else [(0, t) for t in range(500)]:
            at = 16 * rb + 8 * (t % 16)
            pool[int(tables[s, t // 16]), 1, at:at + 8] = nan
            hit[s, G:] = True
    got = attend(pk, pools, kd, vd, q, tables, way, part)
    assert np.array_equal(np.isnan(got), np.broadcast_to(hit[..., None], got.shape))
    assert max_error(got[~hit], ref[~hit], "bf16", TOL["bf16"], float(np.abs(pools.vh).max())) <= TOL["bf16"]


@pytest.mark.parametrize("part", [2, 32])
@pytest.mark.parametrize("way", ["dense", "sparse"])
@pytest.mark.parametrize("kv", KVS)
def test_scores_past_binary32(pk, kv, way, part):
    """Blocks whose scores all overflow to -inf weigh nothing beside blocks with finite scores."""
    rng = np.random.default_rng(3)
    D, Hkv, G, bits = 128, 1, 4, qu.BITS[kv]
    NB, tables = qu.make_tables(rng, LENS)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = torch.from_numpy((np.abs(rng.standard_normal((3, Hkv * G, D))) + 0.5) * 1e25).to(torch.bfloat16)
    k = rng.standard_normal((NB, Hkv, 16, D)) * 1e-26
    for s, L in enumerate(LENS):  # all but the last two blocks: q . k = -1e50
        k[tables[s, :max(0, (L + 15) // 16 - 2)]] = -1e25
    k = qu.round_to(k, "bf16")
    pools.kh, pools.k_host = qu.held(k, bits), qu.pack(k, bits, False)
    ref = qu.ref_dense(q, pools, tables, LENS, D ** -0.5)
    got = attend(pk, pools, *pools.dev(), q, tables, way, part)
    assert max_error(got, ref, "bf16", TOL["bf16"], float(np.abs(pools.vh).max())) <= TOL["bf16"]
