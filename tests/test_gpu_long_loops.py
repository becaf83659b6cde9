"""The steady state of the loops over a row's blocks: rings that are filled again, windows of list entries that are
loaded again, runs of several tiles a warp.  Short cases end before these begin.

Values carry a mark: channel j % D of block j is 2^e higher than the rest, and queries are small enough for a nearly
flat softmax, so that a block that is left out, or attended to twice, moves that channel by 16 * 2^e / L, several times
the tolerance (each test checks that on the CPU by leaving a block out of the reference)."""
import numpy as np
import pytest
import torch

import quant_util as qu
from parity_util import TOL, max_error

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


def marked(rng, kv, lens, Hkv, D, mark):
    """Pools over shuffled blocks whose values carry the marks."""
    NB, tables = qu.make_tables(rng, lens)
    v_scale = mark / 256.0
    pools = qu.Pools(rng, NB, Hkv, D, kv, v_scale=v_scale)
    v = rng.standard_normal((NB, Hkv, 16, D))
    for s, L in enumerate(lens):
        for j in range((L + 15) // 16):
            v[tables[s, j], :, :, j % D] += mark
    if kv in qu.BITS:
        v = qu.round_to(v, "bf16")
        pools.vh, pools.v_host = qu.held(v, qu.BITS[kv]), qu.pack(v, qu.BITS[kv], True)
    elif kv == "e4m3":
        c = torch.from_numpy(v / v_scale).clamp(-448, 448).float().to(torch.float8_e4m3fn)
        pools.vh, pools.v_host = c.float().double().numpy() * np.float64(np.float32(v_scale)), c.view(torch.uint8).numpy()
    else:
        t = torch.from_numpy(v).to(qu.TORCH[kv])
        pools.vh, pools.v_host = t.double().numpy(), t.view(torch.int16).numpy()
    return pools, tables


def assert_marks_show(q, pools, tables, L, scale, s=0):
    """A reference without one block, the middle one, is far outside the tolerance."""
    n = (L + 15) // 16
    sel = np.arange(n, dtype=np.int32)[None, None].repeat(pools.Hkv, 1)
    less = sel.copy()
    less[..., n // 2] = -1
    refs = [qu.ref_sparse(q[s:s + 1], pools, tables[s:s + 1], [L], x, scale) for x in (sel, less)]
    assert np.abs(refs[0] - refs[1]).max() > 5 * TOL["bf16"]


LENS = [5003, 4801, 130, 4096]


@pytest.mark.parametrize("kv", ["int8", "int4"])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (128, 8)])
@pytest.mark.parametrize("part", [0, 4096, 8192])
def test_dense_decode_over_long_partitions(pk, kv, D, G, part):
    rng = np.random.default_rng(part + D + G)
    Hkv, scale, mx = 2, D ** -0.5, max(LENS)
    pools, tables = marked(rng, kv, LENS, Hkv, D, 64.0)
    q = qu.queries(rng, len(LENS), Hkv * G, D, "bf16", 0.1)
    assert_marks_show(q, pools, tables, LENS[0], scale)
    kd, vd = pools.dev()
    pools.spoil_tail(tables, LENS, kd, vd)
    out = torch.full(q.shape, 7.0, device="cuda").to(q.dtype)
    ws = torch.full((max(16, pk.decode_workspace_bytes(len(LENS), Hkv * G, D, mx, part)),), 255, dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(LENS), mx, scale, out, workspace=ws,
                              partition_tokens=part)
    assert pk.get_device_error() == 0
    ref = qu.ref_dense(q, pools, tables, LENS, scale)
    assert max_error(out.double().cpu().numpy(), ref, "bf16", TOL["bf16"], 70.0) <= TOL["bf16"]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8", "int4"])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (64, 4), (128, 8)])
@pytest.mark.parametrize("part", [0, 150, 320])
def test_sparse_decode_over_long_lists(pk, kv, D, G, part):
    """Lists of 320 entries in any order: all of a row's blocks, repeats, gaps, an end inside a partition."""
    rng = np.random.default_rng(part + D + G)
    Hkv, scale, n = 2, D ** -0.5, 320
    pools, tables = marked(rng, kv, LENS, Hkv, D, 64.0)
    q = qu.queries(rng, len(LENS), Hkv * G, D, "bf16", 0.1)
    assert_marks_show(q, pools, tables, LENS[0], scale)
    sel = np.full((len(LENS), Hkv, n), -1, np.int32)
    for s, L in enumerate(LENS):
        nb = (L + 15) // 16
        for h in range(Hkv):
            m = min(n, nb) - 7 * h
            sel[s, h, np.sort(rng.permutation(n)[:m])] = rng.permutation(nb)[:m]
    sel[1, 1, [3, 200, 319]] = 17  # one block several times
    kd, vd = pools.dev()
    pools.spoil_tail(tables, LENS, kd, vd)
    out = torch.full(q.shape, 7.0, device="cuda").to(q.dtype)
    ws = torch.full((max(16, pk.decode_sparse_workspace_bytes(len(LENS), Hkv * G, D, n, part)),), 255, dtype=torch.uint8,
                    device="cuda")
    pk.paged_attention_decode_sparse(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(LENS), dev32(sel), scale, out,
                                     workspace=ws, partition_blocks=part)
    assert pk.get_device_error() == 0
    ref = qu.ref_sparse(q, pools, tables, LENS, sel, scale)
    assert max_error(out.double().cpu().numpy(), ref, "bf16", TOL["bf16"], 70.0) <= TOL["bf16"]


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_rows_of_twenty_thousand_tokens(pk, kv):
    """The automatic partitions of a long row: a partition or block that is lost or counted twice shows."""
    rng = np.random.default_rng(11)
    lens, Hkv, G, D, scale = [20000, 3, 9001], 1, 8, 128, 128 ** -0.5
    pools, tables = marked(rng, kv, lens, Hkv, D, 128.0)
    q = qu.queries(rng, 3, G, D, "bf16", 0.1)
    assert_marks_show(q, pools, tables, lens[0], scale)
    kd, vd = pools.dev()
    pools.spoil_tail(tables, lens, kd, vd)
    out = torch.full(q.shape, 7.0, device="cuda").to(q.dtype)
    ws = torch.full((pk.decode_workspace_bytes(3, G, D, 20000, 0),), 255, dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(lens), 20000, scale, out, workspace=ws)
    assert pk.get_device_error() == 0
    ref = qu.ref_dense(q, pools, tables, lens, scale)
    assert max_error(out.double().cpu().numpy(), ref, "bf16", TOL["bf16"], 140.0) <= TOL["bf16"]


def score_tiles(S, Hkv, D, max_len, sms):
    """Tiles a warp of the score kernel takes in a run, by the rule of pkv_select_blocks."""
    cdiv = lambda a, b: -(-a // b)
    row_tiles, slots = cdiv(cdiv(max_len, 16), 16), (3 if D == 128 else 5) * sms
    return min(range(1, 65), key=lambda run: (cdiv(cdiv(cdiv(row_tiles, run) * Hkv, 4) * S, slots) * (run + 3), run))


# runs of 5, 6, 7, 10 and 12 tiles on 152 SMs
@pytest.mark.parametrize("dtype,D,Hkv,G,S,blocks", [("bf16", 128, 8, 1, 24, 600), ("f16", 128, 8, 2, 32, 600),
                                                    ("bf16", 64, 8, 4, 40, 900), ("f16", 64, 2, 8, 96, 2100),
                                                    ("bf16", 128, 4, 1, 64, 1300)])
def test_selection_with_runs_of_many_tiles(pk, dtype, D, Hkv, G, S, blocks):
    """Many rows over one set of blocks, with ragged ends: a warp's run of tiles goes round its ring several times."""
    rng = np.random.default_rng(blocks)
    tiles = score_tiles(S, Hkv, D, 16 * blocks, torch.cuda.get_device_properties(0).multi_processor_count)
    assert tiles >= 5
    a, b = rng.standard_normal((2, blocks, Hkv, D))
    bounds = torch.from_numpy(np.stack([np.minimum(a, b) - 0.5, np.maximum(a, b) + 0.5], 2)).to(qu.TORCH[dtype])
    tables = np.stack([rng.permutation(blocks) for _ in range(S)]).astype(np.int32)
    lens = [int(x) for x in rng.integers(1, 16 * blocks + 1, S)]
    lens[0], lens[1], lens[2] = 16 * blocks, 16 * (blocks - 1) + 1, 16 * 16 * (tiles + 1) + 1  # runs of one block more
    q = qu.queries(rng, S, Hkv * G, D, dtype)
    n = 24
    desc = pk.CacheDesc(num_blocks=blocks, num_kv_heads=Hkv, head_size=D, kv_dtype=dtype)
    ws = torch.full((pk.select_blocks_workspace_bytes(S, Hkv, 16 * blocks),), 255, dtype=torch.uint8, device="cuda")
    sel = torch.full((S, Hkv, n), -9, dtype=torch.int32, device="cuda")
    pk.select_blocks(q.cuda(), bounds.cuda(), desc, dev32(tables), dev32(lens), 16 * blocks, sel, ws, sink_blocks=1,
                     recent_blocks=2)
    assert pk.get_device_error() == 0
    want = qu.ref_select(q, bounds.double().numpy(), tables, lens, n, 1, 2, Hkv)
    assert np.array_equal(sel.cpu().numpy(), want)
