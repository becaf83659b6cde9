"""Integer-coded pools on the GPU: append, read, copy, swap, decode and prefill
against the plain 64-bit forms.  Codes and parameters are compared byte for
byte; attention within the parity bounds of the 16-bit output formats, on the
values the pools hold."""
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


def rows(rng, T, H, D, dtype, kind="normal"):
    x = rng.standard_normal((T, H, D))
    if kind == "edge":  # constant rows, tiny and huge ranges, one outlier, grid values that tie half-way
        x[0::6] = x[0::6, :, :1]
        x[1::6] *= 1e-30 if dtype == "bf16" else 1e-6
        x[2::6] *= 1e30 if dtype == "bf16" else 1e4
        x[3::6, :, 5] = 50.0
        x[4::6] = np.round(x[4::6] * 4) / 4
        x[5::6] = 0.0
    return torch.from_numpy(x).to(qu.TORCH[dtype])


@pytest.mark.parametrize("kind", ["normal", "edge"])
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 5), (128, 2), (128, 8)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 37, 300])
def test_append_writes_the_defined_bytes(pk, kv, D, Hkv, dtype, T, kind):
    """Whole pools, byte for byte: the written rows and every byte around them."""
    rng = np.random.default_rng(T * 1000 + D + Hkv)
    NB = T // 8 + 3
    k, v = rows(rng, T, Hkv, D, dtype, kind), rows(rng, T, Hkv, D, dtype, kind)
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    if T > 2:
        slots[::5] = -1
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv)
    fill = rng.integers(0, 256, (2, NB, Hkv, pk.block_bytes(desc) // Hkv), dtype=np.uint8)
    want = fill.copy()
    for t, slot in enumerate(slots):
        if slot >= 0:
            for h in range(Hkv):
                for z, x in ((0, k), (1, v)):
                    qu.write_row(want[z], D, qu.BITS[kv], bool(z), slot // 16, h, slot % 16, x[t, h].float().numpy())
    kd, vd = torch.from_numpy(fill[0].copy()).cuda(), torch.from_numpy(fill[1].copy()).cuda()
    pk.paged_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), kd, vd, desc)
    assert pk.get_device_error() == 0
    assert np.array_equal(kd.cpu().numpy(), want[0]) and np.array_equal(vd.cpu().numpy(), want[1])


def test_append_flags_a_slot_outside_the_pool(pk):
    desc = pk.CacheDesc(num_blocks=2, num_kv_heads=2, head_size=64, kv_dtype="int4")
    kd, vd = (torch.zeros(2, 2, pk.block_bytes(desc) // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.randn(3, 2, 64, device="cuda").half()
    slots = torch.tensor([32, -5, 1 << 40], device="cuda")
    pk.paged_kv_append(x, x, slots, kd, vd, desc)
    assert pk.get_device_error() == pk.DEVERR_SLOT
    assert int(kd.sum()) == 0 and int(vd.sum()) == 0
    out = torch.full((3, 2, 64), 7.0, device="cuda").half()
    pk.paged_kv_read(slots, kd, vd, desc, out, out.clone())
    assert pk.get_device_error() == pk.DEVERR_SLOT and bool((out == 7).all())


@pytest.mark.parametrize("kv", KVS + ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 8)])
@pytest.mark.parametrize("out_dtype", ["f16", "bf16"])
def test_read_returns_the_held_values(pk, kv, D, Hkv, out_dtype):
    if kv in qu.TORCH and kv != out_dtype:
        pytest.skip("a 16-bit pool is read in its own type (refused otherwise, tested on the CPU)")
    rng = np.random.default_rng(D + Hkv)
    NB, T = 9, 70
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kd, vd = pools.dev()
    slots = rng.integers(0, NB * 16, T).astype(np.int64)  # some slots twice
    slots[7] = -1
    ko = torch.full((T, Hkv, D), 9.0, device="cuda").to(qu.TORCH[out_dtype])
    vo = ko.clone()
    pk.paged_kv_read(torch.from_numpy(slots).cuda(), kd, vd, pools.desc, ko, vo)
    assert pk.get_device_error() == 0
    eps = torch.finfo(qu.TORCH[out_dtype]).eps
    for got, held in ((ko, pools.kh), (vo, pools.vh)):
        got = got.double().cpu().numpy()
        assert np.all(got[7] == 9.0)
        ref = held[slots // 16, :, slots % 16]
        # one binary32 operation (relative 2^-24 of the result), then one rounding to 16 bits
        tol = (eps / 2 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25
        bad = np.abs(got - ref) > tol
        bad[7] = False
        assert not bad.any()


@pytest.mark.parametrize("kv", KVS)
def test_copy_and_swap_move_codes_and_parameters(pk, kv):
    rng = np.random.default_rng(5)
    pools = qu.Pools(rng, 6, 3, 64, kv)
    kd, vd = pools.dev()
    pairs = torch.tensor([[1, 4], [2, 5]], dtype=torch.int32, device="cuda")
    pk.copy_blocks(kd, vd, pools.desc, pairs)
    want = pools.k_host.copy()
    want[[4, 5]] = want[[1, 2]]
    assert np.array_equal(kd.cpu().numpy(), want)
    kh, vh = (torch.zeros(2, *pools.k_host.shape[1:], dtype=torch.uint8).pin_memory() for _ in range(2))
    sw = torch.tensor([[3, 0], [0, 1]], dtype=torch.int32, device="cuda")
    pk.swap_blocks(kd, vd, pools.desc, kh, vh, sw, pk.SWAP_OUT)
    torch.cuda.synchronize()
    assert np.array_equal(vh.numpy(), pools.v_host[[3, 0]])
    kd[3] = 0
    pk.swap_blocks(kd, vd, pools.desc, kh, vh, sw, pk.SWAP_IN)
    torch.cuda.synchronize()
    assert np.array_equal(kd.cpu().numpy(), want) and pk.get_device_error() == 0


EDGE_LENS = [1, 15, 16, 17, 31, 33, 100, 255, 511, 512, 513, 1000, 0]


def run_decode(pk, pools, q, tables, lens, scale, part=0, spoil=True, fn=None):
    kd, vd = pools.dev()
    if spoil:
        pools.spoil_tail(tables, lens, kd, vd)
    S, Hq, D = q.shape
    mx = int(max(lens))
    out = torch.full((S, Hq, D), 7.0, device="cuda").to(q.dtype)
    ws = torch.full((max(16, pk.decode_workspace_bytes(S, Hq, D, mx, part)),), 255, dtype=torch.uint8, device="cuda")
    (fn or pk.paged_attention_decode)(q.cuda(), kd, vd, pools.desc, torch.from_numpy(tables).cuda(),
                                      torch.tensor(lens, dtype=torch.int32).cuda(), mx, scale, out, workspace=ws,
                                      partition_tokens=part)
    return out


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("part", [0, 16, 48, 512])
def test_decode_matches_64_bits(pk, kv, D, G, dtype, part):
    """Every element of an edge-length batch; rows past each sequence's end hold all-ones bytes."""
    rng = np.random.default_rng(D + G + part)
    Hkv = 2
    NB, tables = qu.make_tables(rng, EDGE_LENS)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = qu.queries(rng, len(EDGE_LENS), Hkv * G, D, dtype)
    scale = D ** -0.5
    out = run_decode(pk, pools, q, tables, EDGE_LENS, scale, part)
    assert pk.get_device_error() == 0
    ref = qu.ref_dense(q, pools, tables, EDGE_LENS, scale)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)) and np.all(got[-1] == 0)
    assert max_error(got, ref, dtype, TOL[dtype], float(np.abs(pools.vh).max())) <= TOL[dtype]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("qs,vs", [(30.0, 1.0), (1e-3, 1.0), (1.0, 1e-6), (1.0, 300.0), (0.0, 1.0)])
def test_decode_scales_of_queries_and_values(pk, kv, qs, vs):
    """Sharp and flat softmaxes, all-zero queries, tiny and large values (relative to the values' size)."""
    rng = np.random.default_rng(3)
    lens = [1, 40, 700]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 128, kv)
    v = qu.round_to(rng.standard_normal(pools.vh.shape) * vs, "bf16")
    v[::3] *= 2.0 ** -9  # scales that differ from row to row
    pools.vh, pools.v_host = qu.held(v, qu.BITS[kv]), qu.pack(v, qu.BITS[kv], True)
    q = qu.queries(rng, 3, 8, 128, "bf16", qs)
    out = run_decode(pk, pools, q, tables, lens, 128 ** -0.5)
    ref = qu.ref_dense(q, pools, tables, lens, 128 ** -0.5)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)) and pk.get_device_error() == 0
    vmax = float(np.abs(pools.vh).max())
    assert max_error(got / vmax, ref / vmax, "bf16", TOL["bf16"], 1.0) <= TOL["bf16"]
    # tiny values keep their own precision: half an ulp plus the binary32 terms
    eps = 2.0 ** -8
    # p carries 22 bits, scores a binary32 sum: |d score| <= 2^-16 |q|_1 scale (max |k| + range), in nats
    a1 = float(np.abs(q.double().numpy()).sum(-1).max()) * 128 ** -0.5 * 2 * float(np.abs(pools.kh).max())
    tol = eps * np.abs(ref) + vmax * (2 * 2.0 ** -16 * a1 + 2.0 ** -12)
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("kv", KVS)
def test_decode_many_rows_and_long_rows(pk, kv):
    rng = np.random.default_rng(11)
    for lens, Hkv, G, D in (([rng.integers(1, 300) for _ in range(700)], 1, 4, 64), ([20000, 3, 9000], 1, 8, 128)):
        lens = [int(x) for x in lens]
        NB, tables = qu.make_tables(rng, lens)
        pools = qu.Pools(rng, NB, Hkv, D, kv)
        q = qu.queries(rng, len(lens), Hkv * G, D, "bf16")
        out = run_decode(pk, pools, q, tables, lens, D ** -0.5)
        ref = qu.ref_dense(q, pools, tables, lens, D ** -0.5)
        assert pk.get_device_error() == 0
        assert max_error(out.double().cpu().numpy(), ref, "bf16", TOL["bf16"], float(np.abs(pools.vh).max())) <= TOL["bf16"]


@pytest.mark.parametrize("kv", KVS)
def test_decode_flags_bad_ids_and_lengths(pk, kv):
    rng = np.random.default_rng(2)
    lens = [40, 20]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 64, kv)
    q = qu.queries(rng, 2, 4, 64, "bf16")
    bad = tables.copy()
    bad[0, 1] = NB
    out = run_decode(pk, pools, q, bad, lens, 0.125, spoil=False)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
    ref = qu.ref_dense(q, pools, tables, lens, 0.125)
    assert max_error(out.double().cpu().numpy()[1], ref[1], "bf16", TOL["bf16"]) <= TOL["bf16"]
    kd, vd = pools.dev()
    o = torch.empty(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    pk.paged_attention_decode(q.cuda(), kd, vd, pools.desc, torch.from_numpy(tables).cuda(),
                              torch.tensor([-3, 49], dtype=torch.int32).cuda(), 40, 0.125, o)
    assert pk.get_device_error() & pk.DEVERR_SEQ_LEN
    assert bool((o[0] == 0).all())


@pytest.mark.parametrize("kv", KVS)
def test_decode_noalloc_and_graph_and_stream(pk, kv):
    """The built-in scratch, a captured and replayed call whose inputs change, and another stream."""
    rng = np.random.default_rng(8)
    lens = [600, 33]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 128, kv)
    q = qu.queries(rng, 2, 8, 128, "bf16")
    want = run_decode(pk, pools, q, tables, lens, 0.1, 64)
    got = run_decode(pk, pools, q, tables, lens, 0.1, 64,
                     fn=lambda *a, workspace, **k: pk.paged_attention_decode_noalloc(*a, **k))
    assert torch.equal(want, got)
    kd, vd = pools.dev()
    t, l = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qd, out = torch.zeros_like(q).cuda(), torch.zeros_like(q).cuda()
    ws = torch.zeros(pk.decode_workspace_bytes(2, 8, 128, 600, 64), dtype=torch.uint8, device="cuda")
    call = lambda: pk.paged_attention_decode(qd, kd, vd, pools.desc, t, l, 600, 0.1, out, workspace=ws, partition_tokens=64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    qd.copy_(q)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("D,G,dtype", [(64, 1, "f16"), (128, 4, "bf16"), (128, 8, "f16")])
def test_prefill_over_integer_coded_pools(pk, kv, D, G, dtype):
    """Chunked prefill: the staged copy rounds each held value once to q's type."""
    rng = np.random.default_rng(D + G)
    ctx, new = [0, 37, 200], [20, 70, 5]
    lens = [a + b for a, b in zip(ctx, new)]
    Hkv = 2
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kd, vd = pools.dev()
    pools.spoil_tail(tables, lens, kd, vd)
    q = qu.queries(rng, sum(new), Hkv * G, D, dtype)
    out = torch.zeros_like(q).cuda()
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ws = torch.full((pk.prefill_workspace_bytes(kv, 3, Hkv, D, tables.shape[1]),), 255, dtype=torch.uint8, device="cuda")
    pk.paged_attention_prefill(q.cuda(), kd, vd, pools.desc, torch.from_numpy(qs).cuda(), max(new),
                               torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5,
                               out, workspace=ws)
    assert pk.get_device_error() == 0
    pools.kh, pools.vh = qu.round_to(pools.kh, dtype).astype(np.float64), qu.round_to(pools.vh, dtype).astype(np.float64)
    got = out.double().cpu().numpy()
    for s in range(3):
        for j in range(new[s]):
            L = ctx[s] + j + 1
            r = qs[s] + j
            ref = qu.ref_dense(q[r:r + 1], pools, tables[s:s + 1], [L], D ** -0.5)
            assert max_error(got[r:r + 1], ref, dtype, TOL[dtype], float(np.abs(pools.vh).max())) <= TOL[dtype]
