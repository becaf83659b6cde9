"""Sparse decode on the GPU: key bounds and block selection exactly, attention
over selected blocks within the parity bounds, and the calls run together as a
decode loop makes them."""
import numpy as np
import pytest
import torch

import quant_util as qu
from parity_util import TOL, max_error

pytestmark = pytest.mark.gpu

ALL_KV = [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("int8", "bf16"), ("int8", "f16"), ("int4", "bf16")]


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


# ------------------------------------------------------------------- bounds
@pytest.mark.parametrize("kv,dtype", ALL_KV + [("e4m3", "f16"), ("int4", "f16")])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 20), (128, 3)])
def test_bounds_of_touched_blocks(pk, kv, dtype, D, Hkv):
    """Touched blocks get their tokens' extrema (rounded outwards), others stay as they were."""
    rng = np.random.default_rng(D + Hkv)
    lens, new = [1, 16, 17, 40, 100, 0, 64, 33], [1, 1, 1, 30, 100, 0, 0, 17]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kd, vd = pools.dev()
    pools.spoil_tail(tables, lens, kd, vd)
    b0 = qu.round_to(rng.standard_normal((NB, Hkv, 2, D)), dtype)
    bounds = torch.from_numpy(b0).to(qu.TORCH[dtype]).cuda()
    pk.paged_key_bounds(kd, pools.desc, dev32(tables), dev32(lens), dev32(new), 100, bounds)
    assert pk.get_device_error() == 0
    want = qu.ref_bounds(pools, tables, lens, new, b0, dtype)
    assert np.array_equal(bounds.float().cpu().numpy(), want)
    # new_lens None: every block of every sequence
    pk.paged_key_bounds(kd, pools.desc, dev32(tables), dev32(lens), None, max(lens), bounds)
    want = qu.ref_bounds(pools, tables, lens, lens, b0, dtype)
    assert pk.get_device_error() == 0
    assert np.array_equal(bounds.float().cpu().numpy(), want)


def test_bounds_flag_bad_lengths_and_ids(pk):
    rng = np.random.default_rng(1)
    lens = [20, 20, 20, 20]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 64, "bf16")
    kd, _ = pools.dev()
    bounds = torch.zeros(NB, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda l, n, mx=20, t=tables: pk.paged_key_bounds(kd, pools.desc, dev32(t), dev32(l), dev32(n), mx, bounds)
    for l, n, mx in (([20, 20, 20, 33], [0, 0, 0, 1], 20), ([20] * 4, [0, 0, 0, 21], 20), ([20] * 4, [0, 0, 0, -1], 20),
                     ([20] * 4, [0, 0, 0, 9], 8), ([20, 20, 20, -1], [0, 0, 0, 0], 20)):
        call(l, n, mx)
        assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
        assert int(bounds.abs().sum()) == 0
    bad = tables.copy()
    bad[2, 1] = -7
    call(lens, [0, 0, 20, 0], 20, bad)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID


def test_bounds_of_a_block_that_two_sequences_share(pk):
    rng = np.random.default_rng(4)
    pools = qu.Pools(rng, 4, 2, 64, "f16")
    kd, _ = pools.dev()
    tables = np.array([[0, 1], [0, 2]], np.int32)
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.float16, device="cuda")
    pk.paged_key_bounds(kd, pools.desc, dev32(tables), dev32([20, 30]), None, 30, bounds)
    want = qu.ref_bounds(pools, tables, [20, 30], [20, 30], np.zeros((4, 2, 2, 64), np.float32), "f16")
    assert np.array_equal(bounds.float().cpu().numpy(), want)


# ---------------------------------------------------------------- selection
def random_bounds(rng, NB, Hkv, D, dtype):
    a, b = rng.standard_normal((2, NB, Hkv, D))
    x = torch.from_numpy(np.stack([np.minimum(a, b) - 0.5, np.maximum(a, b) + 0.5], 2)).to(qu.TORCH[dtype])
    return x


def run_select(pk, q, bounds, tables, lens, n, sink, recent, Hkv, kv=None):
    S, Hq, D = q.shape
    NB = bounds.shape[0]
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv or ("bf16" if q.dtype == torch.bfloat16 else "f16"))
    mx = max(lens)
    ws = torch.full((pk.select_blocks_workspace_bytes(S, Hkv, mx),), 255, dtype=torch.uint8, device="cuda")
    sel = torch.full((S, Hkv, n), -9, dtype=torch.int32, device="cuda")
    pk.select_blocks(q.cuda(), bounds.cuda(), desc, dev32(tables), dev32(lens), mx, sel, ws, sink_blocks=sink,
                     recent_blocks=recent)
    return sel.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 1), (4, 2), (8, 2)])
@pytest.mark.parametrize("n,sink,recent", [(1, 0, 0), (1, 0, 1), (7, 1, 2), (16, 0, 0), (16, 8, 8), (40, 3, 1)])
def test_selection_is_that_of_exact_arithmetic(pk, dtype, D, G, Hkv, n, sink, recent):
    rng = np.random.default_rng(n + sink + D + G)
    lens = [0, 1, 16, 17, 120, 256, 257, 1000, 3001, 6000]
    NB, tables = qu.make_tables(rng, lens)
    bounds = random_bounds(rng, NB, Hkv, D, dtype)
    q = qu.queries(rng, len(lens), Hkv * G, D, dtype)
    got = run_select(pk, q, bounds, tables, lens, n, sink, recent, Hkv)
    assert pk.get_device_error() == 0
    assert np.array_equal(got, qu.ref_select(q, bounds.double().numpy(), tables, lens, n, sink, recent, Hkv))


def test_selection_with_other_pool_types(pk):
    rng = np.random.default_rng(77)
    lens = [700, 3]
    NB, tables = qu.make_tables(rng, lens)
    for kv in ("e4m3", "int8", "int4"):
        for dtype in ("f16", "bf16"):
            bounds, q = random_bounds(rng, NB, 2, 64, dtype), qu.queries(rng, 2, 4, 64, dtype)
            got = run_select(pk, q, bounds, tables, lens, 9, 1, 1, 2, kv)
            assert np.array_equal(got, qu.ref_select(q, bounds.double().numpy(), tables, lens, 9, 1, 1, 2))


@pytest.mark.parametrize("case", ["equal", "zero_q", "pairs", "outlier", "near", "huge", "tiny", "denormal", "neg_inf", "inf", "nan",
                                  "q_nan", "q_inf"])
def test_selection_ties_and_extreme_scores(pk, case):
    """Equal scores go to the lowest numbers, in bands of two blocks and of all; scores next to the
    border, far outliers, overflow, infinities and NaN leave the answer defined."""
    rng = np.random.default_rng(5)
    D, Hkv, G, n = 128, 2, 4, 33
    lens = [16 * 1200, 16 * 600 - 3, 16 * 40]
    NB, tables = qu.make_tables(rng, lens)
    bounds = random_bounds(rng, NB, Hkv, D, "bf16")
    q = qu.queries(rng, 3, Hkv * G, D, "bf16")
    if case == "equal":
        bounds[:] = bounds[:1]
    elif case == "zero_q":
        q[:] = 0
    elif case == "pairs":
        half = NB // 2
        bounds[half:2 * half] = bounds[:half]
    elif case == "outlier":
        bounds[tables[0, 5], :, 1] = 1e30
        bounds[tables[0, 6], :, :] = -1e30
    elif case == "near":  # one element's last bit between neighbours
        bounds[:] = bounds[:1]
        bounds[:, :, 1, 0] = torch.from_numpy(1 + rng.integers(0, 4, (NB, Hkv)) * 2.0 ** -7).bfloat16()
    elif case == "huge":
        bounds *= 1e36
        q *= 1e4
    elif case == "tiny":
        bounds *= 1e-30
        q *= 1e-8
    elif case == "denormal":  # products below the smallest normal binary32
        bounds *= 1e-36
        q *= 1e-3
    elif case == "q_nan":
        q[0, 3, 5] = float("nan")
        q[1] = float("nan")
    elif case == "q_inf":
        q[0, 3, 5] = float("inf")
        q[1, :, 0] = float("-inf")
    elif case == "neg_inf":
        bounds[::7] = float("-inf")
    elif case == "inf":
        bounds[::300, :, 1] = float("inf")
    elif case == "nan":
        bounds[::5] = float("nan")
    got = run_select(pk, q, bounds, tables, lens, n, 2, 3, Hkv)
    assert pk.get_device_error() == 0
    assert np.array_equal(got, qu.ref_select(q, bounds.double().numpy(), tables, lens, n, 2, 3, Hkv))


def test_selection_of_a_row_longer_than_shared_memory(pk):
    rng = np.random.default_rng(6)
    lens = [16 * 20000 - 1, 16 * 16384, 50]
    NB, tables = qu.make_tables(rng, lens)
    bounds = random_bounds(rng, NB, 1, 64, "f16")
    q = qu.queries(rng, 3, 2, 64, "f16")
    got = run_select(pk, q, bounds, tables, lens, 500, 4, 16, 1)
    assert pk.get_device_error() == 0
    assert np.array_equal(got, qu.ref_select(q, bounds.double().numpy(), tables, lens, 500, 4, 16, 1))
    q[:] = 0  # every score equal: the widest band
    got = run_select(pk, q, bounds, tables, lens, 500, 4, 16, 1)
    assert np.array_equal(got, qu.ref_select(q, bounds.double().numpy(), tables, lens, 500, 4, 16, 1))


def test_selection_flags_bad_lengths_and_ids(pk):
    rng = np.random.default_rng(9)
    lens = [400, 400]
    NB, tables = qu.make_tables(rng, lens)
    bounds, q = random_bounds(rng, NB, 1, 64, "bf16"), qu.queries(rng, 2, 2, 64, "bf16")
    bad = tables.copy()
    bad[0, 4] = NB
    got = run_select(pk, q, bounds, bad, lens, 10, 1, 1, 1)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
    assert 4 not in got[0, 0]
    want = qu.ref_select(q, bounds.double().numpy(), tables, lens, 10, 1, 1, 1)
    assert np.array_equal(got[1], want[1])
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=1, head_size=64)
    ws = torch.zeros(pk.select_blocks_workspace_bytes(2, 1, 400), dtype=torch.uint8, device="cuda")
    sel = torch.zeros(2, 1, 10, dtype=torch.int32, device="cuda")
    pk.select_blocks(q.cuda(), bounds.cuda(), desc, dev32(tables), dev32([-5, 10 ** 9]), 400, sel, ws)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    assert bool((sel[0] == -1).all())


# ---------------------------------------------------------------- attention
def random_lists(rng, lens, Hkv, n):
    """Lists in any order with gaps; one empty; some rows with every block."""
    sel = np.full((len(lens), Hkv, n), -1, np.int32)
    for s, L in enumerate(lens):
        nb = (L + 15) // 16
        for h in range(Hkv):
            m = min(n, nb, int(rng.integers(0, n + 1)) if (s + h) % 3 else n)
            sel[s, h, rng.permutation(n)[:m]] = rng.permutation(nb)[:m]
    return sel


def run_sparse(pk, pools, q, tables, lens, sel, scale, part):
    kd, vd = pools.dev()
    pools.spoil_tail(tables, lens, kd, vd)
    S, Hq, D = q.shape
    out = torch.full((S, Hq, D), 7.0, device="cuda").to(q.dtype)
    ws = torch.full((max(16, pk.decode_sparse_workspace_bytes(S, Hq, D, sel.shape[2], part)),), 255, dtype=torch.uint8,
                    device="cuda")
    pk.paged_attention_decode_sparse(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(lens), dev32(sel), scale, out,
                                     workspace=ws, partition_blocks=part)
    return out


@pytest.mark.parametrize("kv,dtype", ALL_KV)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n,part", [(1, 0), (13, 0), (13, 1), (40, 0), (40, 3), (40, 16)])
def test_sparse_decode_matches_64_bits(pk, kv, dtype, D, G, n, part):
    rng = np.random.default_rng(n + part + D + G)
    lens = [0, 1, 16, 17, 100, 333, 1000]
    Hkv = 2
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = qu.queries(rng, len(lens), Hkv * G, D, dtype)
    sel = random_lists(rng, lens, Hkv, n)
    out = run_sparse(pk, pools, q, tables, lens, sel, D ** -0.5, part)
    assert pk.get_device_error() == 0
    ref = qu.ref_sparse(q, pools, tables, lens, sel, D ** -0.5)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)) and np.all(got[0] == 0)
    assert max_error(got, ref, dtype, TOL[dtype], float(np.abs(pools.vh).max())) <= TOL[dtype]


@pytest.mark.parametrize("kv,dtype", ALL_KV)
def test_automatic_partitions_fit_the_workspace(pk, kv, dtype):
    """A short launch splits its lists as finely as its workspace holds, and writes nothing behind it."""
    rng = np.random.default_rng(8)
    lens, Hkv, G, D, n = [900, 411], 2, 4, 128, 40
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = qu.queries(rng, len(lens), Hkv * G, D, dtype)
    sel = random_lists(rng, lens, Hkv, n)
    kd, vd = pools.dev()
    sizes = [pk.decode_sparse_workspace_bytes(2, Hkv * G, D, n, part) for part in (8, 16)]
    assert sizes[0] == pk.decode_sparse_workspace_bytes(2, Hkv * G, D, n, 0) > sizes[1]

    def call(part, nbytes):
        out = torch.full((2, Hkv * G, D), 7.0, device="cuda").to(q.dtype)
        ws = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device="cuda")
        pk.paged_attention_decode_sparse(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(lens), dev32(sel), D ** -0.5,
                                         out, workspace=ws[:nbytes], partition_blocks=part)
        assert bool((ws[nbytes:] == 255).all())
        return out

    assert torch.equal(call(0, sizes[0]), call(8, sizes[0]))
    for nbytes in (sizes[1], sizes[0] - 16):
        assert torch.equal(call(0, nbytes), call(16, sizes[1]))
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("kv,dtype", ALL_KV[:1] + ALL_KV[2:4])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128)])
def test_sparse_decode_repeats_and_bad_entries(pk, kv, dtype, G, D):
    """A block listed twice counts twice; an entry past the sequence or the table is flagged and skipped."""
    rng = np.random.default_rng(12)
    lens = [50, 100]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 1, D, kv)
    q = qu.queries(rng, 2, G, D, dtype)
    sel = np.array([[[1, 1, 3, -1, -2 ** 31]], [[0, 6, 2, 2, 2]]], np.int32)
    out = run_sparse(pk, pools, q, tables, lens, sel, 0.1, 2)
    assert pk.get_device_error() == 0
    ref = qu.ref_sparse(q, pools, tables, lens, sel, 0.1)
    assert max_error(out.double().cpu().numpy(), ref, dtype, TOL[dtype]) <= TOL[dtype]
    for wrong in (4, 7, 2 ** 31 - 1):
        bad = sel.copy()
        bad[0, 0, 3] = wrong
        out = run_sparse(pk, pools, q, tables, lens, bad, 0.1, 0)
        assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
        assert max_error(out.double().cpu().numpy(), ref, dtype, TOL[dtype]) <= TOL[dtype]
    t = tables.copy()
    t[1, 6] = NB + 5
    run_sparse(pk, pools, q, t, [50, 96], np.where(sel == 6, 5, sel), 0.1, 0)
    assert pk.get_device_error() == 0  # an id that no entry reaches
    kd, vd = pools.dev()
    o = torch.zeros(2, G, D, dtype=q.dtype, device="cuda")
    pk.paged_attention_decode_sparse(q.cuda(), kd, vd, pools.desc, dev32(t), dev32(lens), dev32(sel), 0.1, o)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID


@pytest.mark.parametrize("kv,dtype", ALL_KV)
def test_every_block_selected_is_dense_decode(pk, kv, dtype):
    rng = np.random.default_rng(21)
    lens = [500, 37, 1]
    D, Hkv, G = 128, 2, 4
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    q = qu.queries(rng, 3, Hkv * G, D, dtype)
    n = tables.shape[1]
    sel = np.stack([np.where(np.arange(n) < (L + 15) // 16, np.arange(n), -1) for L in lens])[:, None].repeat(Hkv, 1)
    a = run_sparse(pk, pools, q, tables, lens, sel, 0.1, 0).double().cpu().numpy()
    kd, vd = pools.dev()
    out = torch.empty_like(q).cuda()
    ws = torch.zeros(max(16, pk.decode_workspace_bytes(3, Hkv * G, D, 500, 0)), dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode(q.cuda(), kd, vd, pools.desc, dev32(tables), dev32(lens), 500, 0.1, out, workspace=ws)
    b = out.double().cpu().numpy()
    # both are one rounding from the same real numbers
    assert np.all(np.abs(a - b) <= torch.finfo(q.dtype).eps * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -11)


# ------------------------------------------------------------ as it is used
@pytest.mark.parametrize("kv,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("int8", "bf16"), ("int4", "f16")])
def test_decode_loop(pk, kv, dtype):
    """A prompt, then steps of append, bounds, selection and sparse attention through a captured graph,
    with forked sequences and copy-on-write; every step against the 64-bit forms of the pool's own values."""
    rng = np.random.default_rng(31)
    D, Hkv, G, n = 64, 2, 2, 6
    NB = 64
    alloc = pk.Allocator(NB, 16)
    alloc.seq_new(0, 150)
    alloc.seq_new(1, 40)
    alloc.fork(0, 2)
    seqs = [0, 1, 2]
    shape = (NB, Hkv, 16, D)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kd, vd = pools.dev()
    bounds = torch.zeros(NB, Hkv, 2, D, dtype=qu.TORCH[dtype], device="cuda")
    MB = 16
    t, l = torch.zeros(3, MB, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    tables, lens = alloc.export(seqs, max_blocks=MB)
    pk.paged_key_bounds(kd, pools.desc, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), None, 150, bounds)
    q, out = (torch.zeros(3, Hkv * G, D, dtype=qu.TORCH[dtype], device="cuda") for _ in range(2))
    kn, vn = (torch.zeros(3, Hkv, D, dtype=qu.TORCH[dtype], device="cuda") for _ in range(2))
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    sel = torch.zeros(3, Hkv, n, dtype=torch.int32, device="cuda")
    ws1 = torch.zeros(pk.select_blocks_workspace_bytes(3, Hkv, MB * 16), dtype=torch.uint8, device="cuda")
    ws2 = torch.zeros(max(16, pk.decode_sparse_workspace_bytes(3, Hkv * G, D, n, 2)), dtype=torch.uint8, device="cuda")

    def step():
        pk.paged_kv_append(kn, vn, slots, kd, vd, pools.desc)
        pk.paged_key_bounds(kd, pools.desc, t, l, one, 1, bounds)
        pk.select_blocks(q, bounds, pools.desc, t, l, MB * 16, sel, ws1)
        pk.paged_attention_decode_sparse(q, kd, vd, pools.desc, t, l, sel, D ** -0.5, out, workspace=ws2, partition_blocks=2)

    graph = None
    for it in range(20):
        sl, pairs = alloc.append_batch(seqs)
        if len(pairs):  # copy-on-write: the block, and its bounds
            pr = torch.from_numpy(pairs.reshape(-1, 2)).cuda()
            pk.copy_blocks(kd, vd, pools.desc, pr)
        tables, lens = alloc.export(seqs, max_blocks=MB)
        t.copy_(torch.from_numpy(tables))
        l.copy_(torch.from_numpy(lens))
        slots.copy_(torch.from_numpy(sl))
        for x in (q, kn, vn):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape))))
        if graph is None:
            step()  # warm up; the step is idempotent
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        torch.cuda.synchronize()
        assert pk.get_device_error() == 0
        # the pool's values, read back by slot (tested on its own)
        every = torch.arange(NB * 16, device="cuda")
        ko = torch.zeros(NB * 16, Hkv, D, dtype=qu.TORCH[dtype], device="cuda")
        vo = ko.clone()
        pk.paged_kv_read(every, kd, vd, pools.desc, ko, vo)
        as_held = lambda x: x.double().cpu().numpy().reshape(NB, 16, Hkv, D).transpose(0, 2, 1, 3)
        pools.kh, pools.vh = as_held(ko), as_held(vo)
        ls = lens.tolist()
        b = bounds.double().cpu().numpy()
        eps = torch.finfo(qu.TORCH[dtype]).eps
        for s in range(3):  # bounds hold every key of the sequence (the read rounds scaled codes once)
            for j in range((ls[s] + 15) // 16):
                kk = pools.kh[tables[s, j], :, :min(16, ls[s] - 16 * j)]
                slack = 0 if kv in qu.TORCH else eps
                assert np.all(b[tables[s, j], :, 0] <= kk.min(1) + slack * np.abs(kk.min(1)))
                assert np.all(b[tables[s, j], :, 1] >= kk.max(1) - slack * np.abs(kk.max(1)))
        want = qu.ref_select(q.cpu(), b, tables, ls, n, 1, 1, Hkv)
        assert np.array_equal(sel.cpu().numpy(), want)
        ref = qu.ref_sparse(q.cpu(), pools, tables, ls, want, D ** -0.5)
        # scaled codes: ref is on values rounded once more to 16 bits, half a step of the largest value and key
        extra = 0 if kv in qu.TORCH else eps * float(np.abs(pools.vh).max()) * (1 + float(np.abs(ref).max()))
        assert max_error(out.double().cpu().numpy(), ref, dtype, TOL[dtype], 4.0) <= TOL[dtype] + extra


@pytest.mark.parametrize("kv,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "f16")])
def test_calls_back_to_back_see_their_inputs(pk, kv, dtype):
    """Each call may start while the kernel before it ends: inputs that a kernel writes just before, outputs
    that the call before still reads.  40 steps with changing inputs in the same buffers, nothing waited for
    in between, against the same steps with a wait after every call."""
    rng = np.random.default_rng(41)
    D, Hkv, G, n, S = 128, 2, 4, 9, 5
    lens = [700, 33, 1, 160, 400]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kd, vd = pools.dev()
    dt = qu.TORCH[dtype]
    bounds = torch.zeros(NB, Hkv, 2, D, dtype=dt, device="cuda")
    t = dev32(tables)
    steps = 40
    qs = torch.randn(steps, S, Hkv * G, D, device="cuda").to(dt)
    kn, vn = (torch.randn(steps, S, Hkv, D, device="cuda").to(dt) for _ in range(2))
    ls = torch.stack([dev32([max(1, L - i % 7) for L in lens]) for i in range(steps)])
    slots = torch.stack([torch.tensor([int(tables[s][(int(ls[i][s]) - 1) // 16]) * 16 + (int(ls[i][s]) - 1) % 16
                                       for s in range(S)], device="cuda") for i in range(steps)])
    q, l, sl, one = qs[0].clone(), ls[0].clone(), slots[0].clone(), torch.ones(S, dtype=torch.int32, device="cuda")
    k1, v1 = kn[0].clone(), vn[0].clone()
    sel = torch.zeros(S, Hkv, n, dtype=torch.int32, device="cuda")
    out, dense = torch.zeros_like(q), torch.zeros_like(q)
    ko, vo = torch.zeros_like(k1), torch.zeros_like(v1)
    ws1 = torch.zeros(pk.select_blocks_workspace_bytes(S, Hkv, 700), dtype=torch.uint8, device="cuda")
    ws2 = torch.zeros(pk.decode_sparse_workspace_bytes(S, Hkv * G, D, n, 2), dtype=torch.uint8, device="cuda")
    ws3 = torch.zeros(pk.decode_workspace_bytes(S, Hkv * G, D, 700, 64), dtype=torch.uint8, device="cuda")

    def run(wait):
        kc, vc = kd.clone(), vd.clone()
        bounds.zero_()
        pk.paged_key_bounds(kc, pools.desc, t, ls[0], None, 700, bounds)
        kept = []
        sync = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(steps):
            for dst, src in ((q, qs[i]), (l, ls[i]), (sl, slots[i]), (k1, kn[i]), (v1, vn[i])):
                dst.copy_(src)
                sync()
            pk.paged_kv_append(k1, v1, sl, kc, vc, pools.desc)
            sync()
            pk.paged_kv_read(sl, kc, vc, pools.desc, ko, vo)
            sync()
            pk.paged_key_bounds(kc, pools.desc, t, l, one, 1, bounds)
            sync()
            pk.select_blocks(q, bounds, pools.desc, t, l, 700, sel, ws1)
            sync()
            pk.paged_attention_decode_sparse(q, kc, vc, pools.desc, t, l, sel, 0.1, out, workspace=ws2, partition_blocks=2)
            sync()
            pk.paged_attention_decode(q, kc, vc, pools.desc, t, l, 700, 0.1, dense, workspace=ws3, partition_tokens=64)
            sync()
            kept.append([x.clone() for x in (sel, out, dense, ko, vo)])
        torch.cuda.synchronize()
        return kept

    want = run(True)
    for _ in range(3):
        for i, (a, b) in enumerate(zip(want, run(False))):
            for x, y in zip(a, b):
                assert torch.equal(x, y), i
    assert pk.get_device_error() == 0


def test_two_streams_at_once(pk):
    """The same calls on two streams, each with its own outputs and workspaces."""
    rng = np.random.default_rng(43)
    lens = [3000, 900, 2000, 17]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 128, "int4")
    kd, vd = pools.dev()
    t, l = dev32(tables), dev32(lens)
    q = qu.queries(rng, 4, 16, 128, "bf16").cuda()
    bounds = torch.zeros(NB, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    pk.paged_key_bounds(kd, pools.desc, t, l, None, 3000, bounds)
    torch.cuda.synchronize()

    class One:
        def __init__(self):
            self.stream = torch.cuda.Stream()
            self.sel = torch.zeros(4, 2, 40, dtype=torch.int32, device="cuda")
            self.out, self.dense = torch.zeros_like(q), torch.zeros_like(q)
            self.ws = [torch.zeros(b, dtype=torch.uint8, device="cuda") for b in
                       (pk.select_blocks_workspace_bytes(4, 2, 3000), pk.decode_sparse_workspace_bytes(4, 16, 128, 40, 4),
                        pk.decode_workspace_bytes(4, 16, 128, 3000, 256))]

        def go(self):
            pk.select_blocks(q, bounds, pools.desc, t, l, 3000, self.sel, self.ws[0], stream=self.stream)
            pk.paged_attention_decode_sparse(q, kd, vd, pools.desc, t, l, self.sel, 0.1, self.out, workspace=self.ws[1],
                                             partition_blocks=4, stream=self.stream)
            pk.paged_attention_decode(q, kd, vd, pools.desc, t, l, 3000, 0.1, self.dense, workspace=self.ws[2],
                                      partition_tokens=256, stream=self.stream)

    a, b = One(), One()
    torch.cuda.synchronize()
    a.go()
    torch.cuda.synchronize()
    want = [x.clone() for x in (a.sel, a.out, a.dense)]
    for _ in range(20):
        a.go()
        b.go()
    torch.cuda.synchronize()
    for o in (a, b):
        for x, y in zip(want, (o.sel, o.out, o.dense)):
            assert torch.equal(x, y)
    assert pk.get_device_error() == 0


def test_blocks_past_four_gigabytes(pk):
    """Tables that name the last blocks of pools and bounds larger than 2^32 bytes."""
    rng = np.random.default_rng(47)
    D, Hkv, dtype = 128, 8, "bf16"
    NB = (1 << 32) // (Hkv * 4 * D) + 4000  # bounds alone pass 4 GiB
    lens = [300, 50]
    n_blocks, small = qu.make_tables(rng, lens, spare=0)
    pools = qu.Pools(rng, n_blocks, Hkv, D, "int4")
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype="int4")
    tables = np.where(small >= 0, small + NB - n_blocks, -1).astype(np.int32)
    big = [torch.empty(NB, *a.shape[1:], dtype=torch.uint8, device="cuda") for a in (pools.k_host, pools.v_host)]
    for x, a in zip(big, (pools.k_host, pools.v_host)):
        x[NB - n_blocks:] = torch.from_numpy(a).cuda()
    t, l = dev32(tables), dev32(lens)
    bounds = torch.empty(NB, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    pk.paged_key_bounds(big[0], desc, t, l, None, 300, bounds)
    want = qu.ref_bounds(pools, small, lens, lens, np.zeros((n_blocks, Hkv, 2, D), np.float32), dtype)
    got = bounds[NB - n_blocks:].float().cpu().numpy()
    used = np.unique(small[small >= 0])
    assert np.array_equal(got[used], want[used])
    q = qu.queries(rng, 2, 16, D, dtype)
    sel = torch.zeros(2, Hkv, 5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(pk.select_blocks_workspace_bytes(2, Hkv, 300), dtype=torch.uint8, device="cuda")
    pk.select_blocks(q.cuda(), bounds, desc, t, l, 300, sel, ws)
    assert np.array_equal(sel.cpu().numpy(), qu.ref_select(q, want.astype(np.float64), small, lens, 5, 1, 1, Hkv))
    out = torch.zeros_like(q).cuda()
    pk.paged_attention_decode(q.cuda(), big[0], big[1], desc, t, l, 300, 0.1, out,
                              workspace=torch.zeros(max(16, pk.decode_workspace_bytes(2, 16, D, 300, 0)), dtype=torch.uint8,
                                                    device="cuda"))
    ref = qu.ref_dense(q, pools, small, lens, 0.1)
    assert max_error(out.double().cpu().numpy(), ref, dtype, TOL[dtype], float(np.abs(pools.vh).max())) <= TOL[dtype]
    x = torch.randn(1, Hkv, D, device="cuda").bfloat16()
    slot = torch.tensor([int(tables[0][3]) * 16 + 5], device="cuda")
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    pk.paged_kv_append(x, x, slot, big[0], big[1], desc)
    pk.paged_kv_read(slot, big[0], big[1], desc, ko, vo)
    held = qu.round_to(qu.held(x.float().cpu().numpy(), 4), "bf16")
    # the read forms the value in one binary32 operation: half a step of 16 bits at a tie at most
    assert np.max(np.abs(ko.float().cpu().numpy() - held)) <= 2.0 ** -8 * np.abs(held).max()
    assert torch.equal(ko, vo) and pk.get_device_error() == 0


def test_binding_refusals_on_device_tensors(pk):
    desc = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype="int8")
    pool = torch.zeros(4, 2, 16 * 72, dtype=torch.uint8, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    o = torch.zeros(3, 2, 64, device="cuda").half()
    read = lambda kc=pool, k=o, v=o, s=slots, **kw: pk.paged_kv_read(s, kc, pool, desc, k, v, **kw)
    read()
    for bad, err in ((dict(kc=pool[..., :16 * 64].contiguous()), ValueError),      # no room for the parameters
                     (dict(k=o.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),  # not contiguous
                     (dict(k=o.cpu()), TypeError), (dict(k=o.float(), v=o.float()), TypeError),
                     (dict(v=o.bfloat16()), TypeError), (dict(k=o[:2]), ValueError), (dict(s=slots.int()), TypeError),
                     (dict(out_dtype="f8"), KeyError)):
        with pytest.raises(err):
            read(**bad)
    x = o.clone()
    with pytest.raises(ValueError):
        pk.paged_kv_append(x, x, slots, pool[..., :16 * 64].contiguous(), pool, desc)
    with pytest.raises(pk.PagedKVError):
        pk.paged_attention_decode(torch.zeros(1, 6, 64, device="cuda").half(), pool, pool, desc,
                                  torch.zeros(1, 4, dtype=torch.int32, device="cuda"),
                                  torch.zeros(1, dtype=torch.int32, device="cuda"), 4, 0.1,
                                  torch.zeros(1, 6, 64, device="cuda").half())  # three heads a KV head
    # a stream object, and its handle
    st = torch.cuda.Stream()
    read(stream=st)
    read(stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0


def test_readme_example_of_an_int4_cache_and_sparse_decode():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "int4" in c]
    assert len(code) == 1
    e = {}
    exec(compile(code[0], "README.md example", "exec"), e)
    k, q = e["k"].float().cpu().numpy(), e["q"].double().cpu().numpy()
    kh, vh = qu.held(k, 4), qu.held(e["v"].float().cpu().numpy(), 4)
    start = [0, int(e["lens"][0])]
    sel = e["selected"].cpu().numpy()
    got = e["out"].double().cpu().numpy()
    G = e["Hq"] // e["Hkv"]
    ref = np.zeros_like(got)
    for s in range(e["S"]):
        L = int(e["lens"][s])
        nb = (L + 15) // 16
        for h in range(e["Hkv"]):
            js = sel[s, h][sel[s, h] >= 0]
            assert len(js) == min(nb, e["n"]) and np.all(np.diff(js) > 0) and {0, nb - 2, nb - 1} <= set(js.tolist())
            pos = (js[:, None] * 16 + np.arange(16)).reshape(-1)
            pos = start[s] + pos[pos < L]
            ref[s, h * G:(h + 1) * G] = qu.attend(q[s, h * G:(h + 1) * G], kh[None, pos, h], vh[None, pos, h], [0], [len(pos)],
                                                  e["D"] ** -0.5)
    assert max_error(got, ref, "bf16", TOL["bf16"], float(np.abs(vh).max())) <= TOL["bf16"]
    # the read-back: one binary32 operation, one rounding to bf16
    assert np.all(np.abs(e["k16"].double().cpu().numpy() - kh) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(kh) + 2.0 ** -24)


def test_capture_after_copies_and_across_streams(pk):
    """In one captured graph: calls right after a host-to-device copy, a memset and a device copy, and calls
    on a second stream forked off and joined again."""
    rng = np.random.default_rng(53)
    lens = [900, 40]
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 128, "int8")
    kd, vd = pools.dev()
    t, l = dev32(tables), dev32(lens)
    host = qu.queries(rng, 2, 8, 128, "bf16").pin_memory()
    q, out, dense = (torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    bounds = torch.zeros(NB, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    sel = torch.zeros(2, 2, 12, dtype=torch.int32, device="cuda")
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in
          (pk.select_blocks_workspace_bytes(2, 2, 900), pk.decode_sparse_workspace_bytes(2, 8, 128, 12, 2),
           pk.decode_workspace_bytes(2, 8, 128, 900, 256))]
    side = torch.cuda.Stream()

    def step():
        bounds.zero_()
        pk.paged_key_bounds(kd, pools.desc, t, l, None, 900, bounds)
        q.copy_(host, non_blocking=True)
        pk.select_blocks(q, bounds, pools.desc, t, l, 900, sel, ws[0])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pk.paged_attention_decode(q, kd, vd, pools.desc, t, l, 900, 0.1, dense, workspace=ws[2], partition_tokens=256)
        out.zero_()
        pk.paged_attention_decode_sparse(q, kd, vd, pools.desc, t, l, sel, 0.1, out, workspace=ws[1], partition_blocks=2)
        torch.cuda.current_stream().wait_stream(side)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(3):
        host.copy_(qu.queries(np.random.default_rng(seed), 2, 8, 128, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        want = qu.ref_select(host, bounds.double().cpu().numpy(), tables, lens, 12, 1, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want)
        vmax = float(np.abs(pools.vh).max())
        ref = qu.ref_sparse(host, pools, tables, lens, want, 0.1)
        assert max_error(out.double().cpu().numpy(), ref, "bf16", TOL["bf16"], vmax) <= TOL["bf16"]
        ref = qu.ref_dense(host, pools, tables, lens, 0.1)
        assert max_error(dense.double().cpu().numpy(), ref, "bf16", TOL["bf16"], vmax) <= TOL["bf16"]
    assert pk.get_device_error() == 0
