"""Eviction on the GPU: kept tokens against a sort, moved rows byte for byte over every pool type, in place and into other
blocks, and the whole cycle of rotating, writing, attending, evicting and going on."""
import numpy as np
import pytest
import torch

import quant_util as qu
import score_util as su
from parity_util import TOL, max_error

pytestmark = pytest.mark.gpu

KVS = ["f16", "bf16", "e4m3", "int8", "int4"]


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


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def weights_of(rng, kind, shape):
    w = np.exp(3 * rng.standard_normal(shape) - 5).astype(np.float32)
    if kind == "ties":
        w = np.round(rng.random(shape) * 3).astype(np.float32)
    elif kind == "one_value":
        w[:] = 0.25
    elif kind == "signs":
        w = rng.choice(np.array([0.0, -0.0, -1.5, 2.0 ** -149, -(2.0 ** -149), 3e38, np.inf, -np.inf, np.nan, 1.0], np.float32), shape)
    elif kind == "close":  # differing in the last bits alone
        w = (1 + rng.integers(0, 40, shape) * 2.0 ** -23).astype(np.float32)
    return w


@pytest.mark.parametrize("kind", ["heavy", "ties", "one_value", "signs", "close"])
@pytest.mark.parametrize("n,sink,recent", [(1, 0, 0), (1, 1, 0), (16, 0, 0), (16, 3, 4), (100, 4, 96), (300, 0, 300), (500, 17, 33)])
def test_select_tokens(pk, kind, n, sink, recent):
    rng = np.random.default_rng([n, sink])
    lens = [0, 1, 15, 16, 17, 100, 101, 300, 511, 1025, 2000, 3333]
    NB, tables = qu.make_tables(rng, lens)
    Hkv = 3
    w = weights_of(rng, kind, (NB, Hkv, 16))
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=64, kv_dtype="f16")
    kept = torch.full((len(lens), Hkv, n), 77, dtype=torch.int32, device="cuda")
    pk.select_tokens(torch.from_numpy(w).cuda(), desc, i32(tables), i32(lens), max(lens), kept, sink, recent)
    assert pk.get_device_error() == 0
    assert np.array_equal(kept.cpu().numpy(), su.ref_select_tokens(w, tables, lens, n, sink, recent))


@pytest.mark.parametrize("L,n", [(50000, 300), (50000, 49000), (90001, 12345)])
def test_select_tokens_of_rows_past_the_cached_ones(pk, L, n):
    rng = np.random.default_rng(L + n)
    NB, tables = qu.make_tables(rng, [L, 40])
    w = weights_of(rng, "heavy", (NB, 1, 16))
    w[rng.random(w.shape) < 0.3] = 0
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=1, head_size=64, kv_dtype="f16")
    kept = torch.zeros(2, 1, n, dtype=torch.int32, device="cuda")
    pk.select_tokens(torch.from_numpy(w).cuda(), desc, i32(tables), i32([L, 40]), L, kept, 4, 50)
    assert pk.get_device_error() == 0
    assert np.array_equal(kept.cpu().numpy(), su.ref_select_tokens(w, tables, [L, 40], n, 4, 50))


def moved(pools, kept, tables, dst, w0):
    """Host pools after the compaction, byte by byte of each row."""
    bits = qu.BITS.get(pools.kv)
    out = []
    for pool, value in ((pools.k_host, False), (pools.v_host, True)):
        src, new = pool.copy(), pool.copy()
        rb = pools.D * (bits or 0) // 8
        at = qu.places(pools.D, bits, value) if bits else None
        for s in range(len(kept)):
            for h in range(pools.Hkv):
                for i, t in enumerate(kept[s, h]):
                    if t < 0:
                        continue
                    a, b, x, y = tables[s][t // 16], dst[s][i // 16], t % 16, i % 16
                    if bits:
                        new[b, h, at[y]] = src[a, h, at[x]]
                        new[b, h, 16 * rb + 8 * y:16 * rb + 8 * y + 8] = src[a, h, 16 * rb + 8 * x:16 * rb + 8 * x + 8]
                    else:
                        new[b, h, y] = src[a, h, x]
        out.append(new)
    w = w0.copy()
    for s in range(len(kept)):
        for h in range(pools.Hkv):
            for i, t in enumerate(kept[s, h]):
                if t >= 0:
                    w[dst[s][i // 16], h, i % 16] = w0[tables[s][t // 16], h, t % 16]
    return out[0], out[1], w


@pytest.mark.parametrize("where", ["in_place", "elsewhere", "partly"])
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("D,Hkv,S", [(64, 1, 2), (128, 2, 2), (64, 8, 24), (128, 8, 12)])
@pytest.mark.parametrize("n", [1, 20, 333])
def test_compaction_moves_the_rows(pk, where, kv, D, Hkv, S, n):
    rng = np.random.default_rng([D, Hkv, S, n])
    lens = [int(x) for x in rng.integers(0, 800, S)]
    lens[0], lens[-1] = 700, 1
    NB, tables = qu.make_tables(rng, lens, spare=S * 22 + 3)
    pools = qu.Pools(rng, NB, Hkv, D, kv)
    kept = np.full((S, Hkv, n), -1, np.int32)
    for s, L in enumerate(lens):
        for h in range(Hkv):
            m = min(n, L)
            kept[s, h, :m] = np.sort(rng.choice(L, m, replace=False))
            if m and h == 0:
                kept[s, h, :m] = np.arange(L - m, L)  # the last ones: every row moves by the same distance
    free = [b for b in range(NB) if not np.any(tables == b)]
    dst = np.full((S, max(1, -(-n // 16))), -1, np.int32)
    for s, L in enumerate(lens):
        for j in range(-(-min(n, L) // 16)):
            other = where == "elsewhere" or (where == "partly" and rng.random() < 0.5)
            dst[s, j] = free.pop() if other else tables[s, j]
    w0 = rng.random((NB, Hkv, 16)).astype(np.float32)
    kw, vw, ww = moved(pools, kept, tables, dst, w0)
    kd, vd = pools.dev()
    w = torch.from_numpy(w0.copy()).cuda()
    pk.paged_kv_compact(i32(kept), kd, vd, pools.desc, i32(tables), i32(lens), i32(dst), weights=w)
    assert pk.get_device_error() == 0
    host = lambda t: t.view(torch.int16).cpu().numpy() if t.element_size() == 2 else t.cpu().numpy()
    assert np.array_equal(host(kd).view(kw.dtype), kw) and np.array_equal(host(vd).view(vw.dtype), vw)
    assert np.array_equal(w.cpu().numpy(), ww)
    # without weights the rows move all the same
    kd, vd = pools.dev()
    pk.paged_kv_compact(i32(kept), kd, vd, pools.desc, i32(tables), i32(lens), i32(dst))
    assert np.array_equal(host(kd).view(kw.dtype), kw) and np.array_equal(host(vd).view(vw.dtype), vw)


@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_in_place_over_a_long_row(pk, kv):
    """Many chunks, one pass after another over the same blocks."""
    rng = np.random.default_rng(1)
    L, n = 12000, 9000
    NB, tables = qu.make_tables(rng, [L])
    pools = qu.Pools(rng, NB, 1, 128, kv)
    kept = np.sort(rng.choice(L, n, replace=False)).astype(np.int32).reshape(1, 1, n)
    w0 = rng.random((NB, 1, 16)).astype(np.float32)
    want = moved(pools, kept, tables, tables, w0)
    for _ in range(20):
        kd, vd = pools.dev()
        w = torch.from_numpy(w0.copy()).cuda()
        tb = i32(tables)
        pk.paged_kv_compact(i32(kept), kd, vd, pools.desc, tb, i32([L]), tb, weights=w)
        host = lambda t: t.view(torch.int16).cpu().numpy() if t.element_size() == 2 else t.cpu().numpy()
        assert np.array_equal(host(kd).view(want[0].dtype), want[0]) and np.array_equal(host(vd).view(want[1].dtype), want[1])
        assert np.array_equal(w.cpu().numpy(), want[2])
    assert pk.get_device_error() == 0


def test_bad_entries_are_reported_and_skipped(pk):
    rng = np.random.default_rng(0)
    NB, tables = qu.make_tables(rng, [40, 40])
    pools = qu.Pools(rng, NB, 2, 64, "bf16")
    kd, vd = pools.dev()
    k0 = kd.clone()
    w = torch.ones(NB, 2, 16, device="cuda")
    call = lambda kept, t=tables, d=tables, L=(40, 40): pk.paged_kv_compact(i32(kept), kd, vd, pools.desc, i32(t), i32(L), i32(d), weights=w)
    kept = np.full((2, 2, 3), -1, np.int32)
    call(kept)
    assert pk.get_device_error() == 0
    kept[:, :, 0] = 40
    call(kept)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    kept[:, :, 0] = 20
    t = tables.copy()
    t[:, 1] = NB
    call(kept, t=t)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
    call(kept, d=np.full_like(tables, -7))
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
    kept[:] = -1
    call(kept, L=(-1, 100))
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    assert torch.equal(kd, k0)
    out = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    pk.select_tokens(w, pools.desc, i32(tables), i32([49, -1]), 40, out)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    pk.select_tokens(w, pools.desc, i32(t), i32([40, 40]), 48, out)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID
    assert bool(((out >= 0) & (out < 40)).all()) and not bool(((out >= 16) & (out < 32)).any())


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("capture", [False, True])
def test_a_serving_loop(pk, kv, capture):
    """Prompt, steps with shares, eviction at a budget, steps on: after every part the attention is that of the kept
    rows, which the model of the loop holds in 64 bits."""
    rng = np.random.default_rng(11)
    Hq, Hkv, D, budget, NB = 8, 2, 128, 60, 64
    dt, prompts = torch.bfloat16, [150, 70, 33]
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv)
    kc, vc = (torch.zeros(NB * pk.block_bytes(desc), dtype=torch.uint8, device="cuda") for _ in range(2))
    w = torch.zeros(NB, Hkv, 16, device="cuda")
    freqs = torch.from_numpy(pk.rope_frequencies(D)).cuda()
    alloc = pk.Allocator(NB, 16, rng.permutation(NB).astype(np.int32))
    ids = [0, 1, 2]
    place = [0, 0, 0]  # positions go on through evictions
    rows = [[[] for _ in range(Hkv)] for _ in ids]  # (key, value) held by each head
    share = [[[] for _ in range(Hkv)] for _ in ids]
    for s in ids:
        alloc.seq_new(s, 0)

    def append(counts):
        slots, pairs = alloc.append_tokens(ids, counts)
        assert len(pairs) == 0
        T = sum(counts)
        q, k, v = (torch.from_numpy(rng.standard_normal((T, h, D))).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        pos = np.concatenate([np.arange(place[s], place[s] + n) for s, n in zip(ids, counts)])
        q_out = torch.empty_like(q)
        pk.paged_rope_append(q, k, v, i32(pos), torch.from_numpy(slots).cuda(), freqs, kc, vc, desc, q_out)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        pk.paged_kv_read(torch.from_numpy(slots).cuda(), kc, vc, desc, ko, vo)
        at = 0
        for s, n in zip(ids, counts):
            for j in range(n):
                for h in range(Hkv):
                    rows[s][h].append((ko[at + j, h].double().cpu().numpy(), vo[at + j, h].double().cpu().numpy()))
                    share[s][h].append(0.0)
            at += n
            place[s] += n
        return q_out

    def step():
        q = append([1, 1, 1])
        tables, lens = alloc.export(ids, 12)
        out = torch.zeros(3, Hq, D, dtype=dt, device="cuda")
        ws = torch.zeros(pk.decode_scored_workspace_bytes(3, Hq, D, 192, 0, 64, True), dtype=torch.uint8, device="cuda")
        tb, ln, one = i32(tables), i32(lens), i32([1, 1, 1])
        call = lambda: pk.paged_attention_decode_scored(q, kc, vc, desc, tb, ln, 192, D ** -0.5, out, weights=w, new_lens=one,
                                                        workspace=ws, partition_tokens=64)
        if capture:
            keep = w.clone()
            st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=st):
                call()
            w.copy_(keep)
            g.replay()
        else:
            call()
        got = out.double().cpu().numpy()
        for s in ids:
            for h in range(Hkv):
                kk, vv = (np.stack([r[z] for r in rows[s][h]]) for z in (0, 1))
                x = q[s, 4 * h:4 * h + 4].double().cpu().numpy() @ kk.T * D ** -0.5
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                share[s][h] = list(np.array(share[s][h]) + p.sum(0))
                # the coded rows were read back rounded to 16 bits: half a step of bf16 (2^-8 of it) of keys and values
                slack = 0.0 if kv == "bf16" else 2.0 ** -8 * (1 + 2 * np.abs(q[s, 4 * h:4 * h + 4].double().cpu().numpy()).sum(-1).max()
                                                              * np.abs(kk).max() * D ** -0.5) * np.abs(vv).max()
                assert max_error(got[s, 4 * h:4 * h + 4], p @ vv, "bf16", TOL["bf16"] + slack, float(np.abs(vv).max())) <= TOL["bf16"] + slack

    def evict():
        tables, lens = alloc.export(ids, 12)
        kept = torch.zeros(3, Hkv, budget, dtype=torch.int32, device="cuda")
        pk.select_tokens(w, desc, i32(tables), i32(lens), 192, kept, sink_tokens=2, recent_tokens=8)
        before = w.cpu().numpy()
        alloc.evict_batch(ids, [budget] * 3)
        dst, _ = alloc.export(ids, 12)
        pk.paged_kv_compact(kept, kc, vc, desc, i32(tables), i32(lens), i32(dst), weights=w)
        kk = kept.cpu().numpy()
        assert np.array_equal(kk, su.ref_select_tokens(before, tables, lens, budget, 2, 8))
        after = w.cpu().numpy()
        for s in ids:
            n = min(budget, int(lens[s]))
            for h in range(Hkv):
                rows[s][h] = [rows[s][h][t] for t in kk[s, h, :n]]
                share[s][h] = [share[s][h][t] for t in kk[s, h, :n]]
                got = after[dst[s][np.arange(n) // 16], h, np.arange(n) % 16]
                np.testing.assert_allclose(got, share[s][h], rtol=0.05 if kv == "int8" else 2e-3, atol=1e-6)

    append(prompts)
    for _ in range(6):
        step()
    evict()
    assert [alloc.seq_len(s) for s in ids] == [60, 60, 39]
    for _ in range(20):
        step()
    evict()
    for _ in range(3):
        step()
    assert pk.get_device_error() == 0


def test_more_rows_than_a_grid_axis_holds(pk):
    """20000 sequences of 4 heads: 80000 rows, of two tokens each, the second kept."""
    S, Hkv, D = 20000, 4, 64
    desc = pk.CacheDesc(num_blocks=S, num_kv_heads=Hkv, head_size=D, kv_dtype="bf16")
    kc, vc = (torch.randn(S, Hkv, 16, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    w = torch.rand(S, Hkv, 16, device="cuda")
    w0 = w.clone()
    tables = torch.randperm(S, device="cuda").int()[:, None].contiguous()
    lens = torch.full((S,), 2, dtype=torch.int32, device="cuda")
    kept = torch.ones(S, Hkv, 1, dtype=torch.int32, device="cuda")
    pk.paged_kv_compact(kept, kc, vc, desc, tables, lens, tables, weights=w)
    assert pk.get_device_error() == 0
    for new, old in ((kc, k0), (vc, v0), (w, w0)):
        assert torch.equal(new[:, :, 0], old[:, :, 1]) and torch.equal(new[:, :, 1:], old[:, :, 1:])


def test_readme_example_of_an_eviction_runs():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "paged_kv_compact" in c]
    assert len(code) == 1
    e = {}
    exec(compile(code[0], "README.md example", "exec"), e)
    first, k, D = e["kept"][0], e["k_cache"], e["D"]
    assert bool((first[:, 1:] > first[:, :-1]).all()) and first[:, :4].tolist() == [list(range(4))] * e["Hkv"]
    shares = e["weights"][e["dev"](e["fewer"])[0, : e["keep"] // 16].long()]
    # four steps leave Hq each; besides 68 fixed tokens the 444 largest of 1936 stay, which hold at least 444/1936
    assert bool(torch.isfinite(k.float()).all()) and float(shares.sum()) > 0.999 * 4 * e["Hq"] * 444 / 1936
