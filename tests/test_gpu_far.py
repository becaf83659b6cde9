"""Rotary append, shares, scored attention and eviction where offsets pass 32 bits: pools of more than 4 GiB, more than
2^31 kept scores; and a captured eviction."""
import numpy as np
import pytest
import torch

import quant_util as qu
import score_util as su
from parity_util import TOL, max_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    yield pagedkv
    torch.cuda.empty_cache()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_blocks_past_4_gib(pk, kv):
    """A sequence whose blocks lie at both ends of the pools, written, attended to, evicted, moved."""
    pk.get_device_error()
    rng = np.random.default_rng(0)
    Hq, Hkv, D, L, keep = 32, 8, 128, 180, 70
    NB = (5 << 30) // (Hkv * 16 * D * (2 if kv == "bf16" else 1))
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv)
    assert NB * pk.block_bytes(desc) > 1 << 32
    kc, vc = (torch.zeros(NB * pk.block_bytes(desc), dtype=torch.uint8, device="cuda") for _ in range(2))
    w = torch.zeros(NB, Hkv, 16, device="cuda")
    table = np.array([[NB - 1 - 3 * i if i % 2 else i for i in range(12)]], np.int32)
    at = np.arange(L)
    slots = torch.from_numpy(table[0][at // 16].astype(np.int64) * 16 + at % 16).cuda()
    q, k, v = (torch.from_numpy(rng.standard_normal((L, h, D))).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    freqs = torch.from_numpy(pk.rope_frequencies(D)).cuda()
    qr = torch.empty_like(q)
    pk.paged_rope_append(q, k, v, i32(at), slots, freqs, kc, vc, desc, qr)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    pk.paged_kv_read(slots, kc, vc, desc, ko, vo)
    f8 = lambda t: t.double().cpu().numpy()
    kk, vv, qq = f8(ko), f8(vo), f8(qr)
    # int8 rows are read back rounded to bf16: half a step (2^-8) of keys and values, in the scores and the outputs
    slack = 0.0 if kv == "bf16" else 2.0 ** -8 * (1 + 2 * np.abs(qq).sum(-1).max() * np.abs(kk).max() * D ** -0.5) * np.abs(vv).max()

    def attend(row, n0, n1, kk, vv, h):
        x = qq[row, 4 * h:4 * h + 4] @ kk[n0:n1, h].T * D ** -0.5
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        return p @ vv[n0:n1, h], p

    tb = i32(table)
    out = torch.zeros_like(q)
    ws = torch.zeros(max(pk.prefill_workspace_bytes(kv, 1, Hkv, D, 12), pk.decode_scored_workspace_bytes(1, Hq, D, L, 0, 64, True)),
                     dtype=torch.uint8, device="cuda")
    pk.paged_attention_prefill_scored(qr, kc, vc, desc, i32([0, L]), L, tb, i32([L]), D ** -0.5, out, pk.ScoreMod(window=100), workspace=ws)
    one = torch.zeros(1, Hq, D, dtype=q.dtype, device="cuda")
    pk.paged_attention_decode_scored(qr[L - 1:].contiguous(), kc, vc, desc, tb, i32([L]), L, D ** -0.5, one, weights=w, workspace=ws,
                                     partition_tokens=64)
    kept = torch.zeros(1, Hkv, keep, dtype=torch.int32, device="cuda")
    pk.select_tokens(w, desc, tb, i32([L]), L, kept, 4, 8)
    host_w = w[tb[0].long()].cpu().numpy()
    near = np.arange(12, dtype=np.int32)[None]
    assert np.array_equal(kept.cpu().numpy(), su.ref_select_tokens(host_w, near, [L], keep, 4, 8))
    share = host_w[at // 16, :, at % 16]
    for h in range(Hkv):
        ref, p = attend(L - 1, 0, L, kk, vv, h)
        assert max_error(f8(one)[0, 4 * h:4 * h + 4], ref, "bf16", TOL["bf16"] + slack, np.abs(vv).max()) <= TOL["bf16"] + slack
        assert np.allclose(share[:, h], p.sum(0), rtol=2e-3 if kv == "bf16" else 0.05, atol=1e-6)
        for row in (5, 130, L - 1):
            ref, _ = attend(row, max(0, row - 99), row + 1, kk, vv, h)
            assert max_error(f8(out)[row, 4 * h:4 * h + 4], ref, "bf16", TOL["bf16"] + 2 * slack, np.abs(vv).max()) <= TOL["bf16"] + 2 * slack
    dst = np.array([[NB - 2, 1, NB - 5, 3, NB - 8]], np.int32)  # none of the table's
    assert not set(dst[0]) & set(table[0])
    pk.paged_kv_compact(kept, kc, vc, desc, tb, i32([L]), i32(dst), weights=w)
    i = np.arange(keep)
    moved = torch.from_numpy(dst[0][i // 16].astype(np.int64) * 16 + i % 16).cuda()
    k2, v2 = (torch.zeros(keep, Hkv, D, dtype=q.dtype, device="cuda") for _ in range(2))
    pk.paged_kv_read(moved, kc, vc, desc, k2, v2)
    for h in range(Hkv):
        src = kept[0, h].long()
        assert torch.equal(k2[:, h], ko[src, h]) and torch.equal(v2[:, h], vo[src, h])
        assert np.array_equal(w[dst[0][i // 16], h, i % 16].cpu().numpy(), share[kept[0, h].cpu().numpy(), h])
    assert pk.get_device_error() == 0


def test_more_than_2_31_kept_scores(pk):
    """Many long rows over a few shared blocks; the last row, whose scores lie past 2^31 of them, has its own."""
    pk.get_device_error()
    rng = np.random.default_rng(1)
    S, Hq, Hkv, D, mx = 70, 64, 8, 64, 1 << 19
    rows = [3000] * (S - 1) + [777]
    NB = 240
    pools = qu.Pools(rng, NB, Hkv, D, "f16")
    kd, vd = pools.dev()
    tables = np.zeros((S, mx // 16), np.int32)
    tables[:, :188] = rng.integers(0, 180, (S, 188))
    tables[-1, :49] = np.arange(185, 234)
    q = qu.queries(rng, S, Hq, D, "f16", 2.0)
    assert (S - 1) * Hq * mx > 1 << 31
    ws = torch.empty(pk.decode_scored_workspace_bytes(S, Hq, D, mx, 0, 4096, True), dtype=torch.uint8, device="cuda")
    w, out = torch.zeros(NB, Hkv, 16, device="cuda"), torch.zeros_like(q, device="cuda")
    pk.paged_attention_decode_scored(q.cuda(), kd, vd, pools.desc, i32(tables), i32(rows), mx, D ** -0.5, out, weights=w, workspace=ws,
                                     partition_tokens=4096)
    assert pk.get_device_error() == 0
    ref, shares = su.ref_scored(q[-1:], [(S - 1, 776)], pools, tables, rows, D ** -0.5)
    got = out[-1:].double().cpu().numpy()
    assert max_error(got, ref, "f16", TOL["f16"], float(np.abs(pools.vh).max())) <= TOL["f16"]
    want, step = su.ref_weights(np.zeros((NB, Hkv, 16), np.float32), shares, tables[-1:], rows[-1:], None, Hkv)
    mine = slice(185, 234)
    tol = su.share_bound(q, pools, D ** -0.5, 0.0, None, 777) * step + 8 * 2.0 ** -118
    assert np.all(np.abs(w.double().cpu().numpy() - want)[mine] <= tol[mine])


def test_an_eviction_captured_and_replayed(pk):
    pk.get_device_error()
    rng = np.random.default_rng(2)
    lens, n = [300, 40, 511], 64
    NB, tables = qu.make_tables(rng, lens)
    pools = qu.Pools(rng, NB, 2, 64, "bf16")
    kd, vd = pools.dev()
    k0, v0 = kd.clone(), vd.clone()
    w = torch.zeros(NB, 2, 16, device="cuda")
    kept = torch.zeros(3, 2, n, dtype=torch.int32, device="cuda")
    tb, ln = i32(tables), i32(lens)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        pk.select_tokens(w, pools.desc, tb, ln, 511, kept, 2, 10)
        pk.paged_kv_compact(kept, kd, vd, pools.desc, tb, ln, tb, weights=w)
    for seed in (5, 6):
        w0 = np.random.default_rng(seed).random((NB, 2, 16)).astype(np.float32)
        w.copy_(torch.from_numpy(w0))
        kd.copy_(k0)
        vd.copy_(v0)
        g.replay()
        torch.cuda.synchronize()
        ref = su.ref_select_tokens(w0, tables, lens, n, 2, 10)
        assert np.array_equal(kept.cpu().numpy(), ref)
        for s, L in enumerate(lens):
            for h in range(2):
                src, i = ref[s, h][ref[s, h] >= 0], np.arange(min(n, L))
                for new, old in ((kd, k0), (vd, v0), (w, torch.from_numpy(w0).cuda())):
                    assert torch.equal(new[tables[s][i // 16], h, i % 16], old[tables[s][src // 16], h, src % 16])
    assert pk.get_device_error() == 0
