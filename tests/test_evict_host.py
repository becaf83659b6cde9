"""The allocator's side of eviction against its model, and the refusals of selection and compaction.  CPU only."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.allocator_model import AllocatorModel, OutOfBlocks, prefix_block_hashes


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


def both(pk, NB, order=None):
    return pk.Allocator(NB, 16, order), AllocatorModel(NB, 16, None if order is None else order.tolist())


def same(a, m, seqs):
    for s in seqs:
        assert a.block_table(s) == m.block_table(s) and a.seq_len(s) == m.lens[s]
    assert a.num_free() == m.num_free() and a.num_cached() == m.num_cached()


def test_own_blocks_stay_and_the_rest_is_released(pk):
    a, m = both(pk, 10)
    for x in (a, m):
        x.seq_new(0, 70)
        x.evict_batch([0, -1], [20, 0])
    same(a, m, [0])
    assert len(a.block_table(0)) == 2 and a.num_free() == 8 and a.seq_len(0) == 20
    a.evict_batch([0], [20])  # holds no more than that: as it was
    a.evict_batch([0], [400])
    m.evict_batch([0], [20])
    same(a, m, [0])
    assert a.append_slot(0)[0] == m.append_slot(0)[0]  # the next token follows the kept ones
    for x in (a, m):
        x.evict_batch([0], [0])
    same(a, m, [0])
    assert a.block_table(0) == [] and a.num_free() == 10


def test_shared_and_cached_blocks(pk):
    a, m = both(pk, 12)
    h = prefix_block_hashes(list(range(48)))
    for x in (a, m):
        x.seq_new_prefix(0, np.array(h, np.uint64) if x is a else h, 60)
        x.commit(0, np.array(h, np.uint64) if x is a else h)
        x.fork(0, 1)
        x.seq_new(2, 33)
    before = a.block_table(0), a.block_table(1), a.block_table(2)
    for x in (a, m):
        x.evict_batch([1, 2], [40, 16])
    same(a, m, [0, 1, 2])
    assert a.block_table(0) == before[0] and a.lookup(np.array(h, np.uint64)) == 3  # the other holder's prefix stays cached
    new = a.block_table(1)
    # no block after is one of another sequence's before
    assert not set(new) & (set(before[0]) | set(before[2])) and a.block_table(2) == before[2][:1]
    # alone on cached blocks: they stay, without their hashes
    for x in (a, m):
        x.evict_batch([0], [17])
    same(a, m, [0, 1, 2])
    assert a.block_table(0) == before[0][:2] and a.lookup(np.array(h, np.uint64)) == 0
    for s in (0, 1):
        with pytest.raises(pk.PagedKVError):
            a.commit(s, np.array(h[:1], np.uint64))
    a.fork(1, 5)
    with pytest.raises(pk.PagedKVError):
        a.commit(5, np.array(h[:1], np.uint64))


def test_two_holders_of_one_block_in_one_batch(pk):
    a, m = both(pk, 9)
    for x in (a, m):
        x.seq_new(0, 64)
        x.fork(0, 1)
        x.evict_batch([0, 1], [16, 32])
    same(a, m, [0, 1])
    assert not set(a.block_table(0)) & set(a.block_table(1)) and a.num_free() == 6


def test_all_or_nothing(pk):
    a, _ = both(pk, 6)
    a.seq_new(0, 48)
    a.fork(0, 1)
    a.seq_new(2, 48)
    before = a.block_table(0), a.block_table(1), a.block_table(2), a.num_free()
    state = lambda: (a.block_table(0), a.block_table(1), a.block_table(2), a.num_free())
    with pytest.raises(pk.OutOfBlocks):
        a.evict_batch([2, 0], [16, 32])  # the blocks that 2 gives up come too late for 0
    assert state() == before
    a.free(2)
    a.seq_new(2, 16)
    a.fail_after(2)
    keep = state()
    with pytest.raises(pk.OutOfBlocks):
        a.evict_batch([0], [32])
    assert state() == keep
    for ids, counts, err in (([0, 0], [1, 1], pk.ERR_INVALID), ([7], [1], pk.ERR_NOT_FOUND), ([0], [-1], pk.ERR_INVALID)):
        with pytest.raises(pk.PagedKVError) as e:
            a.evict_batch(ids, counts)
        assert e.value.status == err and state() == keep
    with pytest.raises(ValueError):
        a.evict_batch([0, 1], [1])
    a.evict_batch([], [])


@pytest.mark.parametrize("seed", range(6))
def test_random_streams_match_the_model(pk, seed):
    rng = np.random.default_rng(70 + seed)
    a, m = both(pk, 40, rng.permutation(40).astype(np.int32))
    live, nxt, evicted = [], 0, set()
    h = prefix_block_hashes(list(range(300)))
    for _ in range(250):
        op = rng.random()
        try:
            if op < 0.3:
                n = int(rng.integers(0, 150))
                k = n // 16
                m.seq_new_prefix(nxt, h[:k], n)
                a.seq_new_prefix(nxt, np.array(h[:k], np.uint64), n)
                live.append(nxt)
                nxt += 1
            elif op < 0.4 and live:
                s = int(rng.choice(live))
                m.fork(s, nxt)
                a.fork(s, nxt)
                evicted |= {nxt} if s in evicted else set()
                live.append(nxt)
                nxt += 1
            elif op < 0.55 and live:
                s = int(rng.choice(live))
                if s not in evicted:
                    k = m.lens[s] // 16
                    try:
                        want = m.commit(s, h[:k])
                    except ValueError:
                        continue
                    assert a.commit(s, np.array(h[:k], np.uint64)) == want
            elif op < 0.7 and live:
                s = live.pop(int(rng.integers(0, len(live))))
                m.free_seq(s)
                a.free(s)
            elif op < 0.8 and live:
                s = int(rng.choice(live))
                want = m.append_slot(s)
                assert a.append_slot(s) == want
            elif live:
                pick = [int(s) for s in rng.choice(live, size=min(len(live), int(rng.integers(1, 5))), replace=False)]
                cnt = [int(rng.integers(0, 120)) for _ in pick]
                longer = {s for s, c in zip(pick, cnt) if m.lens[s] > c}
                try:
                    m.evict_batch(pick, cnt)
                except OutOfBlocks:
                    with pytest.raises(pk.OutOfBlocks):
                        a.evict_batch(pick, cnt)
                else:
                    a.evict_batch(pick, cnt)
                    evicted |= longer
        except OutOfBlocks:
            pass
        same(a, m, live)
    for b in range(40):
        assert a.block_hash_of(b) == m.hash_of.get(b) and a.refcount(b) == m.ref[b]


def test_refused_before_any_launch(pk):
    L, at = pk.lib(), 1 << 20  # never followed
    d = lambda D=64, kv="int4": ctypes.byref(pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=D, kv_dtype=kv).c())

    def sel(w=at, D=64, MB=4, mx=64, S=2, n=8, sink=2, rec=3, kept=at, t=at):
        return L.pkv_select_tokens(w, d(D), t, MB, at, mx, S, n, sink, rec, kept, None)

    assert sel(S=0) == pk.OK
    for bad in (dict(S=-1), dict(MB=0), dict(mx=-1), dict(mx=65), dict(n=0), dict(sink=-1), dict(rec=-1), dict(sink=6), dict(w=None),
                dict(kept=None), dict(kept=at + 2), dict(w=at + 1), dict(t=None)):
        assert sel(**bad) == pk.ERR_INVALID, bad
    assert sel(D=96) == pk.ERR_UNSUPPORTED and sel(S=65536) == pk.ERR_UNSUPPORTED
    assert sel(MB=1 << 27, mx=1 << 30) == pk.ERR_UNSUPPORTED and sel(MB=(1 << 27) - 1, mx=(1 << 30) + 1) == pk.ERR_UNSUPPORTED

    def mv(kept=at, n=8, k=at, v=at, w=None, D=64, MB=4, S=2, dst=at, dmb=3):
        return L.pkv_paged_kv_compact(kept, n, k, v, w, d(D), at, MB, at, S, dst, dmb, None)

    assert mv(S=0) == pk.OK
    for bad in (dict(S=-1), dict(n=0), dict(MB=0), dict(dmb=0), dict(kept=None), dict(k=None), dict(v=at + 8), dict(dst=None), dict(w=at + 2)):
        assert mv(**bad) == pk.ERR_INVALID, bad
    assert mv(D=32) == pk.ERR_UNSUPPORTED and mv(dmb=1 << 27) == pk.ERR_UNSUPPORTED and mv(S=1 << 16) == pk.ERR_UNSUPPORTED


def test_operands_refused(pk):
    d = pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=64, kv_dtype="int8")
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    w, pool = torch.zeros(8, 2, 16), torch.zeros(8 * pk.block_bytes(d), dtype=torch.uint8)
    sel = dict(weights=w, desc=d, block_tables=i32(3, 4), seq_lens=i32(3), max_seq_len=64, kept=i32(3, 2, 5))
    with pytest.raises(TypeError, match="CUDA tensor"):
        pk.select_tokens(**sel)
    for bad, err in ((dict(weights=None), TypeError), (dict(kept=i32(3, 1, 5)), ValueError), (dict(kept=i32(2, 2, 5)), ValueError),
                     (dict(block_tables=i32(2, 4)), ValueError), (dict(seq_lens=torch.zeros(3, dtype=torch.int64)), TypeError),
                     (dict(kept=i32(3, 10)), ValueError)):
        with pytest.raises(err):
            pk.select_tokens(**{**sel, **bad})
    mv = dict(kept=i32(3, 2, 5), k_cache=pool, v_cache=pool, desc=d, block_tables=i32(3, 4), seq_lens=i32(3), dst_tables=i32(3, 1))
    with pytest.raises(TypeError, match="CUDA tensor"):
        pk.paged_kv_compact(**mv)
    for bad, err in ((dict(dst_tables=i32(2, 1)), ValueError), (dict(dst_tables=torch.zeros(3, 1)), TypeError), (dict(kept=i32(3, 5, 2)), ValueError)):
        with pytest.raises(err):
            pk.paged_kv_compact(**{**mv, **bad})
