"""Refusals of scored attention: nothing here reaches a device, each call fails a check before any launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


AT = 1 << 20  # never followed


def mod(pk, **k):
    m = dict(cap=0.0, window=0, slopes=None, first=None, prefix_lens=None, **{}) | k
    return ctypes.byref(pk._ScoreMod(m["cap"], m["window"], m["slopes"], m["first"], m["prefix_lens"]))


BAD_MODS = [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=2.0 ** -21), dict(cap=2.0 ** 21), dict(window=-1),
            dict(slopes=AT + 2), dict(first=AT + 1)]


def test_scored_decode_refused(pk):
    L = pk.lib()

    def call(m=None, kv="bf16", S=2, Hq=4, D=128, MB=4, mx=64, scale=0.1, w=None, new=None, ws=AT, n=1 << 30, part=0, q=AT, dt=1, **k):
        d = pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=D, kv_dtype=kv, **k).c()
        return L.pkv_paged_attention_decode_scored(q, dt, S, Hq, AT, AT, ctypes.byref(d), AT, MB, AT, mx, scale, m, w, new, AT, ws, n,
                                                   part, None)

    assert call(S=0) == pk.OK and call(S=0, m=mod(pk, cap=2.0 ** -20, window=5, slopes=AT, first=AT)) == pk.OK
    for bad in BAD_MODS + [dict(prefix_lens=AT)]:
        assert call(m=mod(pk, **bad)) == pk.ERR_INVALID, bad
    assert call(m=mod(pk, cap=2.0 ** -20), scale=1e35) == pk.ERR_INVALID  # the products' factor is not finite
    assert call(new=AT) == pk.ERR_INVALID                                  # new lengths without weights
    assert call(w=AT + 2) == pk.ERR_INVALID and call(w=AT, new=AT + 1) == pk.ERR_INVALID
    assert call(D=96) == pk.ERR_UNSUPPORTED and call(Hq=6) == pk.ERR_UNSUPPORTED and call(Hq=5) == pk.ERR_INVALID
    assert call(dt=0) == pk.ERR_UNSUPPORTED and call(mx=65) == pk.ERR_INVALID and call(part=24) == pk.ERR_INVALID
    assert call(q=AT + 8) == pk.ERR_INVALID and call(kv="e4m3", k_scale=0.0) == pk.ERR_INVALID
    assert call(MB=1 << 27) == pk.ERR_UNSUPPORTED and call(MB=(1 << 27) - 1, part=64, n=1 << 40, mx=64) == pk.ERR_UNSUPPORTED
    assert call(MB=1 << 26, mx=1 << 30, w=AT) == pk.ERR_WORKSPACE and call(MB=1 << 27 >> 1 | 1, mx=(1 << 30) + 1, w=AT) == pk.ERR_UNSUPPORTED
    # the workspace: partials of split rows, and with weights those of every row and the scores
    assert call(part=16, ws=None) == pk.ERR_WORKSPACE and call(w=AT, ws=None) == pk.ERR_WORKSPACE
    for window, part, weights in ((0, 16, 0), (0, 16, 1), (0, 0, 1), (20, 16, 1)):
        need = L.pkv_decode_scored_workspace_bytes(2, 4, 128, 64, window, part or 256, weights)
        assert need > 0
        assert call(m=mod(pk, window=window), part=part, w=AT if weights else None, n=need - 1) == pk.ERR_WORKSPACE


def test_scored_workspace_arithmetic(pk):
    size = pk.decode_scored_workspace_bytes
    up = lambda x: -(-x // 256) * 256
    part = lambda rows, D: 2 * up(4 * rows) + 4 * rows * D
    assert size(3, 8, 128, 500, 0, 512) == 0 and size(3, 8, 128, 0, 0, 16, True) == 0
    assert size(3, 8, 128, 500, 0, 64) == part(24 * 8, 128)            # 512 tokens in whole blocks, 8 partitions
    assert size(3, 8, 128, 500, 0, 64, True) == up(part(24 * 8, 128)) + 24 * 512 * 4
    assert size(3, 8, 64, 5000, 100, 64) == part(24 * 2, 64)           # a window of 100 touches up to 8 blocks
    assert size(3, 8, 64, 5000, 100, 0) == 0                           # one partition
    assert size(3, 8, 64, 5000, 0, 0, True) == size(3, 8, 64, 5000, 0, 256, True)
    for bad in (dict(num_seqs=-1), dict(num_q_heads=0), dict(head_size=0), dict(max_seq_len=-1), dict(window=-1), dict(partition_tokens=24)):
        assert size(**{**dict(num_seqs=3, num_q_heads=8, head_size=64, max_seq_len=500, window=0, partition_tokens=64), **bad}) == 0


def test_scored_prefill_refused(pk):
    L = pk.lib()

    def call(m=None, T=64, S=2, Hq=8, scale=0.1, mq=32, q=AT, D=128, kv="bf16", dt=1, ws=None, n=0, **k):
        d = pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=D, kv_dtype=kv, **k).c()
        return L.pkv_paged_attention_prefill_scored(q, dt, T, Hq, S, AT, mq, AT, AT, ctypes.byref(d), AT, 4, AT, None, 0, scale, m, AT,
                                                    ws, n, None)

    assert call(S=0) == pk.OK and call(T=0) == pk.OK and call(mq=0, m=mod(pk, prefix_lens=AT, first=AT)) == pk.OK
    for bad in BAD_MODS + [dict(prefix_lens=AT + 2)]:
        assert call(m=mod(pk, **bad)) == pk.ERR_INVALID, bad
    assert call(m=mod(pk, cap=2.0 ** -20), scale=1e35) == pk.ERR_INVALID
    assert call(scale=0.0) == pk.ERR_INVALID and call(q=AT + 8) == pk.ERR_INVALID and call(Hq=5) == pk.ERR_INVALID
    assert call(D=96) == pk.ERR_UNSUPPORTED and call(Hq=6) == pk.ERR_UNSUPPORTED and call(dt=0) == pk.ERR_UNSUPPORTED
    assert call(kv="int4") == pk.ERR_WORKSPACE and call(kv="e4m3", v_scale=-1.0, ws=AT, n=1 << 30) == pk.ERR_INVALID


def test_operands_refused(pk):
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype="bf16")
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    rows = lambda n, h=4, dt=torch.bfloat16: torch.zeros(n, h, 64, dtype=dt)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    dec = dict(q=rows(3), k_cache=pool, v_cache=pool, desc=d, block_tables=i32(3, 4), seq_lens=i32(3), max_seq_len=64, scale=0.1,
               out=rows(3))
    pre = dict(q=rows(9), k_cache=pool, v_cache=pool, desc=d, query_start=i32(4), max_query_len=3, block_tables=i32(3, 4),
               seq_lens=i32(3), scale=0.1, out=rows(9))
    for call, good, n in ((pk.paged_attention_decode_scored, dec, 3), (pk.paged_attention_prefill_scored, pre, 9)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call(**good)
        for bad in (dict(out=rows(n - 1)), dict(out=rows(n, 2)), dict(out=rows(n, dt=torch.float16)), dict(block_tables=i32(2, 4)),
                    dict(block_tables=i32(12)), dict(seq_lens=i32(2)), dict(q=torch.zeros(n, 4, 32, dtype=torch.bfloat16))):
            with pytest.raises(ValueError):
                call(**{**good, **bad})
        for name in ("block_tables", "seq_lens"):
            with pytest.raises(TypeError):
                call(**{**good, name: good[name].long()})
    for bad in (dict(k_cache=pool[:3]), dict(v_cache=pool[:3]), dict(query_start=i32(3)), dict(score=pk.ScoreMod(slopes=torch.zeros(3))),
                dict(score=pk.ScoreMod(first=i32(3))), dict(score=pk.ScoreMod(first=torch.zeros(9))), dict(score=pk.ScoreMod(prefix_lens=i32(9)))):
        with pytest.raises(ValueError):
            pk.paged_attention_prefill_scored(**{**pre, **bad})
    with pytest.raises(TypeError):
        pk.paged_attention_prefill_scored(**{**pre, "query_start": torch.zeros(4, dtype=torch.int64)})


def test_sources_read_live_what_earlier_kernels_write():
    """The rules of tests/test_kernel_sources.py for what the newer kernels call after their wait."""
    from test_kernel_sources import functions
    found = {n: body for _, n, _, body in functions()
             if n in ("scored_row", "scored_slope", "row_range", "scored_unit", "load_key", "move_rows", "rotation")}
    assert len(found) == 7
    assert not any("__ldg(" in body for body in found.values())
