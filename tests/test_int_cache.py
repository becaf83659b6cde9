"""Integer-coded pools and sparse decode on the CPU: sizes, the tile layout's
formulas, and the refusals of every new call and of the calls that got new
pool types.  Nothing here reaches a device: each refused call fails its checks
before any launch (the pointers are never followed)."""
import ctypes

import numpy as np
import pytest

import quant_util as qu

FAKE = 1 << 20


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("value", [False, True])
def test_tile_places_are_a_permutation(D, bits, value):
    rb = D * bits // 8
    assert sorted(qu.places(D, bits, value).reshape(-1).tolist()) == list(range(16 * rb))


def test_block_bytes(pk):
    mk = lambda kv, D=128, H=8, b=16: pk.block_bytes(pk.CacheDesc(num_blocks=4, num_kv_heads=H, head_size=D, kv_dtype=kv, block_size=b))
    for D in (64, 128):
        assert mk("f16", D) == mk("bf16", D) == 8 * 16 * D * 2
        assert mk("e4m3", D) == 8 * 16 * D
        assert mk("int8", D) == 8 * 16 * (D + 8)
        assert mk("int4", D) == 8 * 16 * (D // 2 + 8)
    assert mk("int4", 96) == 0 and mk("int8", b=32) == 0


def test_encode_definition():
    """Constant rows, the range's ends and half-way codes."""
    x = np.zeros((4, 64), np.float32)
    x[1] = 3.5
    x[2, 0], x[2, 1:] = -1.0, 2.0
    x[3] = np.linspace(0, 63, 64)
    for bits in (4, 8):
        code, scale, lo = qu.encode(x, bits)
        assert scale[0] == 0 and scale[1] == 0 and lo[1] == 3.5
        assert code[2].max() == 2 ** bits - 1 and code[2, 0] == 0
        h = qu.held(x, bits)
        assert np.all(h[:2] == x[:2])
        assert np.max(np.abs(h[3] - x[3])) <= 63 / (2 ** bits - 1) / 2 * (1 + 2.0 ** -20)


def test_int_pools_in_the_calls_that_were_there(pk):
    L = pk.lib()
    for kv in ("int8", "int4"):
        d = ctypes.byref(pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=128, kv_dtype=kv).c())
        d96 = ctypes.byref(pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=96, kv_dtype=kv).c())
        dec = lambda desc=d, q_dtype=1, Hq=4, P=0, ws=None, nb=0, q=FAKE: L.pkv_paged_attention_decode(
            q, q_dtype, 2, Hq, FAKE, FAKE, desc, FAKE, 4, FAKE, 64, 0.1, FAKE, ws, nb, P, None)
        assert dec(d96) == pk.ERR_UNSUPPORTED
        assert dec(q_dtype=2) == dec(q_dtype=3) == pk.ERR_INVALID
        assert dec(Hq=6) == pk.ERR_UNSUPPORTED and dec(Hq=5) == pk.ERR_INVALID
        assert dec(q=FAKE + 2) == pk.ERR_INVALID
        assert dec(P=16) == pk.ERR_WORKSPACE
        # append: 16-bit inputs only
        app = lambda in_dtype, desc=d: L.pkv_paged_kv_append(FAKE, FAKE, in_dtype, 4, FAKE, FAKE, FAKE, desc, None)
        assert app(2) == pk.ERR_UNSUPPORTED and app(3) == app(4) == pk.ERR_INVALID and app(1, d96) == pk.ERR_UNSUPPORTED
        # the fused append and cascade decode do not serve integer-coded pools
        assert L.pkv_paged_attention_decode_append(FAKE, FAKE, 1, FAKE, None, FAKE, 1, 2, 4, FAKE, FAKE, d, FAKE, 4, FAKE,
                                                   64, 0.1, FAKE, None, 0, 0, None, 0, None) == pk.ERR_UNSUPPORTED
        assert L.pkv_paged_attention_decode_cascade(FAKE, 1, 2, 8, FAKE, FAKE, d, FAKE, 4, FAKE, 64, FAKE, FAKE, FAKE,
                                                    FAKE, 1, 2, 2, 0.1, FAKE, FAKE, 1 << 30, 16, None) == pk.ERR_UNSUPPORTED
        # prefill stages a 16-bit copy and needs its workspace
        pre = lambda ws, nb: L.pkv_paged_attention_prefill(FAKE, 1, 64, 8, 2, FAKE, 32, FAKE, FAKE, d, FAKE, 4, FAKE, None, 0,
                                                           0.1, FAKE, ws, nb, None)
        need = L.pkv_prefill_workspace_bytes(pk.DTYPE_CODE[kv], 2, 2, 128, 4)
        assert need == L.pkv_prefill_workspace_bytes(pk.FP8_E4M3, 2, 2, 128, 4) > 0
        assert pre(None, 0) == pre(FAKE, need - 1) == pk.ERR_WORKSPACE
    bad = pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=128).c()
    bad.kv_dtype = 5
    assert L.pkv_copy_blocks(FAKE, FAKE, ctypes.byref(bad), FAKE, 1, None) == pk.ERR_INVALID
    assert L.pkv_paged_attention_decode(FAKE, 1, 2, 4, FAKE, FAKE, ctypes.byref(bad), FAKE, 4, FAKE, 64, 0.1, FAKE, None, 0,
                                        0, None) == pk.ERR_INVALID


def desc_of(pk, kv="bf16", **kw):
    base = dict(num_blocks=8, num_kv_heads=2, head_size=128, kv_dtype=kv)
    base.update(kw)
    return pk.CacheDesc(**base).c()


def test_read_refusals(pk):
    L = pk.lib()

    def call(desc=None, T=4, slots=FAKE, kc=FAKE, ko=FAKE, out=1):
        return L.pkv_paged_kv_read(slots, T, kc, FAKE, ctypes.byref(desc or desc_of(pk)), ko, FAKE, out, None)

    assert call(T=-1) == pk.ERR_INVALID and call(T=0, slots=None) == pk.OK
    assert call(out=2) == call(out=3) == pk.ERR_INVALID
    assert call(out=0) == pk.ERR_UNSUPPORTED                      # f16 values of a bf16 pool
    assert call(desc_of(pk, head_size=96)) == pk.ERR_UNSUPPORTED
    assert call(desc_of(pk, block_size=32)) == pk.ERR_UNSUPPORTED
    assert call(desc_of(pk, "e4m3", k_scale=0.0)) == pk.ERR_INVALID
    assert call(slots=FAKE + 4) == call(kc=FAKE + 8) == call(ko=FAKE + 2) == call(kc=None) == pk.ERR_INVALID
    assert L.pkv_paged_kv_read(FAKE, 4, FAKE, FAKE, None, FAKE, FAKE, 1, None) == pk.ERR_INVALID


def test_bounds_refusals(pk):
    L = pk.lib()

    def call(desc=None, MB=4, S=2, new=FAKE, max_new=8, bounds=FAKE, dt=1, kc=FAKE):
        return L.pkv_paged_key_bounds(kc, ctypes.byref(desc or desc_of(pk)), FAKE, MB, FAKE, new, max_new, S, bounds, dt, None)

    assert call(S=0) == call(max_new=0) == pk.OK
    assert call(S=-1) == call(MB=0) == call(max_new=-1) == call(max_new=65) == pk.ERR_INVALID
    assert call(dt=2) == call(dt=4) == pk.ERR_INVALID
    assert call(dt=0) == pk.ERR_UNSUPPORTED                       # f16 bounds of a bf16 pool
    assert call(desc_of(pk, head_size=96)) == call(S=65536) == pk.ERR_UNSUPPORTED
    assert call(bounds=None) == call(bounds=FAKE + 8) == call(kc=FAKE + 4) == call(new=FAKE + 2) == pk.ERR_INVALID
    assert call(desc_of(pk, "e4m3", k_scale=-1.0)) == pk.ERR_INVALID


def test_select_refusals(pk):
    L = pk.lib()
    need = pk.select_blocks_workspace_bytes(2, 2, 64)
    assert need > 0 and pk.select_blocks_workspace_bytes(-1, 2, 64) == 0 and pk.select_blocks_workspace_bytes(2, 0, 64) == 0

    def call(desc=None, q=FAKE, dt=1, S=2, Hq=8, MB=4, max_len=64, n=3, sink=1, recent=1, ws=FAKE, nb=need, sel=FAKE):
        return L.pkv_select_blocks(q, dt, S, Hq, FAKE, ctypes.byref(desc or desc_of(pk)), FAKE, MB, FAKE, max_len, n, sink,
                                   recent, sel, ws, nb, None)

    assert call(S=0) == pk.OK
    assert call(n=0) == call(sink=-1) == call(recent=-1) == call(sink=2, recent=2) == pk.ERR_INVALID
    assert call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == pk.ERR_INVALID
    assert call(max_len=65) == call(max_len=-1) == call(MB=0) == call(dt=2) == pk.ERR_INVALID
    assert call(Hq=6) == pk.ERR_UNSUPPORTED and call(Hq=5) == call(Hq=0) == pk.ERR_INVALID
    assert call(dt=0) == pk.ERR_UNSUPPORTED
    assert call(MB=2 ** 28) == pk.ERR_UNSUPPORTED                 # positions past 32 bits
    assert call(q=FAKE + 2) == call(sel=FAKE + 2) == call(sel=None) == pk.ERR_INVALID
    assert call(ws=None) == call(nb=need - 1) == pk.ERR_WORKSPACE


def test_sparse_refusals(pk):
    L = pk.lib()

    def call(desc=None, q=FAKE, dt=1, S=2, Hq=8, MB=4, n=4, scale=0.1, out=FAKE, ws=None, nb=0, part=0, sel=FAKE):
        return L.pkv_paged_attention_decode_sparse(q, dt, S, Hq, FAKE, FAKE, ctypes.byref(desc or desc_of(pk)), FAKE, MB, FAKE,
                                                   sel, n, scale, out, ws, nb, part, None)

    assert call(S=0) == pk.OK
    assert call(n=0) == call(n=-1) == call(part=-1) == call(scale=float("nan")) == call(dt=3) == pk.ERR_INVALID
    assert call(Hq=6) == call(dt=0) == call(desc_of(pk, head_size=96)) == pk.ERR_UNSUPPORTED
    assert call(q=FAKE + 8) == call(out=None) == call(sel=FAKE + 1) == call(MB=0) == pk.ERR_INVALID
    assert call(n=2 ** 28) == call(part=2 ** 28) == pk.ERR_INVALID
    need = pk.decode_sparse_workspace_bytes(2, 8, 128, 4, 1)
    assert need > 0 and pk.decode_sparse_workspace_bytes(2, 8, 128, 16, 0) == 0
    assert pk.decode_sparse_workspace_bytes(2, 8, 128, 17, 0) == pk.decode_sparse_workspace_bytes(2, 8, 128, 17, 8) > 0
    # 50 sequences x 4 partitions of eight blocks are more than one CTA an SM: sixteen
    assert pk.decode_sparse_workspace_bytes(50, 8, 128, 32, 0) == pk.decode_sparse_workspace_bytes(50, 8, 128, 32, 16)
    assert pk.decode_sparse_workspace_bytes(38, 8, 128, 32, 0) == pk.decode_sparse_workspace_bytes(38, 8, 128, 32, 8)
    small = pk.decode_sparse_workspace_bytes(2, 8, 128, 17, 16)
    assert call(n=17) == call(n=17, ws=FAKE, nb=small - 1) == call(n=17, ws=FAKE + 4, nb=small) == pk.ERR_WORKSPACE
    assert call(part=1) == call(part=1, ws=FAKE, nb=need - 1) == call(part=1, ws=FAKE + 4, nb=need) == pk.ERR_WORKSPACE
    for kv in ("int8", "int4"):
        assert call(desc_of(pk, kv), dt=2) == pk.ERR_INVALID
        assert call(desc_of(pk, kv), part=1) == pk.ERR_WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_shapes(pk):
    import torch
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype="int8")
    z = torch.zeros(1)
    with pytest.raises(TypeError):
        pk.paged_kv_read(torch.zeros(3, dtype=torch.int32), z, z, d, z, z)
    with pytest.raises(ValueError):
        pk.paged_kv_read(torch.zeros(3, dtype=torch.int64), z, z, d, torch.zeros(2, 2, 64, dtype=torch.bfloat16), z)
    with pytest.raises(ValueError):
        pk.paged_key_bounds(z, d, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), None, 4,
                            torch.zeros(4, 2, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        pk.select_blocks(torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 2, 64, dtype=torch.float16), d,
                         torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 64,
                         torch.zeros(2, 2, 3, dtype=torch.int32), z)
    with pytest.raises(ValueError):
        pk.paged_attention_decode_sparse(torch.zeros(2, 4, 64, dtype=torch.bfloat16), z, z, d,
                                         torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                                         torch.zeros(2, 3, 3, dtype=torch.int32), 0.1,
                                         torch.zeros(2, 4, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_binding_refuses_short_operands_of_coded_pools(pk, kv):
    """Rows that the tensors do not hold are refused before anything is launched; sound ones get as far as the
    check for CUDA tensors."""
    import torch
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype=kv)
    pool = torch.zeros(4 * pk.block_bytes(d), dtype=torch.uint8)
    rows = lambda n, h=2, dt=torch.bfloat16: torch.zeros(n, h, 64, dtype=dt)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)

    def append(k=rows(3), v=rows(3)):
        pk.paged_kv_append(k, v, torch.zeros(3, dtype=torch.int64), pool, pool, d)

    def decode(q=rows(3, 4), out=rows(3, 4), tables=i32(3, 4), lens=i32(3)):
        pk.paged_attention_decode(q, pool, pool, d, tables, lens, 64, 0.1, out)

    for call, bad in ((append, dict(k=rows(2))), (append, dict(v=rows(3, 1))), (append, dict(v=rows(3, dt=torch.float16))),
                      (decode, dict(out=rows(3, 2))), (decode, dict(out=rows(3, 4, torch.float16))),
                      (decode, dict(tables=i32(2, 4))), (decode, dict(lens=i32(2)))):
        with pytest.raises(ValueError):
            call(**bad)
    for call in (append, decode):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="CUDA tensor"):  # longer ones hold the rows
        append(k=rows(5))
