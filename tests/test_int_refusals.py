"""Refusals on the CPU of calls whose operands do not hold what the kernels would read or write: nothing here
reaches a device, each call fails a check before any launch."""
import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3", "int8", "int4"])
def test_swap_refuses_host_pools_that_do_not_hold_the_blocks(pk, kv):
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype=kv)
    nbytes = pk.block_bytes(d)
    device = torch.zeros(4, nbytes, dtype=torch.uint8)
    host = lambda n=3, b=nbytes: torch.zeros(n, b, dtype=torch.uint8)
    swap = lambda k, v: pk.swap_blocks(device, device, d, k, v, i32(1, 2), pk.SWAP_OUT)
    for k, v in ((host(b=nbytes - 16), host()), (host(), host(b=nbytes - 16)), (host(), host(2))):
        with pytest.raises(ValueError, match="must hold 3 blocks"):
            swap(k, v)
    if kv == "int8":  # one byte an element leaves no room for the rows' scales and zeros
        with pytest.raises(ValueError, match="must hold 3 blocks"):
            swap(*(torch.zeros(3, 2, 16, 64, dtype=torch.uint8) for _ in range(2)))
    with pytest.raises(ValueError, match="pinned"):  # the right size gets as far as the next check
        swap(host(), host())


@pytest.mark.parametrize("kv", ["int8", "int4"])
def test_noalloc_decode_and_prefill_refuse_what_decode_refuses(pk, kv):
    """Short, mixed and foreign operands of the calls over coded pools that are marshalled in Python; sound ones get
    as far as the check for CUDA tensors."""
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype=kv)
    pool = torch.zeros(4 * pk.block_bytes(d), dtype=torch.uint8)
    rows = lambda n, h=4, dt=torch.bfloat16: torch.zeros(n, h, 64, dtype=dt)

    def noalloc(q=rows(3), out=rows(3), tables=i32(3, 4), lens=i32(3), k=pool):
        pk.paged_attention_decode_noalloc(q, k, pool, d, tables, lens, 64, 0.1, out)

    def prefill(q=rows(9), out=rows(9), start=i32(4), tables=i32(3, 4), lens=i32(3), k=pool, work=None):
        pk.paged_attention_prefill(q, k, pool, d, start, 3, tables, lens, 0.1, out, work_units=work)

    for call, n in ((noalloc, 3), (prefill, 9)):
        for bad in (dict(out=rows(n - 1)), dict(out=rows(n, 2)), dict(out=rows(n, dt=torch.float16)), dict(tables=i32(2, 4)),
                    dict(tables=i32(12)), dict(k=pool[:-16]), dict(q=torch.zeros(n, 4, 64, dtype=torch.uint8),
                                                                    out=torch.zeros(n, 4, 64, dtype=torch.uint8))):
            with pytest.raises(ValueError):
                call(**bad)
        with pytest.raises(TypeError, match="must be int32"):
            call(tables=torch.zeros(3, 4, dtype=torch.int64))
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError):
        noalloc(lens=i32(2))
    with pytest.raises(ValueError):
        prefill(start=i32(3))
    for bad in (dict(start=torch.zeros(4, dtype=torch.int64)), dict(work=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError, match="must be int32"):
            prefill(**bad)


def test_operands_on_another_device_are_refused(pk, monkeypatch):
    """With stand-ins for tensors of a second device: nothing here needs one."""
    class On:
        is_cuda, dtype, nbytes, shape = True, torch.bfloat16, 3 * 4 * 64 * 2, (3, 4, 64)

        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

        def dim(self):
            return 2

        def numel(self):
            return 3

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype="int8")
    sound = dict(q=On(0), out=On(0), num_seqs=3, block_tables=On(0), seq_lens=On(0), k_cache=On(0), workspace=None)
    pk._int_operands(d, **sound)
    for n in ("q", "out", "block_tables", "seq_lens", "k_cache", "workspace"):
        with pytest.raises(ValueError, match=f"{n} is on cuda:1"):
            pk._int_operands(d, **{**sound, n: On(1)})


@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_selection_and_sparse_decode_refuse_elements_that_are_not_16_bits(pk, kv):
    """A type declared by name does not make a tensor of bytes hold as many elements as its shape says."""
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=2, head_size=64, kv_dtype=kv)
    tables, lens, sel = i32(3, 4), i32(3), i32(3, 2, 2)
    pool = torch.zeros(4 * pk.block_bytes(d), dtype=torch.uint8)
    for dt, err in ((torch.uint8, "16-bit"), (torch.float32, "16-bit"), (torch.int16, "CUDA tensor")):
        q, bounds = torch.zeros(3, 4, 64, dtype=dt), torch.zeros(4, 2, 2, 64, dtype=dt)
        with pytest.raises(TypeError, match=err):
            pk.select_blocks(q, bounds, d, tables, lens, 64, sel, None, q_dtype="bf16")
        with pytest.raises(TypeError, match=err):
            pk.paged_attention_decode_sparse(q, pool, pool, d, tables, lens, sel, 0.1, q, q_dtype="bf16")
        with pytest.raises(TypeError, match=err):
            pk.paged_key_bounds(pool, d, tables, lens, None, 64, bounds, bounds_dtype="bf16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8", "int4"])
def test_decode_refuses_positions_past_32_bits(pk, kv):
    import ctypes
    L = pk.lib()
    at = 1 << 20  # never followed
    d = ctypes.byref(pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=128, kv_dtype=kv).c())
    call = lambda MB, mx, P: L.pkv_paged_attention_decode(at, 1, 2, 4, at, at, d, at, MB, at, mx, 0.1, at, at, 1 << 40, P, None)
    assert call(2 ** 27, 64, 0) == pk.ERR_UNSUPPORTED                       # 2^31 tokens of table
    assert call(2 ** 27 - 1, 2 ** 31 - 16, 2 ** 30 + 16) == pk.ERR_UNSUPPORTED  # two partitions end past 2^31


def test_copy_and_swap_refuse_lists_without_the_pairs(pk, monkeypatch):
    d = pk.CacheDesc(num_blocks=4, num_kv_heads=1, head_size=64, kv_dtype="int8")
    pool = torch.zeros(4, pk.block_bytes(d), dtype=torch.uint8)
    for pairs, n in ((i32(6), None), (i32(2, 2), 3), (i32(3), 2)):
        with pytest.raises(ValueError, match="pairs"):
            pk.copy_blocks(pool, pool, d, pairs, n)
    with pytest.raises(TypeError, match="CUDA tensor"):
        pk.copy_blocks(pool, pool, d, i32(6), 3)
    monkeypatch.setattr(torch.Tensor, "is_pinned", lambda t: True)
    for pairs in (i32(6), torch.zeros(3, 2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="pairs"):
            pk.swap_blocks(pool, pool, d, pool, pool, pairs, pk.SWAP_OUT)
    with pytest.raises(TypeError, match="CUDA tensor"):
        pk.swap_blocks(pool, pool, d, pool, pool, i32(3, 2), pk.SWAP_OUT)
