"""Rotary frequencies on the host, against their formulas in 64 bits, and what is refused before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    return pagedkv


def turns(f):
    return f.astype(np.float64).sum(-1)


@pytest.mark.parametrize("R,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0), (2, 10.0)])
def test_frequencies(pk, R, base):
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)
    close = lambda got, want: np.testing.assert_allclose(turns(got), want / (2 * math.pi), rtol=2.0 ** -47, atol=0)
    close(pk.rope_frequencies(R, base), f)
    close(pk.rope_frequencies(R, base, "linear", 8.0), f / 8)
    if R >= 4:
        close(pk.rope_frequencies(R, base, "ntk", 4.0), (base * 4.0 ** (R / (R - 2))) ** (-2.0 * i / R))
    for low, high, L0, s in ((1.0, 32.0, 4096, 16.0), (1.0, 4.0, 8192, 8.0)):
        want = []
        for x in f:  # by wavelengths: short ones stay, long ones are divided, a ramp between
            r = L0 / (2 * math.pi / x)
            g = 0.0 if r < low else 1.0 if r > high else (r - low) / (high - low)
            want.append(g * x + (1 - g) * x / s)
        close(pk.rope_frequencies(R, base, "parts", s, L0, low, high), np.array(want))


def test_frequencies_refused(pk):
    L = pk.lib()
    out = np.zeros((64, 2), np.float32).ctypes.data_as(ctypes.c_void_p)
    call = lambda R=64, base=1e4, kind=0, factor=1.0, L0=0, lo=1.0, hi=32.0, o=out: L.pkv_rope_frequencies(R, base, kind, factor, L0, lo, hi, o)
    assert call() == pk.OK
    for bad in (dict(R=0), dict(R=7), dict(base=1.0), dict(base=float("nan")), dict(kind=4), dict(kind=-1), dict(o=None),
                dict(kind=1, factor=0.5), dict(kind=1, factor=float("inf")), dict(kind=2, R=2, factor=2.0), dict(kind=3, L0=0),
                dict(kind=3, L0=10, lo=4.0, hi=4.0)):
        assert call(**bad) == pk.ERR_INVALID, bad
    with pytest.raises(ValueError):
        pk.rope_frequencies(7)
    with pytest.raises(KeyError):
        pk.rope_frequencies(64, scaling="other")


def test_rope_append_refused_before_any_launch(pk):
    L, at = pk.lib(), 1 << 20  # never followed

    def call(kv="bf16", q=at, qs=512, Hq=4, ks=256, vs=256, dt=1, T=3, R=128, m=1.0, o=at, os=512, D=128, k=at, pos=at, freqs=at):
        d = pk.CacheDesc(num_blocks=8, num_kv_heads=2, head_size=D, kv_dtype=kv).c()
        return L.pkv_paged_rope_append(q, qs, Hq, k, ks, at, vs, dt, T, pos, at, freqs, R, 0, m, at, at, ctypes.byref(d), o, os, None)

    assert call(T=0) == pk.OK
    for bad in (dict(T=-1), dict(Hq=-1), dict(R=0), dict(R=8), dict(R=144), dict(R=20), dict(m=float("nan")), dict(m=float("inf")),
                dict(qs=508), dict(ks=255), dict(ks=128), dict(vs=0), dict(q=None), dict(o=None), dict(q=at + 8), dict(o=at + 8),
                dict(os=256), dict(k=None), dict(k=at + 2), dict(pos=None), dict(pos=at + 2), dict(freqs=at + 4), dict(dt=2), dict(dt=7)):
        assert call(**bad) == pk.ERR_INVALID, bad
    assert call(D=96) == pk.ERR_UNSUPPORTED
    assert call(dt=0) == pk.ERR_UNSUPPORTED  # f16 rows into a bf16 pool
    assert call(Hq=1 << 21, qs=1 << 28, os=1 << 28) == pk.ERR_UNSUPPORTED


def test_rope_append_operands_refused(pk):
    d = pk.CacheDesc(num_blocks=2, num_kv_heads=2, head_size=64, kv_dtype="bf16")
    rows = lambda n, h, dt=torch.bfloat16: torch.zeros(n, h, 64, dtype=dt)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    good = dict(q=rows(3, 4), k=rows(3, 2), v=rows(3, 2), positions=torch.zeros(3, dtype=torch.int32),
                slot_mapping=torch.zeros(3, dtype=torch.int64), freqs=torch.zeros(32, 2), k_cache=pool, v_cache=pool, desc=d,
                q_out=rows(3, 4))
    with pytest.raises(TypeError, match="CUDA tensor"):
        pk.paged_rope_append(**good)
    # more are met on the GPU, where operands have a device
    for bad, err in ((dict(q=None), ValueError), (dict(k=rows(2, 2)), ValueError), (dict(k=rows(3, 1)), ValueError),
                     (dict(k=rows(3, 2, torch.float32)), TypeError), (dict(k=rows(3, 2).transpose(0, 1)), ValueError),
                     (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), TypeError), (dict(freqs=torch.zeros(32, 3)), ValueError),
                     (dict(freqs=torch.zeros(32, 2).double()), ValueError), (dict(slot_mapping=torch.zeros(3, 1, dtype=torch.int64)), ValueError),
                     (dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16)[:, :, ::2]), ValueError), (dict(positions=None), TypeError)):
        with pytest.raises(err):
            pk.paged_rope_append(**{**good, **bad})
