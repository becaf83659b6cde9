"""Rotary append on the GPU against the rotation in 64 bits; rows into coded pools against the plain append of the
rotated rows, byte for byte."""
import math

import numpy as np
import pytest
import torch

import quant_util as qu

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


FAR = [0, 1, 4095, 4096, 131071, (1 << 24) + 1, (1 << 31) - 1, -1, -70000, 1000003]


def rotated(x, pos, freqs, inter, m):
    """x [T, H, D] float64; (result, bound on the error in front of the final rounding)."""
    R = 2 * len(freqs)
    ang = pos.astype(np.float64)[:, None] * (freqs.astype(np.float64).sum(-1) * 2 * math.pi)
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * c - b * s, b * c + a * s
    # an angle within 2^-23 of a turn and pos 2^-51, sincospi, the magnitude, two products and a sum: 2^-24 and less each
    off = 2 * math.pi * (2.0 ** -23 + np.abs(pos.astype(np.float64)) * 2.0 ** -51) + 5 * 2.0 ** -24
    e = np.broadcast_to(abs(m) * off[:, None, None] * (np.abs(a) + np.abs(b)), u.shape)
    out, err = x.copy(), np.zeros_like(x)
    if inter:
        out[..., 0:R:2], out[..., 1:R:2], err[..., 0:R:2], err[..., 1:R:2] = u, v, e, e
    else:
        out[..., :R // 2], out[..., R // 2:R], err[..., :R // 2], err[..., R // 2:R] = u, v, e, e
    return out, err


def close(got, x, pos, freqs, inter, m, dtype):
    ref, err = rotated(x.double().cpu().numpy(), pos, freqs, inter, m)
    t = qu.TORCH[dtype]
    # rounded once: half a step of the value, of a subnormal's step below the normal range
    tol = err + torch.finfo(t).eps / 2 * (np.abs(ref) + err) + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) - tol).max())
    R = 2 * len(freqs)
    assert np.array_equal(got[..., R:], x.double().cpu().numpy()[..., R:])


def inputs(rng, T, Hq, Hkv, D, dtype, fused):
    t = qu.TORCH[dtype]
    if fused:
        x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv + 1, D))).to(t).cuda()
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    return tuple(torch.from_numpy(rng.standard_normal((T, h, D))).to(t).cuda() for h in (Hq, Hkv, Hkv))


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,R,Hq,Hkv", [(64, 64, 3, 1), (64, 16, 8, 8), (128, 128, 32, 8), (128, 32, 5, 5), (128, 112, 2, 1)])
@pytest.mark.parametrize("T", [1, 2, 37, 700])
def test_rotation_and_append(pk, T, D, R, Hq, Hkv, dtype, inter, fused):
    rng = np.random.default_rng([T, D, R, Hq])
    NB = T // 8 + 3
    q, k, v = inputs(rng, T, Hq, Hkv, D, dtype, fused)
    pos = rng.integers(0, 200000, T).astype(np.int32)
    pos[:len(FAR)] = FAR[:T]
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    if T > 2:
        slots[::5] = -1
    freqs = pk.rope_frequencies(R, scaling="parts", factor=16.0, original_len=4096)
    m = 1.0 if T % 2 else 1.277
    desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=dtype)
    kc = torch.from_numpy(rng.standard_normal((NB, Hkv, 16, D))).to(qu.TORCH[dtype]).cuda()
    vc = kc.flip(0).contiguous()
    k0, v0 = kc.clone(), vc.clone()
    q_out = torch.zeros(T, Hq, D, dtype=q.dtype, device="cuda")
    dp, ds, df = (torch.from_numpy(a).cuda() for a in (pos, slots, freqs))
    pk.paged_rope_append(q, k, v, dp, ds, df, kc, vc, desc, q_out, interleaved=inter, magnitude=m)
    assert pk.get_device_error() == 0
    close(q_out, q, pos, freqs, inter, np.float64(np.float32(m)), dtype)
    live = slots >= 0
    b, o = slots[live] // 16, slots[live] % 16
    close(kc[b, :, o], k[torch.from_numpy(live).cuda()], pos[live], freqs, inter, np.float64(np.float32(m)), dtype)
    assert torch.equal(vc[b, :, o], v[torch.from_numpy(live).cuda()])
    k0[b, :, o], v0[b, :, o] = kc[b, :, o], vc[b, :, o]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # other rows as they were
    # without queries, and in place: the same bits
    k1, v1 = torch.zeros_like(kc), torch.zeros_like(vc)
    pk.paged_rope_append(None, k, v, dp, ds, df, k1, v1, desc, None, interleaved=inter, magnitude=m)
    assert torch.equal(k1[b, :, o], kc[b, :, o]) and torch.equal(v1[b, :, o], vc[b, :, o])
    rows_k = k.clone() if fused else None
    pk.paged_rope_append(q, k, v, dp, ds, df, k1, v1, desc, q, interleaved=inter, magnitude=m)
    assert torch.equal(q, q_out) and (rows_k is None or torch.equal(k, rows_k))
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,R,Hq,Hkv,inter", [(64, 64, 4, 1, False), (64, 32, 1, 3, True), (128, 128, 8, 8, False), (128, 64, 0, 2, True)])
@pytest.mark.parametrize("T", [1, 45, 650])
def test_coded_pools_hold_what_the_append_writes(pk, kv, dtype, D, R, Hq, Hkv, inter, T):
    rng = np.random.default_rng([T, D, Hkv])
    NB = T // 8 + 3
    q, k, v = inputs(rng, T, max(Hq, 1), Hkv, D, dtype, True)
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32)).cuda()
    slots = torch.from_numpy(rng.permutation(NB * 16)[:T].astype(np.int64)).cuda()
    slots[1::4] = -1
    freqs = torch.from_numpy(pk.rope_frequencies(R)).cuda()
    d16 = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=dtype)
    d = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv, k_scale=0.05, v_scale=0.04)
    every = torch.arange(T, device="cuda")
    k16, v16 = (torch.zeros(NB, Hkv, 16, D, dtype=k.dtype, device="cuda") for _ in range(2))
    pk.paged_rope_append(None, k, v, pos, every, freqs, k16, v16, d16, None, interleaved=inter)
    turned = k16.transpose(1, 2).reshape(-1, Hkv, D)[:T].contiguous()
    fill = torch.from_numpy(rng.integers(0, 256, (2, NB * pk.block_bytes(d)), dtype=np.uint8)).cuda()
    ka, va, kb, vb = fill[0].clone(), fill[1].clone(), fill[0].clone(), fill[1].clone()
    pk.paged_kv_append(turned, v.contiguous(), slots, ka, va, d)
    qq = q if Hq else None
    pk.paged_rope_append(qq, k, v, pos, slots, freqs, kb, vb, d, None if qq is None else torch.empty(T, Hq, D, dtype=q.dtype, device="cuda"),
                         interleaved=inter)
    assert pk.get_device_error() == 0
    assert torch.equal(ka, kb) and torch.equal(va, vb)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_slot_outside_the_pool_is_reported_and_skipped(pk, kv):
    d = pk.CacheDesc(num_blocks=2, num_kv_heads=2, head_size=64, kv_dtype=kv)
    kc, vc = (torch.zeros(2 * pk.block_bytes(d), dtype=torch.uint8, device="cuda") for _ in range(2))
    x = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.zeros_like(x)
    freqs = torch.from_numpy(pk.rope_frequencies(64)).cuda()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    pk.paged_rope_append(x, x, x, pos, torch.tensor([32, -5, 1 << 40], device="cuda"), freqs, kc, vc, d, q)
    assert pk.get_device_error() == pk.DEVERR_SLOT
    assert int(kc.sum()) == 0 and int(vc.sum()) == 0 and torch.equal(q, x)  # position 0 turns nothing


def test_operands_of_the_wrong_device_or_layout(pk):
    d = pk.CacheDesc(num_blocks=2, num_kv_heads=2, head_size=64, kv_dtype="bf16")
    mk = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    x = lambda n, h: mk(n, h, 64, dtype=torch.bfloat16)
    good = dict(q=x(3, 4), k=x(3, 2), v=x(3, 2), positions=mk(3, dtype=torch.int32), slot_mapping=mk(3, dtype=torch.int64),
                freqs=mk(32, 2), k_cache=x(32, 2), v_cache=x(32, 2), desc=d, q_out=x(3, 4))
    pk.paged_rope_append(**{**good, "k_cache": mk(2, 2, 16, 64, dtype=torch.bfloat16), "v_cache": mk(2, 2, 16, 64, dtype=torch.bfloat16)})
    for bad, err in ((dict(q_out=x(3, 3)), ValueError), (dict(q_out=None), ValueError), (dict(v=x(3, 1)), ValueError),
                     (dict(q_out=x(3, 4).half()), ValueError), (dict(positions=mk(2, dtype=torch.int32)), ValueError),
                     (dict(positions=mk(3, dtype=torch.int64)), ValueError), (dict(k_cache=x(31, 2)), ValueError),
                     (dict(freqs=mk(2, 32).t()), ValueError), (dict(positions=torch.zeros(3, dtype=torch.int32)), TypeError),
                     (dict(v=x(4, 2).transpose(0, 1)[:, :3].transpose(0, 1).transpose(1, 2)), ValueError),
                     (dict(k=mk(3, 2 * 64 + 4, dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64))), pk.PagedKVError),
                     (dict(k=x(1, 2).expand(3, 2, 64)), pk.PagedKVError)):
        with pytest.raises(err):
            pk.paged_rope_append(**{**good, **bad})


def test_captured_and_on_another_stream(pk):
    rng = np.random.default_rng(3)
    T, Hq, Hkv, D = 40, 8, 2, 128
    q, k, v = inputs(rng, T, Hq, Hkv, D, "bf16", True)
    d = pk.CacheDesc(num_blocks=8, num_kv_heads=Hkv, head_size=D, kv_dtype="bf16")
    kc, vc = (torch.zeros(8, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots, freqs = torch.arange(T, device="cuda"), torch.from_numpy(pk.rope_frequencies(D)).cuda()
    want, got = torch.zeros(T, Hq, D, dtype=q.dtype, device="cuda"), torch.zeros(T, Hq, D, dtype=q.dtype, device="cuda")
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        pk.paged_rope_append(q, k, v, pos, slots, freqs, kc, vc, d, got)
    pos += 1000
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    kg = kc.clone()
    pk.paged_rope_append(q, k, v, pos, slots, freqs, kc.zero_(), vc, d, want, stream=torch.cuda.default_stream())
    assert torch.equal(got, want) and torch.equal(kg, kc)
    assert pk.get_device_error() == 0
