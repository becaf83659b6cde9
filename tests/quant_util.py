"""Plain 64-bit forms of the integer-coded pools and of sparse decode, in numpy.

Rows are encoded by their definition (each step one binary32 operation), tiles
are laid out byte by byte from the ABI's formulas, and attention, bounds and
block scores are computed in float64 on the values the pools hold.
"""
from __future__ import annotations

import numpy as np
import torch

B = 16
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"int8": 8, "int4": 4}


def round_to(x: np.ndarray, dtype: str) -> np.ndarray:
    """float64 -> the 16-bit type's values, as float32."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(TORCH[dtype]).float().numpy()


def encode(x: np.ndarray, bits: int):
    """x [..., D] float32 -> codes uint8, scale, zero (float32)."""
    x = np.asarray(x, np.float32)
    top = np.float32(2 ** bits - 1)
    lo, hi = x.min(-1), x.max(-1)
    scale = (hi - lo) / top
    scale[scale < np.float32(2.0 ** -126)] = 0
    inv = np.zeros_like(scale)
    np.divide(np.float32(1), scale, out=inv, where=scale > 0)
    code = np.minimum(np.rint((x - lo[..., None]) * inv[..., None]), top)
    return code.astype(np.uint8), scale, lo


def held(x: np.ndarray, bits: int) -> np.ndarray:
    """The values the rows are held as, float64."""
    code, scale, lo = encode(x, bits)
    return lo[..., None].astype(np.float64) + scale[..., None].astype(np.float64) * code.astype(np.float64)


def byte_place(D: int, bits: int, value: bool, t: int, k: int) -> int:
    rb = D * bits // 8
    if not value:
        w = min(rb, 64)
        return (k // 64) * 16 * w + t * w + k % 64
    x = (k // 2) * 4 + (t % 2) * 2 + k % 2
    return (x // 32) * 256 + (t // 2) * 32 + x % 32


def places(D, bits, value):
    rb = D * bits // 8
    return np.array([[byte_place(D, bits, value, t, k) for k in range(rb)] for t in range(B)])


def write_row(pool, D, bits, value, blk, h, t, x):
    """Writes one row x [D] into a uint8 pool [NB, Hkv, tile]."""
    code, scale, lo = encode(x[None], bits)
    code = code[0]
    if bits == 4:
        code = code[0::2] | (code[1::2] << 4)
    rb = D * bits // 8
    pool[blk, h, places(D, bits, value)[t]] = code
    pool[blk, h, 16 * rb + 8 * t:16 * rb + 8 * t + 8] = np.array([scale[0], lo[0]], np.float32).view(np.uint8)


def pack(x: np.ndarray, bits: int, value: bool) -> np.ndarray:
    """[NB, Hkv, 16, D] values -> uint8 pool [NB, Hkv, tile bytes]."""
    NB, H, _, D = x.shape
    rb = D * bits // 8
    code, scale, lo = encode(x, bits)
    if bits == 4:
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    pool = np.zeros((NB, H, 16 * rb + 128), np.uint8)
    pool[:, :, places(D, bits, value).reshape(-1)] = code.reshape(NB, H, -1)
    par = np.stack([scale, lo], -1).astype(np.float32)
    pool[:, :, 16 * rb:] = np.ascontiguousarray(par).view(np.uint8).reshape(NB, H, 128)
    return pool


class Pools:
    """A pair of pools of any type with known held values (float64 [NB, Hkv, 16, D])."""

    def __init__(self, rng, NB, Hkv, D, kv, k_scale=0.03, v_scale=0.02, spread=1.0):
        from paged_kv_cache_10_gb300 import pagedkv as pk
        self.NB, self.Hkv, self.D, self.kv = NB, Hkv, D, kv
        shape = (NB, Hkv, B, D)
        k, v = rng.standard_normal(shape) * spread, rng.standard_normal(shape) * spread
        k = k + (rng.random(D) < 0.1) * 2.0
        self.k_scale = self.v_scale = 1.0
        if kv in BITS:
            b = BITS[kv]
            k, v = round_to(k, "bf16"), round_to(v, "bf16")
            self.kh, self.vh = held(k, b), held(v, b)
            self.k_host, self.v_host = pack(k, b, False), pack(v, b, True)
        elif kv == "e4m3":
            self.k_scale, self.v_scale = k_scale, v_scale
            kc = torch.from_numpy(k / k_scale).clamp(-448, 448).float().to(torch.float8_e4m3fn)
            vc = torch.from_numpy(v / v_scale).clamp(-448, 448).float().to(torch.float8_e4m3fn)
            self.kh = kc.float().double().numpy() * np.float64(np.float32(k_scale))
            self.vh = vc.float().double().numpy() * np.float64(np.float32(v_scale))
            self.k_host, self.v_host = kc.view(torch.uint8).numpy(), vc.view(torch.uint8).numpy()
        else:
            kt, vt = torch.from_numpy(k).to(TORCH[kv]), torch.from_numpy(v).to(TORCH[kv])
            self.kh, self.vh = kt.double().numpy(), vt.double().numpy()
            self.k_host, self.v_host = kt.view(torch.int16).numpy(), vt.view(torch.int16).numpy()
        self.desc = pk.CacheDesc(num_blocks=NB, num_kv_heads=Hkv, head_size=D, kv_dtype=kv, k_scale=self.k_scale,
                                 v_scale=self.v_scale)

    def dev(self):
        """Device pools."""
        out = []
        for a in (self.k_host, self.v_host):
            t = torch.from_numpy(np.array(a)).cuda()
            out.append(t.view(TORCH[self.kv]) if self.kv in TORCH else t)
        return out

    def spoil_tail(self, tables, lens, kd, vd):
        """Rows past every sequence's end get all-ones bytes (NaN as floats), codes and parameters alike."""
        for s, L in enumerate(lens):
            if L % B == 0:
                continue
            blk, t0 = int(tables[s][L // B]), L % B
            for pool, value in ((kd, False), (vd, True)):
                if self.kv in BITS:
                    bits = BITS[self.kv]
                    rb = self.D * bits // 8
                    at = places(self.D, bits, value)[t0:].reshape(-1)
                    pool[blk, :, torch.from_numpy(at).cuda()] = 255
                    pool[blk, :, 16 * rb + 8 * t0:] = 255
                elif self.kv == "e4m3":
                    pool[blk, :, t0:] = 0x7F
                else:
                    pool[blk, :, t0:] = float("nan")


def make_tables(rng, lens, spare=3):
    nb = [(L + B - 1) // B for L in lens]
    NB = sum(nb) + spare
    ids = rng.permutation(NB)
    MB = max(1, max(nb))
    t = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for s, n in enumerate(nb):
        t[s, :n] = ids[at:at + n]
        at += n
    return NB, t


def queries(rng, S, Hq, D, dtype, spread=1.0):
    return torch.from_numpy(rng.standard_normal((S, Hq, D)) * spread).to(TORCH[dtype])


def attend(q, kh, vh, blocks, valid, scale):
    """One (sequence, KV head): q [G, D] float64; blocks: physical ids; valid: tokens of each."""
    D = q.shape[-1]
    ks = [kh[b, :n] for b, n in zip(blocks, valid)]
    if not ks:
        return np.zeros_like(q)
    k, v = np.concatenate(ks), np.concatenate([vh[b, :n] for b, n in zip(blocks, valid)])
    if not len(k):
        return np.zeros_like(q)
    sc = q @ k.T * scale
    p = np.exp(sc - sc.max(-1, keepdims=True))
    return (p / p.sum(-1, keepdims=True)) @ v


def ref_dense(q, pools, tables, lens, scale):
    q = q.double().numpy()
    S, Hq, D = q.shape
    G = Hq // pools.Hkv
    out = np.zeros_like(q)
    for s, L in enumerate(lens):
        nb = (L + B - 1) // B
        blocks = tables[s][:nb]
        valid = [min(B, L - j * B) for j in range(nb)]
        for h in range(pools.Hkv):
            out[s, h * G:(h + 1) * G] = attend(q[s, h * G:(h + 1) * G], pools.kh[:, h], pools.vh[:, h], blocks, valid, scale)
    return out


def ref_sparse(q, pools, tables, lens, selected, scale):
    q = q.double().numpy()
    S, Hq, D = q.shape
    G = Hq // pools.Hkv
    out = np.zeros_like(q)
    for s, L in enumerate(lens):
        for h in range(pools.Hkv):
            js = [int(j) for j in selected[s, h] if j >= 0 and j * B < L]
            blocks, valid = [tables[s][j] for j in js], [min(B, L - j * B) for j in js]
            out[s, h * G:(h + 1) * G] = attend(q[s, h * G:(h + 1) * G], pools.kh[:, h], pools.vh[:, h], blocks, valid, scale)
    return out


def ref_select(q, bounds, tables, lens, n, sink, recent, Hkv):
    """bounds float64 [NB, Hkv, 2, D]; the definition, block by block."""
    q = q.double().numpy()
    S, Hq, D = q.shape
    G = Hq // Hkv
    out = np.full((S, Hkv, n), -1, np.int32)
    for s, L in enumerate(lens):
        nb = (L + B - 1) // B
        if nb <= n:
            out[s, :, :nb] = np.arange(nb)
            continue
        bd = bounds[tables[s][:nb]]
        for h in range(Hkv):
            qq = q[s, h * G:(h + 1) * G]
            lo, hi = bd[:, h, 0], bd[:, h, 1]
            with np.errstate(invalid="ignore"):
                u = np.stack([np.where(x < 0, x * lo, x * hi).sum(-1) for x in qq])
            u = np.where(np.isnan(u), -np.inf, u).max(0)
            forced = np.zeros(nb, bool)
            forced[:sink] = True
            forced[nb - recent:] = True
            order = np.lexsort((np.arange(nb), -u, ~forced))
            out[s, h] = np.sort(order[:n])
    return out


def ref_bounds(pools, tables, lens, new, bounds0, dtype):
    """bounds0 float32 [NB, Hkv, 2, D] updated for the blocks with new tokens, rounded outwards to dtype."""
    out = bounds0.copy()
    for s, (L, n) in enumerate(zip(lens, new)):
        if n <= 0:
            continue
        for j in range((L - n) // B, (L - 1) // B + 1):
            # keys in binary32, as every reader forms them (float64 holds scale * code exactly)
            k = pools.kh[tables[s][j], :, :min(B, L - j * B)].astype(np.float32).astype(np.float64)
            out[tables[s][j], :, 0] = outward(k.min(1), dtype, False)
            out[tables[s][j], :, 1] = outward(k.max(1), dtype, True)
    return out


def outward(x, dtype, up):
    """Directed rounding of float64 values to the 16-bit type."""
    r = torch.from_numpy(np.asarray(x, np.float64)).to(TORCH[dtype])
    wrong = r.double().numpy() < x if up else r.double().numpy() > x
    bits = r.view(torch.int16).numpy().view(np.uint16).astype(np.int64)
    # the next representable value outwards, on the ordered integers of the type
    key = np.where(bits & 0x8000, -(bits & 0x7FFF), bits)
    key = np.where(wrong, key + (1 if up else -1), key)
    nb = np.where(key < 0, (-key) | 0x8000, key).astype(np.uint16)
    return torch.from_numpy(nb.view(np.int16).copy()).view(TORCH[dtype]).float().numpy()
