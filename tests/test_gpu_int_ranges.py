"""Decode over integer-coded pools whose value rows differ widely in range: a row that the query does not attend
to takes no bits of the others, and the weights' scale follows the largest contribution up and down.

Errors are bounded in units of what the attended rows hold, U = sum_t p_t max_d |v_td| per query head (p the softmax
in 64 bits), so that a wide row that is not attended to loosens nothing:

  |got - ref| <= half a step of the output + U (2 delta + w)

delta bounds the error of a score in nats.  q . n is a chain of D / 16 MMAs, each within 17 * 2^-23 of the sum of
magnitudes |q|_1 (2^b - 1), so s (q . n) is within D / 16 * 17 * 2^-23 |q|_1 (max k - min k); the products and sums
around it are binary32 operations on terms of at most |q|_1 max |k|, five of them, and a score in log2 units passes
its own rounding and ex2's, 2^-21 of it at most.  An error of delta in every score moves the output by at most
2 delta U.  w covers the weights and their sums: two MMAs a block within 17 * 2^-23 of the sum of magnitudes p s' n <=
2 p max |v|, for the at most `blocks` blocks of a row, and 2^-16 for the weights' 22 bits, ex2, the merges and the
sums of p and of p z'.
"""
import itertools

import numpy as np
import pytest
import torch

import quant_util as qu

pytestmark = pytest.mark.gpu

KVS = ["int8", "int4"]
WAYS = ["dense", "split", "sparse", "sparse_split"]


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


class Rows:
    """Sequences given as token rows k, v [L, Hkv, D], packed into pools over shuffled blocks."""

    def __init__(self, rng, ks, vs, kv):
        self.lens = [len(k) for k in ks]
        self.Hkv, self.D = ks[0].shape[1:]
        NB, self.tables = qu.make_tables(rng, self.lens)
        kp, vp = (np.zeros((NB, self.Hkv, 16, self.D), np.float32) for _ in range(2))
        for s, L in enumerate(self.lens):
            for t in range(L):
                kp[self.tables[s, t // 16], :, t % 16] = ks[s][t]
                vp[self.tables[s, t // 16], :, t % 16] = vs[s][t]
        kp, vp = qu.round_to(kp, "bf16"), qu.round_to(vp, "bf16")
        bits = qu.BITS[kv]
        self.pools = qu.Pools(rng, NB, self.Hkv, self.D, kv)
        self.pools.kh, self.pools.vh = qu.held(kp, bits), qu.held(vp, bits)
        self.pools.k_host, self.pools.v_host = qu.pack(kp, bits, False), qu.pack(vp, bits, True)

    def run(self, pk, q, scale, way):
        kd, vd = self.pools.dev()
        S, Hq, D = q.shape
        t, l = torch.from_numpy(self.tables).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        out = torch.full((S, Hq, D), 7.0, device="cuda").to(q.dtype)
        mx, n = max(self.lens), self.tables.shape[1]
        buf = lambda b: torch.full((max(16, b),), 255, dtype=torch.uint8, device="cuda")
        if way.startswith("sparse"):
            sel = np.stack([np.where(np.arange(n) < (L + 15) // 16, np.arange(n), -1) for L in self.lens])
            sel = torch.from_numpy(np.repeat(sel[:, None], self.Hkv, 1).astype(np.int32)).cuda()
            part = 2 if way.endswith("split") else n
            pk.paged_attention_decode_sparse(q.cuda(), kd, vd, self.pools.desc, t, l, sel, scale, out,
                                             workspace=buf(pk.decode_sparse_workspace_bytes(S, Hq, D, n, part)),
                                             partition_blocks=part)
        else:
            part = 32 if way == "split" else (mx + 15) // 16 * 16
            pk.paged_attention_decode(q.cuda(), kd, vd, self.pools.desc, t, l, mx, scale, out,
                                      workspace=buf(pk.decode_workspace_bytes(S, Hq, D, mx, part)), partition_tokens=part)
        assert pk.get_device_error() == 0
        return out.double().cpu().numpy()

    def check(self, pk, q, scale, way, attended=None):
        """attended: a mask over a sequence's tokens whose scores and keys set delta (others have no weight)."""
        got = self.run(pk, q, scale, way)
        assert np.all(np.isfinite(got))
        eps = torch.finfo(q.dtype).eps
        G = q.shape[1] // self.Hkv
        for s, L in enumerate(self.lens):
            at = self.tables[s, np.arange(L) // 16], np.arange(L) % 16
            for hq in range(q.shape[1]):
                h = hq // G
                k, v = self.pools.kh[at[0], h, at[1]], self.pools.vh[at[0], h, at[1]]
                x = q[s, hq].double().numpy()
                sc = k @ x * scale
                p = np.exp(sc - sc.max())
                p /= p.sum()
                ref, U = p @ v, float(p @ np.abs(v).max(-1))
                on = np.ones(L, bool) if attended is None else attended[:L]
                ka, q1 = k[on], np.abs(x).sum() * scale
                delta = q1 * (self.D / 16 * 17 * 2.0 ** -23 * (ka.max(-1) - ka.min(-1)).max() + 5 * 2.0 ** -23 * np.abs(ka).max())
                delta += 2.0 ** -21 * np.abs(sc[on]).max() * 1.4427
                w = 2 * -(-L // 16) * 17 * 2.0 ** -23 * 2 + 2.0 ** -16
                tiny = 2.0 ** -25 if q.dtype == torch.float16 else 2.0 ** -134
                err = np.abs(got[s, hq] - ref)
                bound = eps / 2 * np.abs(ref) * (1 + 2 * delta) + U * (2 * delta + w) * (1 + eps) + tiny
                assert np.all(err <= bound), (s, hq, float(err.max()), float(bound[err.argmax()]), U)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("ratio", [12, 18, 24, 60])
@pytest.mark.parametrize("D,G,dtype", [(128, 1, "f16"), (128, 4, "bf16"), (128, 8, "f16"), (64, 8, "bf16"), (64, 2, "f16")])
@pytest.mark.parametrize("kv", KVS)
def test_a_wide_row_that_is_not_attended_to(pk, kv, D, G, dtype, ratio, way):
    """Rows 2^ratio wider than the others, at a score of -60 or below: first, last, and one in 37 between."""
    rng = np.random.default_rng(ratio + D + G)
    lens, Hkv, scale = [300, 50, 17], 2, D ** -0.5
    q = torch.from_numpy(np.abs(rng.standard_normal((3, Hkv * G, D))) + 0.5).to(qu.TORCH[dtype])
    low = -60 / (float(q.double().sum(-1).min()) * scale)
    ks, vs = [], []
    wide = np.arange(300) % 37 == 0
    for L in lens:
        k, v = rng.standard_normal((L, Hkv, D)) * 0.25, rng.standard_normal((L, Hkv, D))
        w = wide[:L].copy()
        w[L - 1] = True
        k[w], v[w] = low * 1.02, v[w] * 2.0 ** ratio
        ks.append(k)
        vs.append(v)
    rows = Rows(rng, ks, vs, kv)
    on = ~wide
    on[[L - 1 for L in lens]] = False
    rows.check(pk, q, scale, way, on)


@pytest.mark.parametrize("way", ["dense", "sparse_split"])
@pytest.mark.parametrize("ds,dv", list(itertools.product([-2.5, -1.0, 0.0, 1.0, 2.5], [-2, 0, 2])))
@pytest.mark.parametrize("kv", KVS)
def test_contributions_that_drift(pk, kv, ds, dv, way):
    """Scores that rise or fall by ds a block and value ranges by 2^dv: the largest contribution moves either way."""
    rng = np.random.default_rng(int(10 * ds + dv) + 100)
    D, Hkv, G, scale = 128, 1, 4, 128 ** -0.5
    lens = [700, 90, 33]
    q = torch.from_numpy(np.abs(rng.standard_normal((3, Hkv * G, D))) + 0.5).to(torch.bfloat16)
    unit = float(q.double().sum(-1).mean()) * scale
    ks, vs = [], []
    for L in lens:
        j = (np.arange(L) // 16)[:, None, None]
        ks.append(rng.standard_normal((L, Hkv, D)) * 0.05 + ds * j / unit)
        vs.append(rng.standard_normal((L, Hkv, D)) * np.exp2(dv * (j - 22.0)))
    Rows(rng, ks, vs, kv).check(pk, q, scale, way)


@pytest.mark.parametrize("way", ["dense", "split"])
@pytest.mark.parametrize("const", [0.0, 3.0])
@pytest.mark.parametrize("kv", KVS)
def test_attended_rows_without_a_range(pk, kv, const, way):
    """The attended rows are constant (no range at all); the others, 20 nats below, hold the output's small part."""
    rng = np.random.default_rng(17)
    D, Hkv, G, scale = 128, 2, 4, 128 ** -0.5
    q = torch.from_numpy(np.abs(rng.standard_normal((2, Hkv * G, D))) + 0.5).to(torch.bfloat16)
    unit = float(q.double().sum(-1).mean()) * scale
    ks, vs = [], []
    for L in (200, 31):
        k, v = rng.standard_normal((L, Hkv, D)) * 0.05, rng.standard_normal((L, Hkv, D))
        k[::5], v[::5] = 20 / unit, const
        ks.append(k)
        vs.append(v)
    Rows(rng, ks, vs, kv).check(pk, q, scale, way)


@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e30, 1e34])
@pytest.mark.parametrize("kv", KVS)
def test_values_near_the_ends_of_binary32(pk, kv, size):
    """|v| to the ends of bf16's range; scores within one nat, so that no sum of weights leaves binary32."""
    rng = np.random.default_rng(19)
    D, Hkv, scale = 64, 2, 0.125
    q = qu.queries(rng, 2, Hkv * 2, D, "bf16", 0.1)
    ks = [rng.standard_normal((L, Hkv, D)) for L in (60, 17)]
    vs = [rng.standard_normal((L, Hkv, D)) * size for L in (60, 17)]
    Rows(rng, ks, vs, kv).check(pk, q, scale, "dense")


@pytest.mark.parametrize("way", ["dense", "sparse_split"])
@pytest.mark.parametrize("e", [-124, -120, -105, 100, 110, 116])
@pytest.mark.parametrize("kv", KVS)
def test_queries_near_the_ends_of_binary32(pk, kv, e, way):
    """Queries of 2^e against keys of 2^-e: scores of a few nats, neither lost nor overflowing."""
    rng = np.random.default_rng(23)
    D, Hkv, scale = 128, 2, 128 ** -0.5
    q = (qu.queries(rng, 2, Hkv * 4, D, "f16", 0.5).double().clamp(-3, 3) * 2.0 ** e).to(torch.bfloat16)
    ks = [rng.standard_normal((L, Hkv, D)).clip(-3, 3) * 2.0 ** -e for L in (200, 17)]
    vs = [rng.standard_normal((L, Hkv, D)) for L in (200, 17)]
    Rows(rng, ks, vs, kv).check(pk, q, scale, way)


@pytest.mark.parametrize("seed", range(16))
@pytest.mark.parametrize("kv", KVS)
def test_rows_of_every_size_at_any_score(pk, kv, seed):
    """Value ranges over 2^+-40 and scores over tens of nats, row by row and at random; constant and zero rows."""
    rng = np.random.default_rng(1000 + seed)
    D, Hkv, G = int(rng.choice([64, 128])), int(rng.choice([1, 3])), int(rng.choice([1, 2, 4, 8]))
    dtype, way, scale = ["bf16", "f16"][seed % 2], WAYS[seed % 4], D ** -0.5
    spread = 40 if dtype == "bf16" else 12  # outputs within f16's range
    lens = [int(x) for x in rng.integers(1, 600, 4)]
    q = torch.from_numpy(np.abs(rng.standard_normal((4, Hkv * G, D))) + 0.5).to(qu.TORCH[dtype])
    unit = float(q.double().sum(-1).mean()) * scale
    ks, vs = [], []
    for L in lens:
        k = rng.standard_normal((L, Hkv, D)) * 0.1 + rng.standard_normal((L, Hkv, 1)) * 15 / unit
        v = rng.standard_normal((L, Hkv, D)) * np.exp2(rng.uniform(-spread, spread, (L, Hkv, 1)))
        v[rng.random(L) < 0.1] = 0.0
        flat = rng.random(L) < 0.1
        v[flat] = v[flat][..., :1]
        ks.append(k)
        vs.append(v)
    Rows(rng, ks, vs, kv).check(pk, q, scale, way)
