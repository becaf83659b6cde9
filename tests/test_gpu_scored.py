"""Scored decode on the GPU: capped, biased and masked scores over every pool type, and the cached tokens' shares,
against the plain 64-bit forms on the values that the pools hold."""
import numpy as np
import pytest
import torch

import quant_util as qu
import score_util as su
from parity_util import TOL, max_error

pytestmark = pytest.mark.gpu

KVS = ["f16", "bf16", "e4m3", "int8", "int4"]
LENS = [1, 15, 16, 17, 33, 100, 255, 256, 257, 513, 700, 0]
SCORES = {
    "plain": dict(),
    "cap": dict(cap=5.0),
    "wide_cap": dict(cap=50.0),
    "window_1": dict(window=1),
    "window_16": dict(window=16),
    "window_17": dict(window=17),
    "window_100": dict(window=100),
    "slopes": dict(slopes=True),
    "first": dict(first=True),
    "all": dict(cap=20.0, window=230, slopes=True, first=True),
}


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


class Case:
    """A batch with its reference; rows outside what a sequence attends to hold NaN, blocks wholly outside have table
    entries that name no block."""

    def __init__(self, pk, kv, D, Hkv, G, q_dtype, mod, seed=0, lens=LENS, spread=2.0, spoil=True):
        rng = np.random.default_rng([seed, D, Hkv, G, KVS.index(kv)])
        self.pk, self.lens, self.D, self.Hq = pk, lens, D, Hkv * G
        S = len(lens)
        NB, self.tables = qu.make_tables(rng, lens)
        self.pools = qu.Pools(rng, NB, Hkv, D, kv)
        self.q = qu.queries(rng, S, self.Hq, D, q_dtype, spread)
        self.scale, self.q_dtype, self.kv = D ** -0.5, q_dtype, kv
        self.cap, self.window = mod.get("cap", 0.0), mod.get("window", 0)
        # falling and (one head) rising with the distance
        self.slopes = None
        if mod.get("slopes"):
            self.slopes = (2.0 ** -(1 + 8 * np.arange(self.Hq) / self.Hq)).astype(np.float32)
            self.slopes[-1] = -0.01
        self.first = None
        if mod.get("first"):
            # padding in front, a negative entry, a row with nothing left, one with its last token alone
            self.first = np.array([int(rng.integers(0, L + 1)) for L in lens], np.int32)
            self.first[3 % S], self.first[5 % S], self.first[7 % S] = -5, lens[5 % S] + 3, max(0, lens[7 % S] - 1)
        where = [(s, L - 1) for s, L in enumerate(lens)]
        self.ref, self.shares = su.ref_scored(self.q, where, self.pools, self.tables, lens, self.scale, self.cap, self.window,
                                              self.slopes, self.first)
        self.kd, self.vd = self.pools.dev()
        self.dev_tables = self.tables.copy()
        if spoil:
            self.pools.spoil_tail(self.tables, lens, self.kd, self.vd)
            self.spoil_front()

    def spoil_front(self):
        for s, (t, _) in enumerate(self.shares):
            lo = int(t[0]) if len(t) else self.lens[s]
            self.dev_tables[s, :lo // 16] = 1 << 28
            if lo % 16 and len(t):
                spoil_rows(self.pools, self.kd, self.vd, int(self.tables[s][lo // 16]), 0, lo % 16)

    def score(self):
        return self.pk.ScoreMod(cap=self.cap, window=self.window,
                                slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                                first=None if self.first is None else i32(self.first))

    def run(self, part=0, weights=None, new=None, q=None, out=None, ws=None, stream=None, score=None):
        pk, S = self.pk, len(self.lens)
        mx = max(max(self.lens), 1)
        q = self.q.cuda() if q is None else q
        out = torch.full_like(q, 7.0) if out is None else out
        need = pk.decode_scored_workspace_bytes(S, self.Hq, self.D, mx, self.window, part, weights is not None)
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        pk.paged_attention_decode_scored(q, self.kd, self.vd, self.pools.desc, i32(self.dev_tables), i32(self.lens), mx,
                                         self.scale, out, self.score() if score is None else score, weights=weights,
                                         new_lens=new, workspace=ws, partition_tokens=part, stream=stream)
        return out

    def check(self, out):
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        vmax = float(np.abs(self.pools.vh).max())
        err = max_error(got, self.ref, self.q_dtype, TOL["f16" if self.q_dtype == "f16" and self.kv != "e4m3" else "bf16"], vmax)
        assert err <= TOL["f16" if self.q_dtype == "f16" and self.kv != "e4m3" else "bf16"], err
        for s, (t, _) in enumerate(self.shares):
            if not len(t):
                assert np.all(got[s] == 0.0)


def spoil_rows(pools, kd, vd, blk, t0, t1):
    """Rows t0 .. t1 - 1 of a block become NaN in every head, codes and parameters alike."""
    for pool, value in ((kd, False), (vd, True)):
        if pools.kv in qu.BITS:
            bits = qu.BITS[pools.kv]
            rb = pools.D * bits // 8
            pool[blk, :, torch.from_numpy(qu.places(pools.D, bits, value)[t0:t1].reshape(-1)).cuda()] = 255
            pool[blk, :, 16 * rb + 8 * t0:16 * rb + 8 * t1] = 255
        elif pools.kv == "e4m3":
            pool[blk, :, t0:t1] = 0x7F
        else:
            pool[blk, :, t0:t1] = float("nan")


def q_types(kv):
    return [kv] if kv in ("f16", "bf16") else ["f16", "bf16"]


@pytest.mark.parametrize("mod", list(SCORES))
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (64, 1, 8), (64, 2, 4), (128, 2, 1), (128, 2, 2), (128, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("kv", KVS)
def test_decode_scored(pk, kv, D, Hkv, G, mod):
    c = Case(pk, kv, D, Hkv, G, q_types(kv)[-1], SCORES[mod])
    for part in (0, 16, 64):
        c.check(c.run(part))
    if kv not in qu.BITS and D == 128 and G > 1:
        with pk.decode_path(pk.PATH_CUDA_CORES):
            c.check(c.run(48))
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 4)])
def test_decode_scored_f16_queries(pk, kv, D, G):
    c = Case(pk, kv, D, 2, G, "f16", SCORES["all"], seed=3)
    for part in (0, 32):
        c.check(c.run(part))
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("mod", ["plain", "all", "window_17", "first"])
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (64, 2, 4), (128, 3, 1), (128, 2, 2), (128, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("new", ["all", "one", "mixed"])
def test_weights(pk, kv, D, Hkv, G, mod, new):
    c = Case(pk, kv, D, Hkv, G, q_types(kv)[0], SCORES[mod], seed=1)
    rng = np.random.default_rng(5)
    w0 = (rng.random((c.pools.NB, Hkv, 16)) * 3).astype(np.float32)
    fresh = {"all": None, "one": np.minimum(1, c.lens), "mixed": np.array([int(rng.integers(0, L + 1)) for L in c.lens])}[new]
    # an entry's block outside the row's range is still written where it is set anew
    if new != "one":
        c.dev_tables = c.tables.copy()
    want, step = su.ref_weights(w0, c.shares, c.tables, c.lens, fresh, Hkv)
    # a new token whose table entry names no block (the row's range does not reach it) is reported and keeps its entry
    lost = [(c.tables[s][(L - 1) // 16], (L - 1) % 16) for s, L in enumerate(c.lens)
            if new == "one" and L and c.dev_tables[s][(L - 1) // 16] >= c.pools.NB]
    for blk, t in lost:
        want[blk, :, t] = w0[blk, :, t]
    # a head's 2^x below binary32's normal range is 0: up to 2^-126 each, times a sum's reciprocal of at most 1 (the
    # largest share's term is at least 2^-8, the reference maximum moving only by more: 2^8)
    tol = su.share_bound(c.q, c.pools, c.scale, c.cap, c.slopes, 700) * step + 2.0 ** -24 * want + G * 2.0 ** -118
    for part in (0, 64):
        w = torch.from_numpy(w0.copy()).cuda()
        c.check(c.run(part, weights=w, new=None if fresh is None else i32(fresh)))
        got = w.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) - tol).max())
        still = np.ones_like(w0, bool)
        for s, (t, _) in enumerate(c.shares):
            L = c.lens[s]
            t = np.union1d(t, np.arange(L - (L if fresh is None else fresh[s]), L)).astype(int)
            still[c.tables[s][t // 16], :, t % 16] = False
        assert np.array_equal(w.cpu().numpy()[still], w0[still])
    assert pk.get_device_error() == (pk.DEVERR_BLOCK_ID if lost else 0)


@pytest.mark.parametrize("kv,G", [("bf16", 4), ("bf16", 1), ("int4", 8)])
def test_long_row_and_its_shares(pk, kv, G):
    lens = [20011, 5]
    c = Case(pk, kv, 128, 1, G, "bf16", dict(slopes=True, cap=30.0), seed=9, lens=lens)
    w = torch.zeros(c.pools.NB, 1, 16, device="cuda")
    c.check(c.run(0, weights=w))
    want, step = su.ref_weights(w.cpu().numpy() * 0, c.shares, c.tables, lens, None, 1)
    tol = su.share_bound(c.q, c.pools, c.scale, c.cap, c.slopes, 20011) * step + G * 2.0 ** -118  # as above
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= tol)
    assert abs(float(w.double().sum()) - 2 * G) < 1e-3
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("kv", ["f16", "int8"])
@pytest.mark.parametrize("G", [1, 4])
def test_plain_scores_give_what_decode_gives(pk, kv, G):
    c = Case(pk, kv, 128, 2, G, "f16", {}, seed=4, spoil=False)
    want = torch.zeros_like(c.q, device="cuda")
    ws = torch.zeros(pk.decode_workspace_bytes(len(c.lens), c.Hq, 128, 700, 64), dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.tables), i32(c.lens), 700, c.scale, want,
                              workspace=ws, partition_tokens=64)
    assert torch.equal(c.run(64), want)
    out = torch.zeros_like(want)  # no ScoreMod at all
    ws = torch.zeros(pk.decode_scored_workspace_bytes(len(c.lens), c.Hq, 128, 700, 0, 64), dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.tables), i32(c.lens), 700, c.scale, out,
                                     workspace=ws, partition_tokens=64)
    assert torch.equal(out, want)


def test_wrong_lengths_and_blocks_are_reported(pk):
    c = Case(pk, "bf16", 128, 2, 4, "bf16", {}, lens=[100, 40], spoil=False)
    w = torch.zeros(c.pools.NB, 2, 16, device="cuda")
    c.lens = [100, -3]
    c.run(0, weights=w)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    c.lens = [100, 5000]
    out = torch.zeros_like(c.q, device="cuda")
    ws = torch.zeros(pk.decode_scored_workspace_bytes(2, 8, 128, 112, 0, 0, True), dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.tables), i32([100, 5000]), 112, c.scale, out,
                                     weights=w, workspace=ws)
    assert pk.get_device_error() & pk.DEVERR_SEQ_LEN
    pk.paged_attention_decode_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.tables), i32([100, 40]), 112, c.scale, out,
                                     weights=w, new_lens=i32([101, -1]), workspace=ws)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    t = c.tables.copy()
    t[0, 2] = c.pools.NB
    pk.paged_attention_decode_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(t), i32([100, 40]), 112, c.scale, out,
                                     weights=w, workspace=ws)
    assert pk.get_device_error() == pk.DEVERR_BLOCK_ID


def test_captured_and_replayed_with_two_workspaces_and_streams(pk):
    """Two captured calls on two streams, replayed together after their inputs changed."""
    cs = [Case(pk, kv, 128, 2, 4, "bf16", SCORES["all"], seed=20 + i) for i, kv in enumerate(("bf16", "int4"))]
    graphs = []
    for c in cs:
        st = torch.cuda.Stream()
        c.qd, c.w = torch.zeros_like(c.q, device="cuda"), torch.zeros(c.pools.NB, 2, 16, device="cuda")
        c.sc, c.ot = c.score(), torch.zeros_like(c.q, device="cuda")
        c.tb, c.ln = i32(c.dev_tables), i32(c.lens)
        c.ws = torch.zeros(pk.decode_scored_workspace_bytes(len(c.lens), 8, 128, 700, c.window, 64, True), dtype=torch.uint8,
                           device="cuda")
        c.new = i32(np.minimum(1, c.lens))
        call = lambda c=c: pk.paged_attention_decode_scored(c.qd, c.kd, c.vd, c.pools.desc, c.tb, c.ln, 700, c.scale, c.ot, c.sc,
                                                            weights=c.w, new_lens=c.new, workspace=c.ws, partition_tokens=64)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append((g, st))
    for c in cs:
        c.qd.copy_(c.q)
        c.w.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check(c.ot)
        want = su.ref_weights(np.zeros((c.pools.NB, 2, 16), np.float32), c.shares, c.tables, c.lens, None, 2)[0]
        last = np.zeros_like(want, bool)
        for s, L in enumerate(c.lens):
            if L:
                last[c.tables[s][(L - 1) // 16], :, (L - 1) % 16] = True
        got = c.w.double().cpu().numpy()
        tol = 4 * su.share_bound(c.q, c.pools, c.scale, c.cap, c.slopes, 700) * want + 1e-30
        assert np.all(np.abs(got - np.where(last, want, 3 * want)) <= tol)  # added three times, the new token's set
    assert pk.get_device_error() == 0
