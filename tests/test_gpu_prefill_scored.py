"""Scored prefill on the GPU: capped, biased and masked scores, documents packed in a sequence and prefixes, against the
plain 64-bit form on the values that the pools hold, with values that are not finite wherever a row may not look."""
import numpy as np
import pytest
import torch

import quant_util as qu
import score_util as su
from parity_util import TOL, max_error
from test_gpu_scored import spoil_rows

pytestmark = pytest.mark.gpu

CHUNKS = [(0, 1), (0, 17), (37, 130), (200, 64), (5, 0), (513, 300), (1000, 3)]  # (context, new tokens)
SCORES = {
    "plain": dict(),
    "cap_of_small_scores": dict(cap=60.0),
    "cap_of_large_scores": dict(cap=1.5),
    "window_1": dict(window=1),
    "window_16": dict(window=16),
    "window_129": dict(window=129),
    "slopes": dict(slopes=True),
    "docs": dict(docs=6),
    "docs_window": dict(docs=2, window=70),
    "empty_rows": dict(docs=3, empty=True),
    "prefix": dict(prefix=150),
    "prefix_slopes": dict(prefix=400, slopes=True),
    "all": dict(cap=20.0, slopes=True, docs=2, window=200, prefix=60, empty=True),
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
    def __init__(self, pk, kv, D, Hkv, G, q_dtype, mod, seed=0, chunks=CHUNKS, spread=2.0):
        rng = np.random.default_rng([seed, D, Hkv, G])
        self.pk, self.kv, self.D, self.Hq, self.q_dtype = pk, kv, D, Hkv * G, q_dtype
        new = np.array([n for _, n in chunks])
        self.lens = [c + n for c, n in chunks]
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_max, self.T = int(new.max()), int(new.sum())
        NB, self.tables = qu.make_tables(rng, self.lens)
        self.pools = qu.Pools(rng, NB, Hkv, D, kv)
        self.q = qu.queries(rng, self.T, self.Hq, D, q_dtype, spread)
        self.scale = D ** -0.5
        self.where = [(s, c + j) for s, (c, n) in enumerate(chunks) for j in range(n)]
        self.cap, self.window = mod.get("cap", 0.0), mod.get("window", 0)
        self.slopes = (2.0 ** -(1 + 8 * np.arange(self.Hq) / self.Hq)).astype(np.float32) if mod.get("slopes") else None
        self.first = None
        if mod.get("docs"):
            first = []
            for s, (c, n) in enumerate(chunks):
                cuts = np.sort(np.append(rng.integers(0, max(1, c + n), mod["docs"]), -1))
                first += [int(cuts[cuts <= c + j][-1]) for j in range(n)]
            self.first = np.array(first, np.int32)
            if mod.get("empty"):  # rows with nothing to attend to, a whole chunk of them among these
                self.first[rng.random(self.T) < 0.1] = 1 << 30
                self.first[self.start[1]:self.start[2]] = 4000
        self.prefix = np.array([mod["prefix"] + 30 * s for s in range(len(chunks))], np.int32) if mod.get("prefix") else None
        self.ref, self.shares = su.ref_scored(self.q, self.where, self.pools, self.tables, self.lens, self.scale, self.cap,
                                              self.window, self.slopes, self.first, self.prefix)
        self.kd, self.vd = self.pools.dev()
        self.dev_tables = self.tables.copy()
        self.pools.spoil_tail(self.tables, self.lens, self.kd, self.vd)
        # what no row of the sequence sees
        for s, L in enumerate(self.lens):
            seen = np.zeros(L, bool)
            for r in range(self.start[s], self.start[s + 1]):
                seen[self.shares[r][0]] = True
            for t in np.flatnonzero(~seen):
                spoil_rows(self.pools, self.kd, self.vd, int(self.tables[s][t // 16]), t % 16, t % 16 + 1)
            if seen.any() and kv in qu.TORCH:
                self.dev_tables[s, :int(np.argmax(seen)) // 16] = 1 << 28

    def score(self):
        dev = lambda a: None if a is None else i32(a)
        return self.pk.ScoreMod(cap=self.cap, window=self.window, slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                                first=dev(self.first), prefix_lens=dev(self.prefix))

    def run(self, plan=False, out=None):
        pk = self.pk
        q = self.q.cuda()
        out = torch.full_like(q, 7.0) if out is None else out
        S, MB = self.tables.shape
        need = pk.prefill_workspace_bytes(self.kv, S, self.pools.Hkv, self.D, MB)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
        work = i32(pk.prefill_plan(self.start, self.lens, self.Hq, self.pools.Hkv, self.n_max)) if plan else None
        pk.paged_attention_prefill_scored(q, self.kd, self.vd, self.pools.desc, i32(self.start), self.n_max, i32(self.dev_tables),
                                          i32(self.lens), self.scale, out, self.score(), work_units=work, workspace=ws)
        return out

    def check(self, out, rows=slice(None)):
        got = out.double().cpu().numpy()[rows]
        assert np.all(np.isfinite(got)), np.argwhere(~np.isfinite(got))[:5]
        tol = TOL["f16" if self.q_dtype == "f16" and self.kv == "f16" else "bf16"]
        vmax = float(np.abs(self.pools.vh).max())
        err = max_error(got, self.ref[rows], self.q_dtype, tol, vmax)
        assert err <= tol, err
        for r in np.arange(self.T)[rows]:
            if not len(self.shares[r][0]):
                assert bool((out[int(r)] == 0).all())


@pytest.mark.parametrize("mod", list(SCORES))
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (64, 1, 8), (128, 2, 1), (128, 1, 2), (128, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill_scored(pk, dtype, D, Hkv, G, mod):
    c = Case(pk, dtype, D, Hkv, G, dtype, SCORES[mod])
    c.check(c.run())
    c.check(c.run(plan=True))
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("mod", ["cap_of_large_scores", "all"])
@pytest.mark.parametrize("kv", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("D,G,q_dtype", [(64, 2, "f16"), (128, 4, "bf16")])
def test_prefill_scored_over_staged_pools(pk, kv, D, G, q_dtype, mod):
    c = Case(pk, kv, D, 2, G, q_dtype, SCORES[mod], seed=2)
    if kv in qu.BITS:
        # the copy that is attended to holds the values rounded once to q's type
        c.pools.kh, c.pools.vh = (qu.round_to(x, q_dtype).astype(np.float64) for x in (c.pools.kh, c.pools.vh))
        c.ref, c.shares = su.ref_scored(c.q, c.where, c.pools, c.tables, c.lens, c.scale, c.cap, c.window, c.slopes, c.first, c.prefix)
    c.check(c.run())
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(pk, D, G, bad):
    """A token of one document and a late token of another hold such values: the other rows are what they were."""
    c = Case(pk, "bf16", D, 1, G, "bf16", dict(docs=3), chunks=[(100, 700), (0, 90)], seed=6)
    hit = [(0, 250), (0, 640), (0, 799), (1, 41)]
    for s, t in hit:
        c.vd[int(c.tables[s][t // 16]), :, t % 16, 3 + t % 50] = bad
    out = c.run()
    sees = np.array([any(hs == s and ht in set(t.tolist()) for hs, ht in hit) for (s, _), (t, _) in zip(c.where, c.shares)])
    assert sees.any() and not sees.all()
    c.check(out, ~sees)
    got = out.double().cpu().numpy()[sees]
    assert np.all((~np.isfinite(got)).any(-1))  # NaN in whole, or where the products give it
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("short", [0, 1])
@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 1), (128, 1, 1), (128, 1, 8), (64, 20, 1)])
def test_one_half_of_a_unit_is_through_long_before_the_other(pk, D, Hkv, G, short):
    """Rows of one Q tile see nothing, those of the other a long context; then the next unit, and the other way round.
    Few units have one Q tile each, unless a plan names them; 20 heads' have two."""
    RQ, ctx = 128 // G, 2600
    n = 4 * RQ
    c = Case(pk, "f16", D, Hkv, G, "f16", {}, chunks=[(ctx, n), (0, 40)], seed=9)
    first = np.zeros(n + 40, np.int32)
    half = np.arange(n) // RQ % 2 == short
    first[:n][half] = ctx + 4 * RQ  # nothing to see: the unit's one tile
    c.first = first
    c.ref, c.shares = su.ref_scored(c.q, c.where, c.pools, c.tables, c.lens, c.scale, 0.0, 0, None, first, None)
    c.check(c.run())
    c.check(c.run(plan=True))
    for t in (3, 127, ctx - 1):  # seen by the other half alone
        c.vd[int(c.tables[0][t // 16]), :, t % 16, 1 + t % 60] = float("nan")
    for plan in (False, True):
        out = c.run(plan)
        c.check(out, np.append(half, np.ones(40, bool)))
        got = out.double().cpu().numpy()[:n][~half]
        assert np.all((~np.isfinite(got)).any(-1))
    assert pk.get_device_error() == 0


def test_long_context_behind_a_window(pk):
    """Many tiles in front of the window, a ring of value masks gone round many times."""
    c = Case(pk, "bf16", 128, 1, 4, "bf16", dict(window=3000, cap=40.0, docs=40), chunks=[(9000, 200)], seed=8)
    c.check(c.run())
    c = Case(pk, "bf16", 64, 1, 8, "bf16", dict(slopes=True), chunks=[(6000, 100)], seed=8)
    c.check(c.run())
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_plain_scores_give_what_prefill_gives(pk, dtype):
    c = Case(pk, dtype, 128, 2, 4, dtype, {}, seed=4)
    want = torch.zeros_like(c.q, device="cuda")
    pk.paged_attention_prefill(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.start), c.n_max, i32(c.tables), i32(c.lens), c.scale, want)
    assert torch.equal(c.run(), want)
    out = torch.zeros_like(want)
    pk.paged_attention_prefill_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.start), c.n_max, i32(c.tables), i32(c.lens), c.scale, out)
    assert torch.equal(out, want)


def test_one_row_gives_what_scored_decode_gives(pk):
    """The last row of each sequence, as a chunk of one and as a decode step: within the rounding of the output."""
    c = Case(pk, "f16", 128, 2, 4, "f16", dict(cap=20.0, window=100, slopes=True), chunks=[(99, 1), (300, 1), (0, 1)], seed=3)
    out = c.run()
    c.check(out)
    dec = torch.zeros_like(out)
    ws = torch.zeros(pk.decode_scored_workspace_bytes(3, 8, 128, 301, 100), dtype=torch.uint8, device="cuda")
    pk.paged_attention_decode_scored(c.q.cuda(), c.kd, c.vd, c.pools.desc, i32(c.dev_tables), i32(c.lens), 301, c.scale, dec, c.score(), workspace=ws)
    c.check(dec)
    assert pk.get_device_error() == 0


def test_captured_and_replayed_after_its_masks_changed(pk):
    c = Case(pk, "bf16", 128, 2, 4, "bf16", SCORES["all"], seed=5)
    q, out = c.q.cuda(), torch.zeros_like(c.q, device="cuda")
    st, lens, tb = i32(c.start), i32(c.lens), i32(c.dev_tables)
    sc = c.score()
    first = sc.first.clone()
    sc.first.zero_()
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        pk.paged_attention_prefill_scored(q, c.kd, c.vd, c.pools.desc, st, c.n_max, tb, lens, c.scale, out, sc)
    sc.first.copy_(first)
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(out)
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("S", [1, 31, 32, 33, 70])
def test_many_sequences_in_the_order_of_their_reach(pk, S):
    """Without a plan, batches of up to 32 sequences are taken by their reach, larger ones in the order of the grid."""
    rng = np.random.default_rng(S)
    chunks = [(int(rng.integers(0, 200)), int(rng.choice([0, 1, 40, 64, 65, 130]))) for _ in range(S)]
    chunks[0] = (77, 133)
    c = Case(pk, "bf16", 64, 1, 4, "bf16", dict(window=90, cap=30.0), chunks=chunks, seed=S)
    c.check(c.run())
    c.check(c.run(plan=True))
    assert pk.get_device_error() == 0


def test_inconsistent_sequences_are_reported_and_skipped(pk):
    c = Case(pk, "bf16", 128, 1, 4, "bf16", {}, chunks=[(10, 40), (0, 70), (5, 30)])
    q, out = c.q.cuda(), torch.full_like(c.q, 7.0, device="cuda")
    lens = i32([50, 69, 35])  # the second holds fewer tokens than its chunk
    pk.paged_attention_prefill_scored(q, c.kd, c.vd, c.pools.desc, i32(c.start), 70, i32(c.tables), lens, c.scale, out)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    assert bool((out[40:110] == 7).all())
    c.check(out, np.r_[0:40, 110:140])
    # chunks past max_query_len lose rows, and say so; the first rows are there
    out.fill_(7.0)
    pk.paged_attention_prefill_scored(q, c.kd, c.vd, c.pools.desc, i32(c.start), 40, i32(c.tables), i32(c.lens), c.scale, out)
    assert pk.get_device_error() == pk.DEVERR_SEQ_LEN
    c.check(out, np.r_[0:40, 110:140])
