"""Cases of rotary writes, of scored attention and of eviction over the paged cache, with plain forms of all three.

Five operators of a serving step:

  rope     queries and keys rotated by their positions, and the step's keys and
           values written to their slots
  decode   single-query attention whose scores are capped, biased by distance
           and masked by a window and a first position
  prefill  attention of a chunk's rows with the same scores, over documents
           packed in one sequence and over a prefix seen in both directions
  weights  decode that also leaves each cached token's share of the softmax,
           summed over the query heads of its KV head
  evict    the tokens of the highest weights kept: chosen for each (sequence,
           KV head) and moved together into fewer blocks

Rotation: pair i of the first R of a head's D elements turns by the angle
position * f_i; the pair is (i, i + R/2), or (2i, 2i + 1) when interleaved.
f_i = base^(-2i/R), scaled for a context `factor` times the original one of
L0 positions: with r = L0 f_i / 2 pi turns over the original context and g =
clamp((r - 1) / (high - 1), 0, 1), f_i becomes (1 - g) f_i / factor + g f_i,
and cos and sin are multiplied by 0.1 ln(factor) + 1.

Score of the query at position p with the key at position t:
    x = scale * q.k;  x = cap * tanh(x / cap);  x = x - slope_head * |p - t|
where t >= first, t > p - window, and t <= p or t < prefix; -inf elsewhere.  A
row that nothing is left of gives zeros.
"""
import math

import numpy as np
import torch

own = False

B = 16  # tokens of a block
NEG = float("-inf")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of each of 64 sequences, the whole head rotated
        dict(name="rope_step", op="rope", T=64, Hq=32, Hkv=8, D=128, R=128, inter=False, factor=1.0, ctx=4096, pad=0, dtype="bf16"),
        # prefill chunks, 8192 tokens, positions of a context extended 16 times, some padding
        dict(name="rope_chunk", op="rope", T=8192, Hq=32, Hkv=8, D=128, R=128, inter=False, factor=16.0, ctx=131072, pad=100, dtype="bf16"),
        # four short sequences with capped scores: what a call costs at least
        dict(name="decode_cap_tiny", op="decode", S=4, lo=17, hi=100, Hq=8, Hkv=8, D=64, cap=30.0, window=0, slopes=False, lead=True, kv="f16", dtype="f16"),
        # long contexts behind a sliding window, capped: most of the cache is not read
        dict(name="decode_window", op="decode", S=64, lo=2048, hi=16384, Hq=32, Hkv=8, D=128, cap=50.0, window=1024, slopes=False, lead=False, kv="bf16", dtype="bf16"),
        # one query head to a KV head, scores falling with distance
        dict(name="decode_bias_mha", op="decode", S=64, lo=512, hi=4096, Hq=32, Hkv=32, D=128, cap=0.0, window=0, slopes=True, lead=False, kv="bf16", dtype="bf16"),
        # chunks of 512 new tokens after contexts of different lengths, capped
        dict(name="prefill_cap_chunk", op="prefill", S=8, n=512, lo=0, hi=3584, Hq=32, Hkv=8, D=128, cap=50.0, window=0, slopes=False, docs=0, prefix=0, dtype="bf16"),
        # whole prompts of documents packed together, a window of 1024
        dict(name="prefill_docs_window", op="prefill", S=4, n=4096, lo=0, hi=0, Hq=32, Hkv=8, D=128, cap=0.0, window=1024, slopes=False, docs=5, prefix=0, dtype="bf16"),
        # prompts whose first part is seen in both directions, scores falling with distance
        dict(name="prefill_prefix_bias", op="prefill", S=4, n=2048, lo=0, hi=0, Hq=32, Hkv=32, D=128, cap=0.0, window=0, slopes=True, docs=0, prefix=700, dtype="bf16"),
        # one long sequence of a step that is followed by an eviction
        dict(name="weights_one", op="weights", S=1, lo=8190, hi=8190, Hq=64, Hkv=8, D=128, cap=0.0, kv="bf16", dtype="bf16"),
        # a batch of them
        dict(name="weights_batch", op="weights", S=64, lo=512, hi=4096, Hq=32, Hkv=8, D=128, cap=0.0, kv="bf16", dtype="bf16"),
        # that long sequence, a quarter of it kept
        dict(name="evict_one", op="evict", S=1, lo=8190, hi=8190, Hkv=8, D=128, keep=2048, sink=4, recent=64, dtype="bf16"),
        # a batch at its budget, a quarter to a half kept
        dict(name="evict_batch", op="evict", S=32, lo=2048, hi=4096, Hkv=8, D=128, keep=1000, sink=4, recent=256, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "prefill", "prefill", "weights", "evict"])
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "f16"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    cap = rng.choice([0.0, round(rng.uniform(5.0, 60.0), 2)])
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 8192), Hq=min(Hkv * G, 32), Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 16]), inter=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 32.0]), ctx=_log(rng, 128, 1000000), pad=rng.choice([0, 3, 7]), dtype=dtype)
    if op == "prefill":
        Hkv, G = min(Hkv, 4), min(G, 4)
        n = _log(rng, 1, 1500)
        hi = _log(rng, 1, 4000)
        S = _log(rng, 1, max(1, min(8, 12000 // (n + hi))))
        return dict(op=op, S=S, n=n, lo=rng.randrange(0, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, cap=cap, window=rng.choice([0, 0, _log(rng, 1, 2000)]),
                    slopes=rng.random() < 0.5, docs=rng.choice([0, 0, rng.randrange(1, 9)]), prefix=rng.choice([0, 0, _log(rng, 1, n + hi)]), dtype=dtype)
    hi = _log(rng, 1, 32768)
    S = _log(rng, 1, max(1, min(128, 1000000 // (hi * Hkv))))
    lo = rng.randrange(max(1, hi // 2), hi + 1)
    c = dict(op=op, S=S, lo=lo, hi=hi, Hkv=Hkv, D=D, dtype=dtype)
    if op == "evict":
        keep = _log(rng, 1, hi)
        sink = rng.randrange(0, min(keep, 8) + 1)
        return dict(c, keep=keep, sink=sink, recent=rng.randrange(0, keep - sink + 1))
    c.update(Hq=Hkv * G, cap=cap, kv=rng.choice([dtype, dtype, "e4m3"]))
    if op == "decode":
        c.update(window=rng.choice([0, _log(rng, 1, hi)]), slopes=rng.random() < 0.5, lead=rng.random() < 0.3)
    return c


# ----------------------------------------------------------- what is in hand
def _rng(c):
    """Lengths go by the sizes alone, so that work() counts the same ones."""
    return np.random.default_rng(c["S"] * 7919 + c["hi"] * 31 + c["Hkv"])


def _lens(c):
    """(tokens in the cache, new ones among them) of every sequence."""
    r = _rng(c)
    lens = r.integers(c["lo"], c["hi"] + 1, size=c["S"]).astype(np.int64)
    if c["op"] != "prefill":
        return lens, np.ones_like(lens)
    new = c["n"] - r.integers(0, max(1, c["n"] // 8), size=c["S"])
    new[0] = c["n"]
    return lens + new, new


def _first(c, lens, new):
    """First position that each row may attend to."""
    r = _rng(c)
    if c["op"] == "prefill":
        rows = []
        for L, n in zip(lens, new):
            cuts = np.sort(np.append(r.integers(0, L, size=c["docs"]), 0))
            pos = np.arange(L - n, L)
            rows.append(cuts[np.searchsorted(cuts, pos, side="right") - 1])
        return np.concatenate(rows).astype(np.int32)
    return r.integers(0, np.maximum(1, lens // 3 + 1)).astype(np.int32)  # padding in front


def _blocks(n):
    return (n + B - 1) // B


def _tables(counts, gen, spare=4):
    """Block tables over a pool in random order, part of it free; each count a list of blocks a sequence."""
    used = int(sum(int(n.sum()) for n in counts))
    NB = used + used // 10 + spare
    ids = torch.randperm(NB, generator=gen, device="cuda", dtype=torch.int32)[:used].cpu().numpy()
    out, at = [], 0
    for nb in counts:
        t = np.full((len(nb), max(1, int(nb.max()))), -1, np.int32)
        for s, n in enumerate(nb):
            t[s, :n] = ids[at:at + n]
            at += n
        out.append(torch.from_numpy(t).cuda())
    return NB, out


def _randn(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * gain).to(dtype)


def _inv_freq(c):
    """Radians a position turns each pair by, in 64 bits; factor on cos and sin."""
    i = np.arange(c["R"] // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / c["R"])
    if c["factor"] == 1.0:
        return f, 1.0
    g = np.clip((4096 * f / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
    return (1 - g) * f / c["factor"] + g * f, 0.1 * math.log(c["factor"]) + 1.0


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(c)
    dt, H, D = DT[c["dtype"]], c["Hkv"], c["D"]
    if c["op"] == "rope":
        T, Hq = c["T"], c["Hq"]
        NB = _blocks(T) + 5
        # the rows of a fused projection: queries, keys and values of a token side by side
        qkv = _randn(gen, (T, Hq + 2 * H, D), dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
        s["positions"] = torch.randint(0, c["ctx"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        blocks = torch.randperm(NB, generator=gen, device="cuda")[:_blocks(T)]
        slots = (blocks[:, None] * B + torch.arange(B, device="cuda")).reshape(-1)[:T].contiguous()
        live = torch.arange(T)
        if c["pad"]:
            slots[::c["pad"]] = -1  # padding of a batch
            live = live[live % c["pad"] != 0]
        s["slots"], s["live"], s["NB"] = slots, live.cuda(), NB
        f, s["magnitude"] = _inv_freq(c)
        s["inv_freq"] = torch.from_numpy(f).cuda()
        turns = f / (2 * math.pi)  # the table that a program keeps: turns a position, as two binary32
        hi = turns.astype(np.float32)
        s["freqs"] = torch.from_numpy(np.stack([hi, (turns - hi).astype(np.float32)], -1)).cuda()
        s["kc"], s["vc"] = (torch.zeros(NB, H, B, D, dtype=dt, device="cuda") for _ in range(2))
        return s
    lens, new = _lens(c)
    s["max_len"], s["lens"] = int(lens.max()), torch.from_numpy(lens.astype(np.int32)).cuda()
    counts = [_blocks(lens)]
    if c["op"] == "evict":
        counts.append(_blocks(np.minimum(lens, c["keep"])))
    s["NB"], tables = _tables(counts, gen)
    s["tables"] = tables[0]
    k, v = _randn(gen, (s["NB"], H, B, D), dt), _randn(gen, (s["NB"], H, B, D), dt)
    s["k_scale"] = s["v_scale"] = 1.0
    if c.get("kv") == "e4m3":
        s["k_scale"], s["v_scale"] = 0.0125, 0.015625
        k, v = (k.float() / s["k_scale"]).to(torch.float8_e4m3fn), (v.float() / s["v_scale"]).to(torch.float8_e4m3fn)
    s["kc"], s["vc"] = k, v
    if c["op"] == "evict":
        s["dst"] = tables[1]
        # accumulated weights: a few heavy tokens, many light ones, some that nothing ever looked at
        w = torch.exp(3 * torch.randn(s["NB"], H, B, generator=gen, device="cuda") - 6)
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.1, 0.0, w).contiguous()
        s["kept"] = torch.full((c["S"], H, c["keep"]), -1, dtype=torch.int32, device="cuda")
        return s
    T, Hq = int(new.sum()), c["Hq"]
    s["q"] = _randn(gen, (T, Hq, D), dt, 3.0)
    s["out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    s["slopes_t"] = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq) if c.get("slopes") else None
    s["first"] = torch.from_numpy(_first(c, lens, new)).cuda() if c.get("lead") or c.get("docs") else None
    s["prefix_t"] = None
    if c["op"] == "prefill":
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["start"], s["n_max"] = torch.from_numpy(start).cuda(), int(new.max())
        # row j of sequence s as a row of q, and back
        grid = start[:-1, None] + np.minimum(np.arange(s["n_max"])[None, :], new[:, None] - 1)
        s["rows"] = torch.from_numpy(grid).cuda().long()
        s["back"] = torch.from_numpy(np.concatenate([i * s["n_max"] + np.arange(n) for i, n in enumerate(new)])).cuda()
        if c["prefix"]:
            s["prefix_t"] = torch.from_numpy(np.minimum(c["prefix"], lens).astype(np.int32)).cuda()
    if c["op"] == "weights":
        s["weights"] = torch.zeros(s["NB"], H, B, dtype=torch.float32, device="cuda")
    tokens = s["tables"].shape[1] * B
    rows = c["S"] * Hq
    # what a call keeps between its kernels: a maximum, a sum and D values for each query row and stretch of
    # 256 tokens, and for the weights a score for each row and token
    s["ws"] = torch.empty(rows * -(-tokens // 256) * (D + 2) * 4 + (rows * tokens * 4 if c["op"] == "weights" else 0) + 8192,
                          dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, R, inter):
    """x [T, H, D] in 32 bits; cos, sin [T, R/2]."""
    c, n = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * c - b * n, b * c + a * n
    turned = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ((f(angle) * s["magnitude"]).float() for f in (torch.cos, torch.sin))
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, s["R"], s["inter"]))
    live = s["live"]
    slots = s["slots"][live]
    blk, off = torch.div(slots, B, rounding_mode="floor"), slots % B
    s["kc"][blk, :, off] = _rotate(s["k"].float(), cos, sin, s["R"], s["inter"])[live].to(s["kc"].dtype)
    s["vc"][blk, :, off] = s["v"][live]
    return s["q_out"], s["kc"], s["vc"]


def _rows(s, pool, scale):
    """Every sequence's rows of a pool, [S][Hkv][tokens][D] in 32 bits."""
    got = pool[torch.clamp(s["tables"], min=0).long()].float() * scale  # [S][MB][H][B][D]
    return got.permute(0, 2, 1, 3, 4).reshape(s["S"], s["Hkv"], -1, s["D"])


def _attend(s, q, pos, first, prefix):
    """q [S][n][Hq][D] in 32 bits at positions pos [S][n]: outputs [S][n][Hq][D] and the softmax [S][Hkv][G][n][tokens]."""
    S, H, D = s["S"], s["Hkv"], s["D"]
    n, G = q.shape[1], s["Hq"] // H
    k, v = _rows(s, s["kc"], s["k_scale"]), _rows(s, s["vc"], s["v_scale"])
    q = q.reshape(S, n, H, G, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(S, H, G * n, D), k.transpose(-1, -2)).reshape(S, H, G, n, -1) * D ** -0.5
    if s["cap"] > 0:
        x = s["cap"] * torch.tanh(x / s["cap"])
    t = torch.arange(k.shape[2], device="cuda")
    p = pos[..., None]
    if s.get("slopes_t") is not None:
        x = x - s["slopes_t"].reshape(1, H, G, 1, 1) * (p - t).abs().float()[:, None, None]
    ok = (t <= p) if prefix is None else (t <= p) | (t < prefix[:, None, None])
    ok = ok & (t < s["lens"][:, None, None])
    if s.get("window"):
        ok = ok & (t > p - s["window"])
    if first is not None:
        ok = ok & (t >= first[..., None])
    ok = ok[:, None, None]
    x = torch.where(ok, x, NEG)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top > NEG, top, 0.0))
    w = w / torch.clamp(w.sum(-1, keepdim=True), min=1e-30)
    out = torch.matmul(w.reshape(S, H, G * n, -1), v).reshape(S, H, G, n, D)
    return out.permute(0, 3, 1, 2, 4).reshape(S, n, s["Hq"], D), w


def _plain_decode(s):
    first = s["first"][:, None] if s["first"] is not None else None
    out, w = _attend(s, s["q"].float()[:, None], (s["lens"] - 1)[:, None], first, None)
    s["out"].copy_(out[:, 0])
    if s["op"] == "decode":
        return s["out"]
    # every cached token's share, to its slot; entries past a sequence's blocks repeat its first block's
    w = w[:, :, :, 0].sum(2).reshape(s["S"], s["Hkv"], -1, B).permute(0, 2, 1, 3)  # [S][MB][H][B]
    t = s["tables"].long()
    at = torch.where(t >= 0, t, t[:, :1])
    inside = torch.arange(t.shape[1] * B, device="cuda").reshape(1, -1, 1, B) < s["lens"][:, None, None, None]
    w = torch.where(inside, w, s["weights"][at])
    w = torch.where((t >= 0)[:, :, None, None], w, w[:, :1])
    s["weights"][at] = w
    return s["out"], s["weights"]


def _plain_prefill(s):
    rows = s["rows"]
    new = (s["start"][1:] - s["start"][:-1])[:, None]
    j = torch.minimum(torch.arange(s["n_max"], device="cuda", dtype=torch.int32)[None, :], new - 1)
    pos = s["lens"][:, None] - new + j
    first = s["first"][rows] if s["first"] is not None else None
    out, _ = _attend(s, s["q"].float()[rows], pos, first, s["prefix_t"])
    s["out"].copy_(out.flatten(0, 1)[s["back"]])
    return s["out"]


def _plain_evict(s):
    S, H, n = s["S"], s["Hkv"], s["keep"]
    src, dst = torch.clamp(s["tables"], min=0).long(), s["dst"].long()
    L = s["lens"].long()[:, None, None]
    w = s["weights"][src].permute(0, 2, 1, 3).reshape(S, H, -1)
    t = torch.arange(w.shape[-1], device="cuda")
    w = torch.where((t < s["sink"]) | (t >= L - s["recent"]), float("inf"), w)
    w = torch.where(t < L, w, NEG)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :n]
    far = 1 << 30
    order = torch.sort(torch.where(order < L, order, far), dim=-1).values
    s["kept"].fill_(-1)
    s["kept"][..., :order.shape[-1]] = torch.where(order < far, order, -1).int()
    # entry i of a row moves to position i; entries past the row's end repeat its first one
    m = order.shape[-1]
    i = torch.arange(m, device="cuda").expand(S, H, m)
    live = order < far
    i, order = torch.where(live, i, 0), torch.where(live, order, order[..., :1])
    seq, head = torch.arange(S, device="cuda")[:, None, None], torch.arange(H, device="cuda")[None, :, None]
    fb, tb = src[seq, torch.div(order, B, rounding_mode="floor")], dst[seq, torch.div(i, B, rounding_mode="floor")]
    for pool in (s["kc"], s["vc"], s["weights"]):
        pool[tb, head, i % B] = pool[fb, head, order % B]
    return s["kept"], s["kc"], s["vc"], s["weights"]


def _own(s):
    from paged_kv_cache_10_gb300 import pagedkv as pk
    desc = pk.CacheDesc(num_blocks=s["NB"], num_kv_heads=s["Hkv"], head_size=s["D"], kv_dtype=s.get("kv", s["dtype"]),
                        k_scale=s.get("k_scale", 1.0), v_scale=s.get("v_scale", 1.0))
    op = s["op"]
    if op == "rope":
        pk.paged_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"], s["kc"], s["vc"], desc,
                             s["q_out"], interleaved=s["inter"], magnitude=s["magnitude"])
        return s["q_out"], s["kc"], s["vc"]
    if op == "evict":
        pk.select_tokens(s["weights"], desc, s["tables"], s["lens"], s["max_len"], s["kept"], sink_tokens=s["sink"],
                         recent_tokens=s["recent"])
        pk.paged_kv_compact(s["kept"], s["kc"], s["vc"], desc, s["tables"], s["lens"], s["dst"], weights=s["weights"])
        return s["kept"], s["kc"], s["vc"], s["weights"]
    score = pk.ScoreMod(cap=s["cap"], window=s.get("window", 0), slopes=s["slopes_t"], first=s["first"], prefix_lens=s["prefix_t"])
    if op == "prefill":
        pk.paged_attention_prefill_scored(s["q"], s["kc"], s["vc"], desc, s["start"], s["n_max"], s["tables"], s["lens"],
                                          s["D"] ** -0.5, s["out"], score)
        return s["out"]
    weights = s["weights"] if op == "weights" else None
    pk.paged_attention_decode_scored(s["q"], s["kc"], s["vc"], desc, s["tables"], s["lens"], s["max_len"], s["D"] ** -0.5,
                                     s["out"], score, weights=weights, workspace=s["ws"])
    return s["out"] if weights is None else (s["out"], weights)


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "decode": _plain_decode, "weights": _plain_decode, "prefill": _plain_prefill,
            "evict": _plain_evict}[s["op"]](s)


# ------------------------------------------------------ what a pass cannot do without
def _spans(c):
    """Lowest and highest key of every row, and the rows' sequences."""
    lens, new = _lens(c)
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
    seq = np.repeat(np.arange(c["S"]), new)
    lo = np.zeros_like(pos)
    if c.get("lead") or c.get("docs"):
        lo = _first(c, lens, new).astype(np.int64)
    if c.get("window"):
        lo = np.maximum(lo, pos - c["window"] + 1)
    hi = pos + 1
    if c.get("prefix"):
        hi = np.maximum(hi, np.minimum(c["prefix"], lens)[seq])
    return lo, hi, seq


def work(c):
    H, D = c["Hkv"], c["D"]
    if c["op"] == "rope":
        live = c["T"] - (len(range(0, c["T"], c["pad"])) if c["pad"] else 0)
        return {"bytes": c["T"] * (12 + 4 * c["Hq"] * D) + live * H * 8 * D + c["R"] * 4, "flops": (c["T"] * c["Hq"] + live * H) * c["R"] * 3}
    lens, new = _lens(c)
    if c["op"] == "evict":
        kept = int(np.minimum(lens, c["keep"]).sum())
        nb = int(_blocks(lens).sum())
        return {"bytes": int(lens.sum()) * H * 4 + kept * H * (4 + 2 * 4 * D + 4) + 4 * nb + 4 * c["S"], "flops": int(lens.sum()) * H}
    lo, hi, seq = _spans(c)
    each = np.maximum(0, hi - lo)
    pairs = int(each.sum())
    elem = 1 if c.get("kv") == "e4m3" else 2
    # the keys that some row of the sequence attends to
    low, high = np.full(c["S"], 1 << 40), np.zeros(c["S"], np.int64)
    some = each > 0
    np.minimum.at(low, seq[some], lo[some])
    np.maximum.at(high, seq[some], hi[some])
    keys = int(np.maximum(0, high - low).sum())
    io = 2 * int(new.sum()) * c["Hq"] * D * 2
    extra = int(lens.sum()) * H * 4 if c["op"] == "weights" else 0
    return {"bytes": keys * H * 2 * D * elem + io + int(_blocks(lens).sum()) * 4 + extra, "flops": pairs * c["Hq"] * 4 * D}


# ----------------------------------------- the definition in 64 bits, written apart
def _turned(x, angle, magnitude, R, inter):
    """Rotation as a product of complex numbers."""
    first, rest = x[..., :R].double(), x[..., R:].double()
    pairs = first.unflatten(-1, (R // 2, 2)) if inter else first.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    got = torch.view_as_real(z)
    got = got.flatten(-2) if inter else got.transpose(-1, -2).flatten(-2)
    return torch.cat([got, rest], -1)


def exact(c, seed):
    s = prepare(c, seed)
    H, D = c["Hkv"], c["D"]
    if c["op"] == "rope":
        angle = torch.outer(s["positions"].double(), s["inv_freq"])
        q, k = (_turned(s[x], angle, s["magnitude"], c["R"], c["inter"]) for x in ("q", "k"))
        kc, vc = s["kc"].double(), s["vc"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // B, :, slot % B], vc[slot // B, :, slot % B] = k[t], s["v"][t].double()
        return q, kc, vc
    lens, tables = s["lens"].tolist(), s["tables"].long()
    if c["op"] == "evict":
        kept = np.full((c["S"], H, c["keep"]), -1, np.int32)
        pools = [s[x].double() for x in ("kc", "vc", "weights")]
        source = [p.clone() for p in pools]
        for i, L in enumerate(lens):
            w = s["weights"][tables[i, :_blocks(L)]].permute(1, 0, 2).reshape(H, -1)[:, :L].cpu().numpy()
            for h in range(H):
                forced = np.zeros(L, bool)
                forced[:c["sink"]] = True
                forced[L - min(L, c["recent"]):] = True
                order = np.lexsort((np.arange(L), -w[h], ~forced))[:c["keep"]]
                ids = np.sort(order)
                kept[i, h, :len(ids)] = ids
                a = torch.from_numpy(ids).cuda()
                b = torch.arange(len(ids), device="cuda")
                for p, q in zip(pools, source):
                    p[s["dst"][i].long()[b // B], h, b % B] = q[tables[i][a // B], h, a % B]
        return (torch.from_numpy(kept), *pools)
    lo, hi, seq = _spans(c)
    if sum(int((seq == i).sum()) * L for i, L in enumerate(lens)) * c["Hq"] * D > 4e11:
        return None
    G = c["Hq"] // H
    _, new = _lens(c)
    out = torch.zeros(len(seq), c["Hq"], D, dtype=torch.float64, device="cuda")
    weights = torch.zeros(s["NB"], H, B, dtype=torch.float64, device="cuda") if c["op"] == "weights" else None
    at = 0
    for i, L in enumerate(lens):
        n = int(new[i])
        rows = slice(at, at + n)
        a, b = (torch.from_numpy(x[rows]).cuda() for x in (lo, hi))
        t = torch.arange(L, device="cuda")
        hidden = (t < a[:, None]) | (t >= b[:, None])
        gap = (torch.arange(L - n, L, device="cuda")[:, None] - t).abs().double()
        for h in range(H):
            k, v = (s[x][tables[i, :_blocks(L)], h].double().reshape(-1, D)[:L] * s[y] for x, y in (("kc", "k_scale"), ("vc", "v_scale")))
            for g in range(h * G, h * G + G):
                x = s["q"][rows, g].double() @ k.T / math.sqrt(D)
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                if s["slopes_t"] is not None:
                    x = x - s["slopes_t"][g].double() * gap
                p = torch.softmax(x.masked_fill(hidden, NEG), -1).nan_to_num(0.0)
                out[rows, g] = p @ v
                if weights is not None:
                    weights[tables[i][t // B], h, t % B] += p[0]
        at += n
    return out if weights is None else (out, weights)
