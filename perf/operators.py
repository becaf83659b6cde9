"""Cases of the integer-coded KV cache and of sparse decode, with plain forms of both.

Five operators of the decode step over the paged cache:

  write_read  K/V rows quantised to 8 or 4 bits as they are written to their
              slots, and read back to 16 bits by slot
  decode      single-query attention over such a cache
  bounds      channelwise minimum and maximum of the keys of every block that
              received new tokens
  select      the blocks that each (sequence, KV head) attends to: those with
              the highest upper bound of a query's score
  sparse      single-query attention over the selected blocks only

A row (one token of one KV head) of D values is held as unsigned codes of
`bits` bits with a binary32 scale and zero: lo, hi its smallest and largest
value, scale = (hi - lo) / (2^bits - 1) (0 where that is below 2^-126),
zero = lo, code = min(rint((x - lo) * (1 / scale)), 2^bits - 1), every step
in binary32; the value held is zero + scale * code.

A tile (one block of one KV head, 16 tokens) is 16 rows of RB = D * bits / 8
code bytes and then 16 pairs (scale, zero).  Byte b of a row holds element b
(8 bits) or elements 2b (low half) and 2b + 1 (4 bits).  Byte b of token t is
at, for keys, panel b // 64 of [16 tokens][min(RB, 64)] bytes; for values, byte
x = (b // 2) * 4 + (t % 2) * 2 + b % 2 of token pair t // 2, panel x // 32 of
[8 pairs][32] bytes.
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
        # one decode step's new tokens of 64 sequences of a 32-head cache
        dict(name="write_int8_step", op="write_read", T=64, Hkv=32, D=128, bits=8, dtype="bf16", pad=0),
        # a batch of prefill chunks, 8192 tokens, grouped heads, 4 bits
        dict(name="write_int4_chunk", op="write_read", T=8192, Hkv=8, D=128, bits=4, dtype="bf16", pad=100),
        # four short sequences: what a call costs at least
        dict(name="decode_int8_tiny", op="decode", S=4, lo=17, hi=100, Hq=8, Hkv=8, D=64, bits=8, dtype="f16"),
        # many chats of up to 2048 tokens, four query heads to a KV head
        dict(name="decode_int8_gqa", op="decode", S=256, lo=128, hi=2048, Hq=32, Hkv=8, D=128, bits=8, dtype="bf16"),
        # one query head to a KV head: the cache's bytes are all there is
        dict(name="decode_int8_mha", op="decode", S=64, lo=512, hi=4096, Hq=32, Hkv=32, D=128, bits=8, dtype="bf16"),
        # long contexts, eight query heads to a KV head, 4 bits
        dict(name="decode_int4_long", op="decode", S=8, lo=32768, hi=32768, Hq=64, Hkv=8, D=128, bits=4, dtype="bf16"),
        # the block that each of 256 sequences' new token went to
        dict(name="bounds_step", op="bounds", S=256, lo=128, hi=2048, new=1, Hkv=8, D=128, dtype="bf16"),
        # chunks of 1024 new tokens of 8 prompts
        dict(name="bounds_chunk", op="bounds", S=8, lo=1024, hi=8192, new=1024, Hkv=8, D=128, dtype="bf16"),
        # one sequence of 512 blocks: latency
        dict(name="select_one", op="select", S=1, lo=8190, hi=8190, Hq=64, Hkv=8, D=128, n=128, sink=1, recent=2, dtype="bf16"),
        # a batch of long contexts, an eighth of the blocks kept
        dict(name="select_batch", op="select", S=32, lo=30000, hi=32768, Hq=32, Hkv=8, D=128, n=256, sink=4, recent=4, dtype="bf16"),
        # the attention that follows select_one
        dict(name="sparse_one", op="sparse", S=1, lo=8190, hi=8190, Hq=64, Hkv=8, D=128, n=128, kv="bf16", dtype="bf16"),
        # the attention that follows a selection in a batch
        dict(name="sparse_batch", op="sparse", S=32, lo=8192, hi=32768, Hq=32, Hkv=8, D=128, n=256, kv="bf16", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write_read", "decode", "decode", "bounds", "select", "select", "sparse", "sparse"])
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "f16"])
    Hkv, G = rng.choice([1, 2, 4, 8, 8, 32]), rng.choice([1, 2, 4, 8])
    if op == "write_read":
        return dict(op=op, T=_log(rng, 1, 8192), Hkv=min(Hkv, 8), D=D, bits=rng.choice([4, 8]), dtype=dtype, pad=rng.choice([0, 3, 7]))
    if op == "bounds":
        new = _log(rng, 1, 1024)
        S = _log(rng, 1, max(1, min(256, 16384 // new)))
        lo = new + rng.randrange(0, 500)
        return dict(op=op, S=S, lo=lo, hi=lo + rng.randrange(1, 2000), new=new, Hkv=min(Hkv, 8), D=D, dtype=dtype)
    # sequences and lengths whose tokens times heads stay under the listed ones'
    Hkv = min(Hkv, 8) if op != "decode" else Hkv
    hi = _log(rng, 512 if op == "select" else 1, 32768)
    S = _log(rng, 1, max(1, min(256, 2000000 // (hi * Hkv))))
    lo = rng.randrange(max(1, hi // 2), hi + 1)
    if op == "decode":
        return dict(op=op, S=S, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, bits=rng.choice([4, 8]), dtype=dtype)
    if op == "select":  # fewer blocks than the shortest sequence has
        n = _log(rng, 8, max(8, min(256, hi // 48)))
        return dict(op=op, S=S, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, n=n, sink=rng.randrange(0, 4), recent=rng.randrange(1, 4), dtype=dtype)
    n = _log(rng, 8, 256)
    kv = rng.choice([dtype, "int8", "int4"])
    return dict(op=op, S=S, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, n=n, kv=kv, dtype=dtype)


# ----------------------------------------------------------- what is in hand
def _lens(c):
    return np.random.default_rng(c["S"] * 7919 + c["hi"]).integers(c["lo"], c["hi"] + 1, size=c["S"]).astype(np.int32)


def _blocks(L):
    return (L + B - 1) // B


def _tables(lens, gen):
    """Block tables over a pool in random order, a tenth of it free."""
    nb = _blocks(lens.astype(np.int64))
    used, MB = int(nb.sum()), max(1, int(nb.max()))
    NB = used + used // 10 + 4
    ids = torch.randperm(NB, generator=gen, device="cuda", dtype=torch.int32)[:used].cpu().numpy()
    t = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for s, n in enumerate(nb):
        t[s, :n] = ids[at:at + n]
        at += n
    return NB, torch.from_numpy(t).cuda()


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _keys(gen, shape, dtype):
    """Keys: some channels sit off zero, as they do after a projection."""
    off = torch.randn(shape[-1], generator=gen, device="cuda") * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.1) * 3
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) + off).to(dtype)


def _places(D, bits, value):
    """Offset of every code byte of a tile, [16 tokens][RB]."""
    rb = D * bits // 8
    t, b = np.arange(16)[:, None], np.arange(rb)[None, :]
    if not value:
        w = min(rb, 64)
        return (b // 64) * 16 * w + t * w + b % 64
    x = (b // 2) * 4 + (t % 2) * 2 + b % 2
    return (x // 32) * 256 + (t // 2) * 32 + x % 32


def _encode(x, bits):
    x = x.float()
    top = float(2 ** bits - 1)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = (hi - lo) / torch.full_like(lo, top)  # a tensor: a plain number would be turned into its reciprocal
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
    return torch.clamp(torch.round((x - lo) * inv), max=top), scale, lo


def _pool(x, bits, value):
    """[NB][Hkv][16][D] values as a pool of tiles."""
    NB, H, _, D = x.shape
    rb = D * bits // 8
    pool = torch.empty(NB, H, 16 * rb + 128, dtype=torch.uint8, device="cuda")
    at = torch.from_numpy(_places(D, bits, value).reshape(-1)).cuda()
    step = max(1, (1 << 26) // (H * 16 * D))
    for i in range(0, NB, step):
        code, scale, zero = _encode(x[i:i + step], bits)
        code = code.to(torch.uint8)
        if bits == 4:
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        tile = pool[i:i + step]
        tile[:, :, at] = code.reshape(code.shape[0], H, 16 * rb)
        tile[:, :, 16 * rb:] = torch.cat([scale, zero], -1).contiguous().view(torch.uint8).reshape(code.shape[0], H, 128)
    return pool


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(c)
    dt = DT[c["dtype"]]
    H, D = c["Hkv"], c["D"]
    if c["op"] == "write_read":
        T = c["T"]
        NB = _blocks(T) + 5
        s["k"], s["v"] = _keys(gen, (T, H, D), dt), _randn(gen, (T, H, D), dt)
        slots = torch.randperm(NB, generator=gen, device="cuda")[:_blocks(T)]
        slots = (slots[:, None] * B + torch.arange(B, device="cuda")).reshape(-1)[:T].contiguous()
        if c["pad"]:
            slots[:: c["pad"]] = -1  # padding of a batch
        s["slots"], s["NB"] = slots, NB
        tile = 2 * D * c["bits"] + 128
        s["kc"], s["vc"] = (torch.zeros(NB, H, tile, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    else:
        lens = _lens(c)
        s["max_len"] = int(lens.max())
        s["NB"], s["tables"] = _tables(lens, gen)
        s["lens"] = torch.from_numpy(lens).cuda()
        shape = (s["NB"], H, B, D)
        if c["op"] == "bounds":
            s["kc"] = _keys(gen, shape, dt)
            new = np.minimum(c["new"], lens) - np.random.default_rng(seed).integers(0, max(1, c["new"] // 4), size=c["S"])
            s["new"], s["new_max"] = torch.from_numpy(new.astype(np.int32)).cuda(), int(new.max())
            s["bounds"] = torch.zeros(s["NB"], H, 2, D, dtype=dt, device="cuda")
        else:
            s["q"] = _randn(gen, (c["S"], c["Hq"], D), dt)
        if c["op"] == "select":
            k = _keys(gen, (s["NB"], H, 2, D), dt)
            s["bounds"] = torch.stack([k.amin(2) - 1, k.amax(2) + 1], 2).contiguous()
            s["selected"] = torch.empty(c["S"], H, c["n"], dtype=torch.int32, device="cuda")
        if c["op"] in ("decode", "sparse"):
            bits = c["bits"] if c["op"] == "decode" else {"int8": 8, "int4": 4}.get(c["kv"], 0)
            if bits:
                s["kc"] = _pool(_keys(gen, shape, dt), bits, False)
                s["vc"] = _pool(_randn(gen, shape, dt), bits, True)
            else:
                s["kc"], s["vc"] = _keys(gen, shape, dt), _randn(gen, shape, dt)
            s["bits"] = bits
            s["out"] = torch.empty(c["S"], c["Hq"], D, dtype=dt, device="cuda")
        if c["op"] == "sparse":
            n, MB = c["n"], s["tables"].shape[1]
            nb = torch.from_numpy(_blocks(lens.astype(np.int64))).cuda()[:, None, None]
            at = torch.arange(MB, device="cuda")
            score = torch.rand(c["S"], H, MB, generator=gen, device="cuda")
            score = torch.where((at == 0) | (at >= nb - 2), 2.0, score)
            score = torch.where(at < nb, score, NEG)
            keep = min(n, MB)
            got = torch.topk(score, keep, dim=-1)
            ids = torch.where(got.values > NEG, got.indices, 1 << 30).sort(-1).values
            sel = torch.full((c["S"], H, n), -1, dtype=torch.int32, device="cuda")
            sel[:, :, :keep] = torch.where(ids < (1 << 30), ids, -1).int()
            s["selected"] = sel
    s["ws"] = torch.empty(_workspace(c, s), dtype=torch.uint8, device="cuda")
    return s


def _workspace(c, s):
    """Bytes that hold what a call keeps between its kernels: a maximum, a sum and D values in binary32 for
    each query row and stretch of 256 tokens; two scores for each block and KV head."""
    if c["op"] in ("write_read", "bounds"):
        return 16
    rows, MB = c["S"] * c["Hq"], s["tables"].shape[1]
    if c["op"] == "select":
        return c["S"] * c["Hkv"] * (MB + 64) * 16 + 4096
    tokens = MB * B if c["op"] == "decode" else c["n"] * B
    return rows * -(-tokens // 256) * (c["D"] + 2) * 4 + 4096


# ------------------------------------------------------------- plain forms
def _decode_tiles(tiles, D, bits, value):
    """Values of tiles [..., tile bytes] as binary32 [..., 16, D]."""
    rb = D * bits // 8
    at = torch.from_numpy(_places(D, bits, value)).to(tiles.device)
    code = tiles[..., at.reshape(-1)].reshape(*tiles.shape[:-1], 16, rb)
    if bits == 4:
        code = torch.stack([code & 15, code >> 4], -1).reshape(*tiles.shape[:-1], 16, D)
    sz = tiles[..., 16 * rb:].contiguous().view(torch.float32).reshape(*tiles.shape[:-1], 16, 2)
    return sz[..., 1:2] + sz[..., 0:1] * code.float()


def _plain_write_read(s):
    D, bits, H = s["D"], s["bits"], s["Hkv"]
    live = s["slots"] >= 0
    blk, off = torch.div(s["slots"][live], B, rounding_mode="floor"), s["slots"][live] % B
    rb = D * bits // 8
    for x, pool, out, value in ((s["k"], s["kc"], s["k_out"], False), (s["v"], s["vc"], s["v_out"], True)):
        code, scale, zero = _encode(x[live], bits)
        code = code.to(torch.uint8)
        if bits == 4:
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        at = torch.from_numpy(_places(D, bits, value)).cuda()[off]
        head = torch.arange(H, device="cuda")
        pool[blk[:, None, None], head[None, :, None], at[:, None, :]] = code
        par = 16 * rb + off[:, None] * 8 + torch.arange(8, device="cuda")
        sz = torch.cat([scale, zero], -1).contiguous().view(torch.uint8)
        pool[blk[:, None, None], head[None, :, None], par[:, None, :]] = sz
        tok = _decode_tiles(pool[blk], D, bits, value)
        out[live] = tok[torch.arange(len(off), device="cuda"), :, off].to(out.dtype)
    return s["k_out"], s["v_out"]


def _softmax_rows(score):
    """exp(score - max) / sum over the last axis, zero for a row with nothing in it."""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > NEG, top, torch.zeros_like(top)))
    return p / torch.clamp(p.sum(-1, keepdim=True), min=1e-30)


def _plain_attention(s, blocks, pos_ok):
    """blocks: int64 [S][Hkv][n] physical blocks; pos_ok: bool [S][Hkv][n * 16] tokens attended to."""
    S, H, D = s["S"], s["Hkv"], s["D"]
    G = s["Hq"] // H
    n = blocks.shape[-1]
    head = torch.arange(H, device="cuda")[None, :, None]

    def rows(pool, value):
        got = pool[blocks, head]
        got = _decode_tiles(got, D, s["bits"], value) if s["bits"] else got.float()
        return got.reshape(S, H, n * B, D)

    score = torch.matmul(s["q"].float().reshape(S, H, G, D), rows(s["kc"], False).transpose(-1, -2)) * D ** -0.5
    score = torch.where(pos_ok[:, :, None, :], score, NEG)
    p = _softmax_rows(score)
    v = torch.where(pos_ok[..., None], rows(s["vc"], True), 0.0)
    return torch.matmul(p, v).reshape(S, s["Hq"], D).to(s["q"].dtype)


def _plain_decode(s):
    MB, H = s["tables"].shape[1], s["Hkv"]
    blocks = torch.clamp(s["tables"], min=0).long()[:, None, :].expand(-1, H, -1)
    ok = torch.arange(MB * B, device="cuda") < s["lens"][:, None, None]
    return _plain_attention(s, blocks, ok.expand(-1, H, -1))


def _plain_sparse(s):
    sel = s["selected"].long()
    table = torch.clamp(s["tables"], min=0).long()[:, None, :].expand(-1, s["Hkv"], -1)
    blocks = torch.gather(table, 2, torch.clamp(sel, min=0))
    pos = sel[..., None] * B + torch.arange(B, device="cuda")
    ok = (sel[..., None] >= 0) & (pos < s["lens"][:, None, None, None])
    return _plain_attention(s, blocks, ok.reshape(*sel.shape[:2], -1))


def _plain_bounds(s):
    MB = s["tables"].shape[1]
    at = torch.arange(MB, device="cuda")
    first = torch.div(s["lens"] - s["new"], B, rounding_mode="floor")
    hit = (at >= first[:, None]) & (at * B < s["lens"][:, None]) & (s["new"] > 0)[:, None]
    blk = s["tables"][hit].long()
    left = (s["lens"][:, None] - at * B)[hit]
    k = s["kc"][blk].float()
    ok = (torch.arange(B, device="cuda") < left[:, None])[:, None, :, None]
    inf = torch.full_like(k, float("inf"))
    both = torch.stack([torch.where(ok, k, inf).amin(2), torch.where(ok, k, -inf).amax(2)], 2)
    s["bounds"][blk] = both.to(s["bounds"].dtype)
    return s["bounds"]


def _plain_select(s):
    # in 64 bits: which of two blocks comes first hangs on the last digits of their scores
    S, H, D, n = s["S"], s["Hkv"], s["D"], s["n"]
    G, MB = s["Hq"] // H, s["tables"].shape[1]
    nb = torch.div(s["lens"] + B - 1, B, rounding_mode="floor")[:, None, None]
    bd = s["bounds"][torch.clamp(s["tables"], min=0).long()].double()  # [S][MB][H][2][D]
    q = s["q"].double().reshape(S, H, G, D)
    lo, hi = bd[:, :, :, 0].permute(0, 2, 3, 1), bd[:, :, :, 1].permute(0, 2, 3, 1)
    score = torch.matmul(torch.clamp(q, max=0), lo) + torch.matmul(torch.clamp(q, min=0), hi)
    score = score.amax(2)
    at = torch.arange(MB, device="cuda")
    score = torch.where((at < s["sink"]) | (at >= nb - s["recent"]), float("inf"), score)
    score = torch.where(at < nb, score, NEG)
    ids = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    ids = torch.sort(torch.where(ids < nb, ids, 1 << 30), dim=-1).values
    s["selected"].fill_(-1)
    s["selected"][..., : ids.shape[-1]] = torch.where(ids < (1 << 30), ids, -1).int()
    return s["selected"]


def _own(s):
    from paged_kv_cache_10_gb300 import pagedkv as pk
    op = s["op"]
    kv = {8: "int8", 4: "int4"}.get(s.get("bits"), s["dtype"])
    desc = pk.CacheDesc(num_blocks=s["NB"], num_kv_heads=s["Hkv"], head_size=s["D"], kv_dtype=kv)
    if op == "write_read":
        pk.paged_kv_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], desc)
        pk.paged_kv_read(s["slots"], s["kc"], s["vc"], desc, s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if op == "decode":
        pk.paged_attention_decode(s["q"], s["kc"], s["vc"], desc, s["tables"], s["lens"], s["max_len"],
                                  s["D"] ** -0.5, s["out"], workspace=s["ws"])
        return s["out"]
    if op == "bounds":
        pk.paged_key_bounds(s["kc"], desc, s["tables"], s["lens"], s["new"], s["new_max"], s["bounds"])
        return s["bounds"]
    if op == "select":
        pk.select_blocks(s["q"], s["bounds"], desc, s["tables"], s["lens"], s["max_len"], s["selected"],
                         sink_blocks=s["sink"], recent_blocks=s["recent"], workspace=s["ws"])
        return s["selected"]
    pk.paged_attention_decode_sparse(s["q"], s["kc"], s["vc"], desc, s["tables"], s["lens"], s["selected"],
                                     s["D"] ** -0.5, s["out"], workspace=s["ws"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    return {"write_read": _plain_write_read, "decode": _plain_decode, "bounds": _plain_bounds,
            "select": _plain_select, "sparse": _plain_sparse}[s["op"]](s)


# ------------------------------------------------------ what a pass cannot do without
def work(c):
    H, D = c["Hkv"], c["D"]
    if c["op"] == "write_read":
        live = c["T"] - (len(range(0, c["T"], c["pad"])) if c["pad"] else 0)
        row = D * c["bits"] / 8 + 8
        return {"bytes": c["T"] * 8 + live * H * 2 * (2 * D + row + 2 * D), "flops": live * H * 2 * D * 6}
    lens = _lens(c).astype(np.int64)
    nb = int(_blocks(lens).sum())
    if c["op"] == "bounds":
        new = np.minimum(c["new"], lens)
        first = (lens - new) // B
        rows, blocks = int((lens - first * B).sum()), int((_blocks(lens) - first).sum())
        return {"bytes": rows * H * D * 2 + blocks * (H * 4 * D + 4) + 8 * c["S"], "flops": rows * H * D * 2}
    G = c["Hq"] // H
    io = c["S"] * c["Hq"] * D * 2
    if c["op"] == "select":
        return {"bytes": nb * (H * 4 * D + 4) + io + c["S"] * (4 + H * c["n"] * 4), "flops": nb * H * G * 4 * D}
    if c["op"] == "decode":
        tokens, blocks, listed_ids = int(lens.sum()), nb, 4 * nb
    else:
        kept = np.minimum(_blocks(lens), c["n"])
        tokens = int(np.minimum(lens, kept * B).sum())
        listed_ids = int(kept.sum()) * 8 * H
    row = {"int8": D + 8, "int4": D / 2 + 8}.get(c.get("kv", "int%d" % c.get("bits", 0)), 2 * D)
    return {"bytes": tokens * H * 2 * row + 2 * io + listed_ids + 4 * c["S"], "flops": tokens * H * G * 4 * D}


# ----------------------------------------- the definition in 64 bits, written apart
def _tile_values(tile, D, bits, value):
    """[..., tile bytes] -> float64 [..., 16, D], by the panels' shapes."""
    rb = D * bits // 8
    lead = tile.shape[:-1]
    code = tile[..., : 16 * rb]
    if value:
        code = code.reshape(*lead, rb // 16, 8, 8, 2, 2)  # panel, pair, word, token, byte
        n = code.dim()
        code = code.permute(*range(n - 5), n - 4, n - 2, n - 5, n - 3, n - 1)
    else:
        w = min(rb, 64)
        code = code.reshape(*lead, rb // w, 16, w).transpose(-3, -2)
    code = code.reshape(*lead, 16, rb)
    if bits == 4:
        both = torch.empty(*lead, 16, D, dtype=torch.uint8, device=tile.device)
        both[..., 0::2], both[..., 1::2] = code % 16, code // 16
        code = both
    par = tile[..., 16 * rb:].contiguous().view(torch.float32).reshape(*lead, 16, 2).double()
    return code.double() * par[..., :1] + par[..., 1:]


def _exact_rows(x, bits):
    """The values that rows are held as; the code is decided in binary32, as it is defined."""
    x = x.float().cpu().numpy()
    top = np.float32(2 ** bits - 1)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    scale = ((hi - lo) / top).astype(np.float32)
    scale[scale < np.float32(2.0 ** -126)] = 0
    inv = np.divide(np.float32(1), scale, out=np.zeros_like(scale), where=scale > 0)
    code = np.minimum(np.rint((x - lo) * inv), top)
    return torch.from_numpy(lo.astype(np.float64) + scale.astype(np.float64) * code.astype(np.float64))


def exact(c, seed):
    s = prepare(c, seed)
    D, H = c["D"], c["Hkv"]
    if c["op"] == "write_read":
        dead = (s["slots"] < 0).cpu()
        outs = []
        for x in (s["k"], s["v"]):
            y = _exact_rows(x, c["bits"])
            y[dead] = 0
            outs.append(y)
        return tuple(outs)
    tables, lens = s["tables"].long(), s["lens"].tolist()
    if c["op"] == "bounds":
        out = torch.zeros(s["bounds"].shape, dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["new"].tolist()):
            L = lens[i]
            for j in range((L - n) // B, _blocks(L)) if n > 0 else ():
                rows = s["kc"][tables[i, j], :, : min(B, L - j * B)].double()
                out[tables[i, j], :, 0], out[tables[i, j], :, 1] = rows.min(1).values, rows.max(1).values
        return out
    G = c["Hq"] // H
    if c["op"] == "select":
        out = torch.full((c["S"], H, c["n"]), -1, dtype=torch.int32)
        for i, L in enumerate(lens):
            nb = _blocks(L)
            if nb == 0:
                continue
            bd = s["bounds"][tables[i, :nb]].double()
            for h in range(H):
                sc = torch.full((nb,), NEG, dtype=torch.float64, device="cuda")
                for g in range(G):
                    q = s["q"][i, h * G + g].double()
                    sc = torch.maximum(sc, torch.maximum(q * bd[:, h, 0], q * bd[:, h, 1]).sum(-1))
                sc[: c["sink"]] = float("inf")
                sc[max(0, nb - c["recent"]):] = float("inf")
                order = np.lexsort((np.arange(nb), -sc.cpu().numpy()))[: c["n"]]
                out[i, h, : len(order)] = torch.from_numpy(np.sort(order).astype(np.int32))
        return out
    out = torch.zeros(c["S"], c["Hq"], D, dtype=torch.float64, device="cuda")
    for i, L in enumerate(lens):
        if L == 0:
            continue
        for h in range(H):
            if c["op"] == "decode":
                logical = torch.arange(_blocks(L), device="cuda")
            else:
                logical = s["selected"][i, h].long()
                logical = logical[logical >= 0]
            pos = (logical[:, None] * B + torch.arange(B, device="cuda")).reshape(-1)
            kt, vt = s["kc"][tables[i, logical], h], s["vc"][tables[i, logical], h]
            if s["bits"]:
                kt, vt = _tile_values(kt, D, s["bits"], False), _tile_values(vt, D, s["bits"], True)
            k, v = kt.double().reshape(-1, D)[pos < L], vt.double().reshape(-1, D)[pos < L]
            q = s["q"][i, h * G:(h + 1) * G].double()
            out[i, h * G:(h + 1) * G] = torch.softmax(q @ k.T / math.sqrt(D), -1) @ v
    return out
