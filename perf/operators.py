"""What the dense decode path's operators cost: the norm-and-rotation of queries
and keys, and the append to, attention over, and eviction from a key/value cache
held in 8 bits with one scale per block of tokens and head.

`run` computes each operator in elementary torch operations, or, where `own` is
set, through sparse_rank_kv_gb300.binding.  A cache is a pool of blocks of
`block` tokens of one KV head, a table of block ids per (sequence, KV head), the
tokens each holds, and the attention weight each block has gathered:

  k_codes (n_pool, block/8, d/16, 8, 16)  e4m3; token t, dimension j at [t/8, j/16, t%8, j%16]
  v_codes (n_pool, block/16, d, 16)       e4m3; token t, dimension j at [t/16, j, t%16]
  k_scale, v_scale (n_pool,)              f32; a value is its code times its block's scale
  table, weight (b, h_kv, max_blocks)     i32, f32; n_tok (b, h_kv) i32

A scale is the smallest power of two 2^e with max|x| <= 448 2^e over the block.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a Llama-3-8B-style layer, batch 8: latency
        dict(name="norm_rope_decode_b8", op="norm_rope", b=8, s=1, h_q=32, h_kv=8, d=128, rot=128, norm=True,
             dtype="bf16", pos="first", theta=5e5, top=131072),
        # a long prompt, its rows views of the fused projection's output, keys written head by head for prefill
        dict(name="norm_rope_prompt_32k", op="norm_rope", b=1, s=32768, h_q=32, h_kv=8, d=128, rot=128, norm=True,
             dtype="bf16", pos="first", theta=5e5, top=1),
        # packed short prompts in f32, half of each head rotated, an odd number of tokens with positions of their own
        dict(name="norm_rope_packed_f32", op="norm_rope", b=3, s=1021, h_q=4, h_kv=2, d=64, rot=32, norm=True,
             dtype="f32", pos="each", theta=1e4, top=4096),
        # a decode step's new token for 48 sequences, somewhere inside their last blocks
        dict(name="append_decode_b48", op="append", b=48, h_kv=8, d=128, block=64, s=1, held=700, ragged=True, dtype="bf16"),
        # a padded batch of prompts into an empty cache
        dict(name="append_prompt_ragged", op="append", b=4, h_kv=8, d=128, block=64, s=16000, held=0, ragged=True, dtype="bf16"),
        # a second piece of a prompt in f32, 100 tokens held already
        dict(name="append_piece_f32", op="append", b=2, h_kv=2, d=64, block=16, s=777, held=100, ragged=False, dtype="f32"),
        # the first tokens of one answer: latency
        dict(name="attend_short_b1", op="attend", b=1, h_q=32, h_kv=8, d=128, block=64, n=90, ragged=False, weights=False, dtype="bf16"),
        # a mixed batch of middling lengths, weights gathered for eviction
        dict(name="attend_ragged_b16", op="attend", b=16, h_q=32, h_kv=8, d=128, block=64, n=9001, ragged=True, weights=True, dtype="bf16"),
        # the headline context: batch 8 at 128K
        dict(name="attend_b8_s128k", op="attend", b=8, h_q=32, h_kv=8, d=128, block=64, n=131072, ragged=False, weights=True, dtype="bf16"),
        # small f32 heads with small blocks
        dict(name="attend_f32_b2", op="attend", b=2, h_q=4, h_kv=2, d=64, block=16, n=4099, ragged=True, weights=True, dtype="f32"),
        # one short sequence over its budget
        dict(name="evict_b1", op="evict", b=1, h_kv=8, block=64, n=4000, ragged=False, keep=40, sink=1, recent=2),
        # batch 8 at 128K cut to an eighth
        dict(name="evict_b8_s128k", op="evict", b=8, h_kv=8, block=64, n=131072, ragged=True, keep=256, sink=1, recent=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "evict"])
    heads = rng.choice([(4, 2, 64), (32, 8, 128), (16, 16, 64), (64, 8, 128), (8, 1, 128), (16, 8, 128)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm_rope":
        b = rng.randint(1, 8)
        s = rng.choice([1, _log(rng, 2, 16384 // b)])
        d = heads[2]
        return dict(op=op, b=b, s=s, h_q=heads[0], h_kv=heads[1], d=d, rot=rng.choice([d, d, d // 2]),
                    norm=rng.random() < 0.75, dtype=dtype, pos=rng.choice(["first", "each"]),
                    theta=rng.choice([1e4, 5e5]), top=_log(rng, 1, 1 << 20))
    if op == "append":
        b = _log(rng, 1, 16)
        return dict(op=op, b=b, h_kv=heads[1], d=heads[2], block=rng.choice([16, 32, 64, 128]),
                    s=rng.choice([1, _log(rng, 2, 48000 // b)]), held=_log(rng, 1, 2000) - 1,
                    ragged=rng.random() < 0.6, dtype=dtype)
    if op == "attend":
        b = _log(rng, 1, 32)
        return dict(op=op, b=b, h_q=heads[0], h_kv=heads[1], d=heads[2], block=rng.choice([16, 32, 64, 128]),
                    n=_log(rng, 1, 400000 // b), ragged=rng.random() < 0.6, weights=rng.random() < 0.6, dtype=dtype)
    block = rng.choice([16, 32, 64, 128])
    n = _log(rng, 2 * block, 2000 * block)
    blocks = -(-n // block)
    keep = rng.randint(1, blocks)
    sink = rng.randint(0, min(2, keep))
    return dict(op=op, b=_log(rng, 1, max(1, min(48, (1 << 23) // (n * heads[1])))), h_kv=heads[1], block=block, n=n, ragged=rng.random() < 0.6, keep=keep,
                sink=sink, recent=rng.randint(0, min(4, keep - sink)))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(case, seed, most, least=1):
    """One length per sequence: all `most`, or spread below it with one of `most`."""
    r = random.Random(seed * 7919 + 13)
    b = case["b"]
    if not case["ragged"]:
        return [most] * b
    got = [r.randint(min(least, most), most) for _ in range(b)]
    got[r.randrange(b)] = most
    return got


def _scale_of(amax):
    """The power of two 2^e, e >= -100, smallest with amax <= 448 2^e (448 = 0.875 2^9)."""
    f, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (f > 0.875).to(e.dtype), torch.full_like(e, -100)).clamp(min=-100)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _tile_k(x):     # (..., block, d) codes -> the pool's order
    *lead, t, d = x.shape
    n = len(lead)
    return x.reshape(*lead, t // 8, 8, d // 16, 16).transpose(n + 1, n + 2)


def _tile_v(x):
    *lead, t, d = x.shape
    return x.reshape(*lead, t // 16, 16, d).transpose(-1, -2)


def _rows_k(c):     # the pool's order -> (..., block, d)
    *lead, t8, d16, _, _ = c.shape
    return c.transpose(-3, -2).reshape(*lead, t8 * 8, d16 * 16)


def _rows_v(c):
    *lead, t16, d, _ = c.shape
    return c.transpose(-1, -2).reshape(*lead, t16 * 16, d)


def _take(pool, ids):
    return pool.view(torch.uint8)[ids].view(F8)


def _pool(g, n_pool, block, d):
    """Codes and scales of normally distributed blocks, each of its own size."""
    out = []
    for tile in (_tile_k, _tile_v):
        codes, scales = [], []
        step = max(1, (1 << 27) // (block * d))
        for i in range(0, n_pool, step):
            n = min(step, n_pool - i)
            x = torch.randn(n, block, d, generator=g, device="cuda")
            x *= torch.exp2(2 * torch.rand(n, 1, 1, generator=g, device="cuda") - 1)
            s = _scale_of(x.abs().amax((1, 2)))
            codes.append(tile((x / s[:, None, None]).to(F8).view(torch.uint8)).contiguous())
            scales.append(s)
        out += [torch.cat(codes).view(F8), torch.cat(scales)]
    return out


def _cache(case, g, lens, spare, d, filled):
    """A cache that holds lens[i] tokens of sequence i, its blocks in the pool in an order of their own."""
    b, h, block = case["b"], case["h_kv"], case["block"]
    mb = -(-max(lens) // block) + spare
    perm = torch.argsort(torch.rand(b, h, mb, generator=g, device="cuda"), dim=-1)
    base = (torch.arange(b * h, device="cuda") * mb).view(b, h, 1)
    s = dict(table=(perm + base).to(torch.int32).contiguous(),
             n_tok=torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(b, h).contiguous(),
             weight=torch.zeros(b, h, mb, device="cuda"))
    n_pool = b * h * mb
    if filled:
        s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"] = _pool(g, n_pool, block, d)
    else:
        s["k_codes"] = torch.zeros(n_pool, block // 8, d // 16, 8, 16, dtype=torch.uint8, device="cuda").view(F8)
        s["v_codes"] = torch.zeros(n_pool, block // 16, d, 16, dtype=torch.uint8, device="cuda").view(F8)
        s["k_scale"] = torch.zeros(n_pool, device="cuda")
        s["v_scale"] = torch.zeros(n_pool, device="cuda")
    return s


def _handle(s):
    from sparse_rank_kv_gb300 import binding
    return binding.BlockCache(**{k: s[k] for k in ("k_codes", "v_codes", "k_scale", "v_scale", "table", "n_tok", "weight")})


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], TYPES.get(case.get("dtype"))
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if op == "norm_rope":
        b, s, hq, h, d = (case[k] for k in ("b", "s", "h_q", "h_kv", "d"))
        qkv = (randn(b, s, hq + 2 * h, d) * torch.exp2(2 * randn(b, s, 1, 1))).to(dt)   # the projection's output
        r = random.Random(seed)
        starts = [r.randrange(case["top"]) for _ in range(b)]
        pos = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if case["pos"] == "each":
            pos = (pos[:, None] + torch.randint(0, 4096, (b, s), generator=g, device="cuda")).to(torch.int32)
        return dict(case=case, q=qkv[:, :, :hq].transpose(1, 2), k=qkv[:, :, hq:hq + h].transpose(1, 2), pos=pos,
                    q_weight=(1 + 0.2 * randn(d)).to(dt), k_weight=(1 + 0.2 * randn(d)).to(dt),
                    q_out=torch.empty(b, s, hq, d, dtype=dt, device="cuda").transpose(1, 2),
                    k_out=torch.empty(b, h, s, d, dtype=dt, device="cuda"))
    if op == "append":
        b, h, d, block, s = (case[k] for k in ("b", "h_kv", "d", "block", "s"))
        held = _lengths(case, seed, case["held"], 0) if case["held"] else [0] * b
        st = _cache(case, g, held, -(-s // block) + 1, d, filled=case["held"] > 0)
        amp = torch.exp2(2 * torch.rand(b, h, s, 1, generator=g, device="cuda"))
        st.update(case=case, k=(randn(b, h, s, d) * amp).to(dt), v=(randn(b, h, s, d) * amp).to(dt),
                  lens=torch.tensor(_lengths(case, seed + 1, s), dtype=torch.int32, device="cuda"), n_held=st["n_tok"].clone())
        if own:
            st["cache"] = _handle(st)
        return st
    if op == "attend":
        b, h, hq, d = (case[k] for k in ("b", "h_kv", "h_q", "d"))
        st = _cache(case, g, _lengths(case, seed, case["n"]), 1, d, filled=True)
        st.update(case=case, q=randn(b, hq, d).to(dt), lse=torch.empty(b, hq, device="cuda"))
        if own:
            st["cache"] = _handle(st)
        return st
    # evict: weights as attention gathers them, a few blocks with most of it
    b, h = case["b"], case["h_kv"]
    st = _cache(case, g, _lengths(case, seed, case["n"]), 1, 64, filled=False)   # the pool's contents take no part
    st["weight"] = torch.exp(2 * randn(*st["weight"].shape))
    st.update(case=case, kept=torch.empty(b, h, case["keep"], dtype=torch.int32, device="cuda"))
    if own:
        st["cache"] = _handle(st)
        st["after"] = st["cache"].fork()     # takes the tables after the eviction, so the state can be evicted again
    return st


# ------------------------------------------------------------------ the operators
def run(s):
    return {"norm_rope": _norm_rope, "append": _append, "attend": _attend, "evict": _evict}[s["case"]["op"]](s)


def _norm_rope(s):
    c = s["case"]
    if own:
        from sparse_rank_kv_gb300 import binding
        binding.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], eps=1e-6, norm=c["norm"], theta=c["theta"],
                             rot=c["rot"], pos=s["pos"], q_out=s["q_out"], k_out=s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"])
    pos, n = s["pos"], c["s"]
    if pos.dim() == 1:
        pos = pos[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    half = c["rot"] // 2
    freq = c["theta"] ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = pos[:, None, :, None].double() * freq            # far positions: 64 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for key, weight in (("q", s["q_weight"]), ("k", s["k_weight"])):
        x = s[key].float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        x1, x2 = x[..., :half], x[..., half:2 * half]
        x = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., 2 * half:]], -1)
        s[key + "_out"].copy_(x)
        out[key] = s[key + "_out"]
    return out


def _append(s):
    c = s["case"]
    s["n_tok"].copy_(s["n_held"])     # the same tokens once more, so that every pass appends
    if own:
        s["cache"].append(s["k"], s["v"], s["lens"])
    else:
        b, h, block, n, d = c["b"], c["h_kv"], c["block"], c["s"], c["d"]
        first = s["n_held"] // block
        off = s["n_held"] % block
        nb = -(-n // block) + 1                                                  # blocks a sequence may touch
        idx = (first[..., None] + torch.arange(nb, device="cuda")).clamp(max=s["table"].shape[2] - 1)
        ids = torch.gather(s["table"], 2, idx.long()).long()                     # b, h, nb
        t = torch.arange(nb * block, device="cuda") - off[..., None]             # new token at each place
        new = (t >= 0) & (t < s["lens"][:, None, None])
        old = t < 0
        at = t.clamp(0, n - 1)[..., None].expand(b, h, nb * block, d)
        for kind, rows, tile in (("k", _rows_k, _tile_k), ("v", _rows_v, _tile_v)):
            pool, scales = s[kind + "_codes"], s[kind + "_scale"]
            x = torch.where(new[..., None], torch.gather(s[kind].float(), 2, at), 0.0).view(b, h, nb, block, d)
            have = rows(_take(pool, ids)).float()
            was = scales[ids]
            fresh = _scale_of(x.abs().amax((-1, -2)))
            o = old.view(b, h, nb, block)
            touched = new.view(b, h, nb, block).any(-1)
            scale = torch.where(touched, torch.where(o.any(-1), torch.maximum(was, fresh), fresh), was)
            q = (x / scale[..., None, None]).to(F8)
            held = (have * (was / scale)[..., None, None]).to(F8)
            q = torch.where(new.view(b, h, nb, block, 1), q.view(torch.uint8),
                            torch.where(o[..., None] & touched[..., None, None], held.view(torch.uint8), have.to(F8).view(torch.uint8)))
            live = torch.arange(nb, device="cuda") + first[..., None] < s["table"].shape[2]
            ids_ = torch.where(live, ids, ids[..., :1])                          # places past the table: the first block's again
            q = torch.where(live[..., None, None], q, q[:, :, :1])
            scale = torch.where(live, scale, scale[..., :1])
            pool.view(torch.uint8)[ids_] = tile(q)
            scales[ids_] = scale
        s["n_tok"] += s["lens"][:, None]
    return dict(k_codes=s["k_codes"], v_codes=s["v_codes"], k_scale=s["k_scale"], v_scale=s["v_scale"], n_tok=s["n_tok"])


def _attend(s):
    c = s["case"]
    b, h, hq, d, block = (c[k] for k in ("b", "h_kv", "h_q", "d", "block"))
    decay = 0.0 if c["weights"] else None       # 0: each pass's own weights, so that passes give the same
    if own:
        out = s["cache"].attend(s["q"], decay=decay, lse=s["lse"])
        return dict(out=out, lse=s["lse"], **({"weight": s["weight"]} if c["weights"] else {}))
    g, mb = hq // h, s["table"].shape[2]
    ids = s["table"].long().view(b * h, mb)
    keys = (_rows_k(_take(s["k_codes"], ids)).float() * s["k_scale"][ids][..., None, None]).reshape(b * h, mb * block, d)
    q = s["q"].float().view(b * h, g, d)
    logits = torch.bmm(q, keys.transpose(1, 2)) / math.sqrt(d)
    held = torch.arange(mb * block, device="cuda") < s["n_tok"].view(b * h, 1, 1)
    logits = torch.where(held, logits, -math.inf)
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z == 0, 1.0, z)
    values = (_rows_v(_take(s["v_codes"], ids)).float() * s["v_scale"][ids][..., None, None]).reshape(b * h, mb * block, d)
    out = torch.bmm(p, values).view(b, hq, d).to(s["q"].dtype)
    s["lse"].copy_((m + torch.log(z)).view(b, hq))
    if not c["weights"]:
        return dict(out=out, lse=s["lse"])
    w = p.view(b, h, g, mb, block).sum((2, 4))
    used = torch.arange(mb, device="cuda") * block < s["n_tok"][..., None]
    s["weight"].copy_(torch.where(used, w, s["weight"]))
    return dict(out=out, lse=s["lse"], weight=s["weight"])


def _evict(s):
    c = s["case"]
    keep, block = c["keep"], c["block"]
    if own:
        a = s["after"]
        s["cache"].evict(keep, sink=c["sink"], recent=c["recent"], into=a, kept=s["kept"])
        return dict(table=a.table, n_tok=a.n_tok, weight=a.weight, kept=s["kept"])
    mb = s["table"].shape[2]
    i = torch.arange(mb, device="cuda")
    n_tok = s["n_tok"].long()[..., None]
    n = (n_tok + block - 1) // block
    w = torch.where((i < c["sink"]) | (i >= n - c["recent"]), math.inf, s["weight"])
    w = torch.where(i < n, w, -math.inf)
    rank = torch.argsort(torch.argsort(w, dim=-1, descending=True, stable=True), dim=-1, stable=True)
    stays = (rank < keep) & (i < n)
    order = torch.argsort(torch.where(stays, 0, torch.where(i < n, 1, 2)), dim=-1, stable=True)
    nk = n.clamp(max=keep)
    last = torch.gather(stays, 2, (n - 1).clamp(min=0))
    n_new = torch.where(last, (nk - 1) * block + n_tok - (n - 1) * block, nk * block)
    weight = torch.where(i < nk, torch.gather(s["weight"], 2, order), 0.0)
    kept = torch.where(i[:keep] < nk, order[..., :keep], -1).to(torch.int32)
    if mb < keep:
        kept = torch.cat([kept, kept.new_full((*kept.shape[:2], keep - mb), -1)], -1)
    return dict(table=torch.gather(s["table"], 2, order), n_tok=n_new[..., 0].to(torch.int32), weight=weight, kept=kept)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    e = 4 if c.get("dtype") == "f32" else 2
    if op == "norm_rope":
        n = c["b"] * c["s"] * (c["h_q"] + c["h_kv"]) * c["d"]
        return dict(bytes=2 * n * e, flops=(10 if c["norm"] else 6) * n)
    mean = 0.5 if c["ragged"] and c["b"] > 1 else 1.0         # a ragged batch holds about half
    if op == "append":
        n = 2 * c["b"] * c["h_kv"] * c["d"] * max(1, int(c["s"] * mean))
        return dict(bytes=n * (e + 1), flops=4 * n)
    if op == "attend":
        t = c["b"] * max(1, int(c["n"] * mean))
        rest = 2 * c["b"] * c["h_q"] * c["d"] * e + (4 * t * c["h_kv"] // c["block"] if c["weights"] else 0)
        return dict(bytes=2 * t * c["h_kv"] * c["d"] + 12 * t * c["h_kv"] // c["block"] + rest, flops=4 * t * c["h_q"] * c["d"])
    blocks = c["b"] * c["h_kv"] * (-(-c["n"] // c["block"]) + 1)
    return dict(bytes=blocks * 16 + c["b"] * c["h_kv"] * (8 + 4 * c["keep"]), flops=10 * blocks)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return {"norm_rope": _exact_norm_rope, "append": _exact_append, "attend": _exact_attend,
            "evict": lambda s: None}[case["op"]](s)


def _exact_norm_rope(s):
    c = s["case"]
    rot, d = c["rot"], c["d"]
    where = s["pos"].double()
    if where.dim() == 1:
        where = where.unsqueeze(1) + torch.arange(c["s"], device="cuda", dtype=torch.float64).unsqueeze(0)
    out = {}
    for key in "qk":
        x = s[key].double()
        if c["norm"]:
            x = s[key + "_weight"].double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6)
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
        turn = torch.exp(-math.log(c["theta"]) * 2.0 / rot * torch.arange(rot // 2, device="cuda", dtype=torch.float64))
        z = z * torch.polar(torch.ones_like(turn), where.unsqueeze(-1) * turn).unsqueeze(1)
        out[key] = torch.cat([z.real, z.imag, x[..., rot:]], -1)
    return out


def _exact_append(s):
    c = s["case"]
    block, d = c["block"], c["d"]
    got = {}
    for kind, pool_rows, back in (("k", _rows_k, _tile_k), ("v", _rows_v, _tile_v)):
        codes = pool_rows(s[kind + "_codes"].view(torch.uint8)).view(F8).double()
        scale = s[kind + "_scale"].double()
        for i in range(c["b"]):
            for j in range(c["h_kv"]):
                n0, n1 = int(s["n_held"][i, j]), int(s["n_held"][i, j]) + int(s["lens"][i])
                f, l = n0 // block, -(-n1 // block)
                ids = s["table"][i, j, f:l].long()
                x = torch.zeros((l - f) * block, d, dtype=torch.float64, device="cuda")
                x[n0 - f * block:n1 - f * block] = s[kind][i, j, :n1 - n0].double()
                x = x.view(l - f, block, d)
                top = x.abs().amax((1, 2))
                sc = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-30) / 448)))
                sc = torch.where(top > 448 * sc, 2 * sc, torch.where(top <= 224 * sc, sc / 2, sc)).clamp(min=2.0 ** -100)
                place = torch.arange((l - f) * block, device="cuda").view(l - f, block, 1)
                fresh = (place >= n0 - f * block) & (place < n1 - f * block)
                value = codes[ids] * scale[ids, None, None]
                if n0 % block:
                    sc[0] = torch.maximum(sc[0], scale[ids[0]])
                    mine = place < n0 - f * block
                    codes[ids] = torch.where(fresh, x, torch.where(mine, value, codes[ids] * sc[:, None, None])) / sc[:, None, None]
                else:
                    codes[ids] = torch.where(fresh, x / sc[:, None, None], codes[ids])
                scale[ids] = sc
        got[kind + "_codes"], got[kind + "_scale"] = back(codes), scale
    return got


def _exact_attend(s):
    c = s["case"]
    h, g, d, block = c["h_kv"], c["h_q"] // c["h_kv"], c["d"], c["block"]
    out = torch.zeros(c["b"], c["h_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["b"], c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    for i in range(c["b"]):
        for j in range(h):
            n = int(s["n_tok"][i, j])
            nb = -(-n // block)
            ids = s["table"][i, j, :nb].long()
            k = (_rows_k(_take(s["k_codes"], ids)).double() * s["k_scale"][ids].double()[:, None, None]).reshape(-1, d)[:n]
            v = (_rows_v(_take(s["v_codes"], ids)).double() * s["v_scale"][ids].double()[:, None, None]).reshape(-1, d)[:n]
            q = s["q"][i, j * g:(j + 1) * g].double()
            z = (k @ q.T).T * d ** -0.5
            top = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            out[i, j * g:(j + 1) * g] = p @ v
            lse[i, j * g:(j + 1) * g] = top
            col = torch.zeros(nb * block, dtype=torch.float64, device="cuda")
            col[:n] = p.sum(0)
            weight[i, j, :nb] = col.view(nb, block).sum(1)
    return dict(out=out, lse=lse, **({"weight": weight} if c["weights"] else {}))
