"""What the operators around a step of several tokens cost, over the 8-bit block
cache of the dense decode path: attention of a sequence's new tokens (a piece of
a prompt, drafted tokens, or queries over an encoder's states), the verification
of drafted tokens against the target's logits, and the cache's blocks as a pool
that sequences share (rollback, forks, copy on write, compaction).

`run` computes each operator in elementary torch operations, or, where `own` is
set, through sparse_rank_kv_gb300.binding.  A cache is a pool of blocks of
`block` tokens of one KV head:

  k_codes (n_pool, block/8, d/16, 8, 16)  e4m3; token t, dimension j at [t/8, j/16, t%8, j%16]
  v_codes (n_pool, block/16, d, 16)       e4m3; token t, dimension j at [t/16, j, t%16]
  k_scale, v_scale (n_pool,)              f32; a value is its code times its block's scale
  table, weight (b, h_kv, max_blocks)     i32 (-1: no block), f32; n_tok (b, h_kv) i32
  refs (n_pool,)                          i32: table entries that name the block; 0: free
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
        # four drafted tokens and the last accepted one of a short answer: latency
        dict(name="attend_verify_b1", op="attend", b=1, h_q=32, h_kv=8, d=128, block=64, s=5, held=700, ragged=False, causal=True, dtype="bf16"),
        # five drafts for each of 8 sequences at the headline context: the cache is read once
        dict(name="attend_verify_b8_s128k", op="attend", b=8, h_q=32, h_kv=8, d=128, block=64, s=6, held=131066, ragged=False, causal=True, dtype="bf16"),
        # a whole prompt of 16K tokens, just appended
        dict(name="attend_prompt_16k", op="attend", b=1, h_q=32, h_kv=8, d=128, block=64, s=16384, held=0, ragged=False, causal=True, dtype="bf16"),
        # a padded batch of prompt pieces behind what is held already
        dict(name="attend_pieces_ragged", op="attend", b=4, h_q=32, h_kv=8, d=128, block=64, s=2048, held=20001, ragged=True, causal=True, dtype="bf16"),
        # a decoder's queries over an encoder's states of another length, small f32 heads
        dict(name="attend_cross_f32", op="attend", b=3, h_q=4, h_kv=2, d=64, block=16, s=333, held=1021, ragged=True, causal=False, dtype="f32"),
        # one sequence's four drafts: latency
        dict(name="verify_b1", op="verify", b=1, s=4, vocab=32000, probs=True, temperature=1.0, ragged=False, dtype="bf16"),
        # a server's batch, drafts of different lengths, a large vocabulary
        dict(name="verify_b64", op="verify", b=64, s=7, vocab=128256, probs=True, temperature=0.8, ragged=True, dtype="bf16"),
        # drafts looked up in the prompt (no distribution of their own), f32 logits, rows of odd length
        dict(name="verify_lookup_f32", op="verify", b=5, s=3, vocab=50257, probs=False, temperature=1.0, ragged=True, dtype="f32"),
        # between two steps of a small search: rejected drafts off, one sequence forked, room for five tokens
        dict(name="pages_b4", op="pages", b=4, h_kv=8, d=128, block=64, held=900, fan=2, forks=2, s=5),
        # the same for a server's 48 sequences in groups that share a prompt
        dict(name="pages_b48", op="pages", b=48, h_kv=8, d=128, block=64, held=6000, fan=6, forks=16, s=6),
        # a small cache moved to a pool of its size
        dict(name="compact_b2", op="compact", b=2, h_kv=2, d=64, block=16, held=333, fan=1),
        # a server's pool with as many free blocks as used ones, moved to one of two thirds its size
        dict(name="compact_b32", op="compact", b=32, h_kv=8, d=128, block=64, held=16000, fan=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "pages", "compact"])
    heads = rng.choice([(4, 2, 64), (32, 8, 128), (16, 16, 64), (64, 8, 128), (8, 1, 128), (24, 8, 128), (5, 5, 128)])
    block = rng.choice([16, 32, 64, 128])
    if op == "attend":
        b = _log(rng, 1, 16)
        s = rng.choice([_log(rng, 1, 16), _log(rng, 1, 4096 // b)])
        most = min(131072, 400000 // b, int(2e12 / (4 * heads[0] * heads[2] * b * s)))
        return dict(op=op, b=b, h_q=heads[0], h_kv=heads[1], d=heads[2], block=block, s=s, held=_log(rng, 1, max(1, most)) - 1,
                    ragged=rng.random() < 0.6, causal=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "verify":
        b, vocab = _log(rng, 1, 64), _log(rng, 100, 150000)
        return dict(op=op, b=b, s=min(_log(rng, 1, 12), max(1, 64 * 7 * 128256 // (b * vocab))), vocab=vocab, probs=rng.random() < 0.7,
                    temperature=rng.choice([1.0, 0.7, 1.3, 0.0]), ragged=rng.random() < 0.6, dtype=rng.choice(["bf16", "f32"]))
    b = _log(rng, 1, 48)
    fan = rng.choice([f for f in (1, 2, 3, 6) if b % f == 0])
    case = dict(op=op, b=b, h_kv=heads[1], d=heads[2], block=block, held=_log(rng, 1, max(2, min(20000, 4000000 // (b * heads[1])))), fan=fan)
    return case if op == "compact" else dict(case, forks=rng.randint(0, b // 2), s=rng.choice([1, _log(rng, 2, 300)]))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _spread(seed, n, least, most, ragged=True):
    """n whole numbers: all `most`, or spread over least..most with one of `most`."""
    r = random.Random(seed * 7919 + 13)
    if not ragged:
        return [most] * n
    got = [r.randint(min(least, most), most) for _ in range(n)]
    got[r.randrange(n)] = most
    return got


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _scale_of(amax):
    """The power of two 2^e, e >= -100, smallest with amax <= 448 2^e (448 = 0.875 2^9)."""
    f, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (f > 0.875).to(e.dtype), torch.full_like(e, -100)).clamp(min=-100)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _rows_k(c):     # the pool's order -> (..., block, d)
    *lead, t8, d16, _, _ = c.shape
    return c.transpose(-3, -2).reshape(*lead, t8 * 8, d16 * 16)


def _rows_v(c):
    *lead, t16, d, _ = c.shape
    return c.transpose(-1, -2).reshape(*lead, t16 * 16, d)


def _take(pool, ids):
    return pool.view(torch.uint8)[ids].view(F8)


def _pool(g, n_pool, block, d):
    """Codes and scales of normally distributed blocks, each of its own size, in the pool's order."""
    out = {}
    for kind, shape in (("k", (block // 8, d // 16, 8, 16)), ("v", (block // 16, d, 16))):
        codes, scales = [], []
        step = max(1, (1 << 27) // (block * d))
        for i in range(0, n_pool, step):
            n = min(step, n_pool - i)
            x = torch.randn(n, *shape, generator=g, device="cuda")
            x *= torch.exp2(2 * torch.rand(n, generator=g, device="cuda") - 1).view(n, *[1] * len(shape))
            s = _scale_of(x.abs().amax(tuple(range(1, 1 + len(shape)))))
            codes.append((x / s.view(n, *[1] * len(shape))).to(F8).view(torch.uint8))
            scales.append(s)
        out[kind + "_codes"], out[kind + "_scale"] = torch.cat(codes).view(F8), torch.cat(scales)
    return out


def _handle(s, **more):
    from sparse_rank_kv_gb300 import binding
    return binding.BlockCache(**{k: s[k] for k in ("k_codes", "v_codes", "k_scale", "v_scale", "table", "n_tok", "weight")}, **more)


def _shared_cache(case, g, seed, spare):
    """Sequences in groups of `fan` that share their first half's whole blocks, in a pool with free blocks between the used ones."""
    b, h, d, block, fan = (case[k] for k in ("b", "h_kv", "d", "block", "fan"))
    held = torch.tensor(_spread(seed, b, case["held"] // 2, case["held"]))
    mb = -(-case["held"] // block) + spare
    nb = -(-held // block)
    common = (held.view(-1, fan).amin(1) // (2 * block)).repeat_interleave(fan)       # blocks a group shares
    i = torch.arange(mb)
    first = (torch.arange(b) // fan * fan)[:, None]
    owner = torch.where(i < common[:, None], first, torch.arange(b)[:, None])       # whose block it is
    n_pool = b * h * mb * 3 // 2 + 8
    ids = torch.randperm(n_pool, generator=torch.Generator().manual_seed(seed))[:b * h * mb].view(b, h, mb)
    table = torch.where((i < nb[:, None])[:, None], torch.gather(ids, 0, owner[:, None].expand(b, h, mb)), -1).to(torch.int32).cuda()
    s = dict(case=case, table=table, n_tok=held.to(torch.int32)[:, None].expand(b, h).contiguous().cuda(),
             weight=torch.where(table >= 0, torch.rand(b, h, mb, generator=g, device="cuda"), 0.0),
             refs=torch.bincount(table[table >= 0].long(), minlength=n_pool).to(torch.int32), **_pool(g, n_pool, block, d))
    s.update({k + "_was": s[k].clone() for k in ("table", "n_tok", "weight", "refs")})
    return s


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], TYPES.get(case.get("dtype"))
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    if op == "attend":
        b, h, hq, d, block, s = (case[k] for k in ("b", "h_kv", "h_q", "d", "block", "s"))
        lens, held = _spread(seed, b, 1, s, case["ragged"]), _spread(seed + 1, b, 0, case["held"], case["ragged"])
        n = [x + (y if case["causal"] else 1) for x, y in zip(held, lens)]        # the new tokens are in the cache already
        mb = -(-max(n) // block) + 1
        perm = torch.argsort(rand(b, h, mb), dim=-1) + (torch.arange(b * h, device="cuda") * mb).view(b, h, 1)
        st = dict(case=case, table=perm.to(torch.int32).contiguous(), n_tok=_ints(n)[:, None].expand(b, h).contiguous(),
                  weight=torch.zeros(b, h, mb, device="cuda"), **_pool(g, b * h * mb, block, d))
        # queries as a projection leaves them, b x s x h x d
        st.update(q=randn(b, s, hq, d).to(dt).transpose(1, 2), lens=_ints(lens),
                  out=torch.zeros(b, s, hq, d, dtype=dt, device="cuda").transpose(1, 2), lse=torch.zeros(b, hq, s, device="cuda"))
        if own:
            st["cache"] = _handle(st)
        return st
    if op == "verify":
        b, s, v = (case[k] for k in ("b", "s", "vocab"))
        logits = (2.5 * randn(b, s + 1, v) + 6 * rand(b, s + 1, v).pow(400)).to(dt)    # a few likely tokens over many unlikely ones
        scores = logits[:, :s].float() / (case["temperature"] or 1.0) + 0.5 * randn(b, s, v)      # the draft's, near the target's
        probs = torch.softmax(scores, -1)
        drafts = torch.argmax(scores - torch.log(-torch.log(rand(b, s, v).clamp(1e-30, 1 - 1e-7))), -1).to(torch.int32)    # sampled from probs
        return dict(case=case, logits=logits, drafts=drafts, probs=probs if case["probs"] else None, accept=rand(b, s), sample=rand(b),
                    lens=_ints(_spread(seed, b, 0, s, case["ragged"])))
    if op == "pages":
        b, n = case["b"], case["forks"]
        st = _shared_cache(case, g, seed, -(-case["s"] // case["block"]) + 1)
        order = random.Random(seed).sample(range(b), b)
        dst = order[:n]
        src = [order[n + i % (b - n)] for i in range(n)]
        st.update(src=_ints(src), dst=_ints(dst), lens=_ints(_spread(seed + 2, b, 0, case["s"])),
                  drop=_ints([x if i % 5 else 10 ** 9 for i, x in enumerate(_spread(seed + 3, b, 0, 6), 1)]))     # each fifth sequence is done
        if own:
            st["cache"] = _handle(st, refs=st["refs"])
        return st
    st = _shared_cache(case, g, seed, 1)
    n_pool, block, d = st["table"].numel(), case["block"], case["d"]        # enough whatever is shared
    st["to"] = dict(k_codes=torch.zeros(n_pool, block // 8, d // 16, 8, 16, dtype=torch.uint8, device="cuda").view(F8),
                    v_codes=torch.zeros(n_pool, block // 16, d, 16, dtype=torch.uint8, device="cuda").view(F8),
                    k_scale=torch.zeros(n_pool, device="cuda"), v_scale=torch.zeros(n_pool, device="cuda"), table=torch.zeros_like(st["table"]),
                    n_tok=torch.zeros_like(st["n_tok"]), weight=torch.zeros_like(st["weight"]), refs=torch.zeros(n_pool, dtype=torch.int32, device="cuda"))
    if own:
        st["cache"], st["into"] = _handle(st, refs=st["refs"]), _handle(st["to"], refs=st["to"]["refs"])
    return st


# ------------------------------------------------------------------ the operators
def run(s):
    return {"attend": _attend, "verify": _verify, "pages": _pages, "compact": _compact}[s["case"]["op"]](s)


def _attend(s):
    c = s["case"]
    b, h, hq, d, block, n_q = (c[k] for k in ("b", "h_kv", "h_q", "d", "block", "s"))
    if own:
        s["cache"].attend_tokens(s["q"], lens=s["lens"], causal=c["causal"], out=s["out"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    g, mb = hq // h, s["table"].shape[2]
    table, n_tok = s["table"].long().view(b * h, mb), s["n_tok"].view(b * h)
    q = s["q"].reshape(b * h, g, n_q, d)
    lens = s["lens"][:, None].expand(b, h).reshape(b * h)
    t, j = torch.arange(mb * block, device="cuda"), torch.arange(n_q, device="cuda")
    step = max(1, (1 << 30) // (g * n_q * mb * block))                              # pairs at a time, so that the logits fit
    outs, sums = [], []
    for i in range(0, b * h, step):
        ids, n, m = table[i:i + step], n_tok[i:i + step, None], lens[i:i + step, None]
        keys = (_rows_k(_take(s["k_codes"], ids)).float() * s["k_scale"][ids][..., None, None]).flatten(1, 2)
        values = (_rows_v(_take(s["v_codes"], ids)).float() * s["v_scale"][ids][..., None, None]).flatten(1, 2)
        seen = n - m + j + 1 if c["causal"] else n.expand(-1, n_q)                # tokens a query sees
        x = torch.bmm(q[i:i + step].float().flatten(1, 2), keys.transpose(1, 2)).unflatten(1, (g, n_q)) / math.sqrt(d)
        x = torch.where(t < seen[:, None, :, None], x, -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(x - top)
        z = p.sum(-1, keepdim=True)
        outs.append((torch.bmm(p.flatten(1, 2), values).unflatten(1, (g, n_q)) / torch.where(z == 0, 1.0, z)).to(s["q"].dtype))
        sums.append((top + torch.log(z))[..., 0])
    real = j < s["lens"][:, None, None]
    s["out"].copy_(torch.where(real[..., None], torch.cat(outs).view(b, hq, n_q, d), s["out"]))
    s["lse"].copy_(torch.where(real, torch.cat(sums).view(b, hq, n_q), s["lse"]))
    return dict(out=s["out"], lse=s["lse"])


def _verify(s):
    c = s["case"]
    if own:
        from sparse_rank_kv_gb300 import binding
        tokens, accepted = binding.verify_drafts(s["logits"], s["drafts"], s["probs"], s["accept"], s["sample"], lens=s["lens"],
                                                 temperature=c["temperature"])
        return dict(tokens=tokens, accepted=accepted)
    b, n, v = c["b"], c["s"], c["vocab"]
    x = s["logits"].double()                                       # which token a number falls on is decided next to borders: 64 bits
    if c["temperature"] > 0:
        p = torch.exp((x - x.amax(-1, keepdim=True)) / c["temperature"])
        p = p / p.sum(-1, keepdim=True)
    else:
        p = torch.nn.functional.one_hot(x.argmax(-1), v).double()
    at = s["drafts"].long()[..., None]
    q = s["probs"].double() if s["probs"] is not None else torch.zeros(b, n, v, dtype=torch.float64, device="cuda").scatter_(2, at, 1.0)
    yes = s["accept"].double() * torch.gather(q, 2, at)[..., 0] < torch.gather(p[:, :n], 2, at)[..., 0]
    yes &= torch.arange(n, device="cuda") < s["lens"][:, None]
    a = torch.cumprod(yes.long(), 1).sum(1)
    rows = torch.arange(b, device="cuda")
    rest = torch.where((a < s["lens"])[:, None], (p[rows, a] - q[rows, a.clamp(max=n - 1)]).clamp(min=0), p[rows, a])
    if s["probs"] is None:                                             # a token looked up and rejected is not sampled again
        rest = torch.where((a < s["lens"])[:, None], p[rows, a].scatter(1, at[rows, a.clamp(max=n - 1)], 0.0), p[rows, a])
    cum = torch.cumsum(rest, -1)
    token = (cum <= s["sample"].double()[:, None] * cum[:, -1:]).sum(-1)
    i = torch.arange(n + 1, device="cuda")
    tokens = torch.where(i < a[:, None], torch.nn.functional.pad(s["drafts"].long(), (0, 1)), torch.where(i == a[:, None], token[:, None], -1))
    return dict(tokens=tokens.to(torch.int32), accepted=a.to(torch.int32))


def _pages(s):
    c = s["case"]
    for k in ("table", "n_tok", "weight", "refs"):      # the same step once more
        s[k].copy_(s[k + "_was"])
    if own:
        s["cache"].truncate(s["drop"])
        s["cache"].share(s["src"], s["dst"])
        granted = s["cache"].reserve(c["s"], s["lens"])
    else:
        b, h, block = c["b"], c["h_kv"], c["block"]
        table, n_tok, weight, refs = s["table"], s["n_tok"], s["weight"], s["refs"]
        n_pool, mb = refs.shape[0], table.shape[2]
        i = torch.arange(mb, device="cuda")
        named = lambda ids: torch.zeros(n_pool + 1, dtype=torch.int32, device="cuda").index_add_(  # noqa: E731
            0, torch.where(ids < 0, n_pool, ids).long().flatten(), torch.ones_like(ids).flatten())[:n_pool]
        # rejected drafts and finished sequences
        n_tok.copy_((n_tok - s["drop"][:, None]).clamp(min=0))
        past = i >= ((n_tok + block - 1) // block)[..., None]
        refs -= named(torch.where(past, table, -1))
        table.masked_fill_(past, -1)
        weight.masked_fill_(past, 0.0)
        # forks
        src, dst = s["src"].long(), s["dst"].long()
        refs += named(table[src]) - named(table[dst])
        table[dst], n_tok[dst], weight[dst] = table[src], n_tok[src], weight[src]
        # room for the next tokens
        first = (n_tok // block)[..., None]
        writes = (i >= first) & (i < ((n_tok + s["lens"][:, None] + block - 1) // block)[..., None])
        held = (table >= 0) & writes
        shared = held & (refs[table.clamp(min=0).long()] > 1)
        need = writes & (~held | shared)
        per_seq = need.sum((1, 2))
        free = refs == 0
        fits = (per_seq == 0) | (torch.cumsum(per_seq, 0) <= free.sum())
        granted = torch.where(fits, s["lens"], 0)
        rank = (torch.cumsum(need.flatten(), 0) - 1).view(b, h, mb)
        need &= fits[:, None, None]
        lowest = torch.argsort((~free).to(torch.uint8), stable=True)
        new = torch.where(need, lowest[rank.clamp(0, n_pool - 1)].to(torch.int32), -1)
        copies = need & held & (i == first) & (n_tok % block > 0)[..., None]
        nowhere = n_pool
        to, of = torch.where(copies, new, nowhere).flatten().long(), torch.where(copies, table, 0).flatten().long()
        last = int(min(b * h, n_pool))                     # one partly filled block a pair
        pick = torch.argsort((to == nowhere).to(torch.uint8), stable=True)[:last]
        to, of = to[pick], of[pick]
        keep = to == nowhere
        to, of = torch.where(keep, 0, to), torch.where(keep, 0, of)
        to, of = torch.where(keep, to[:1], to), torch.where(keep, of[:1], of)      # the rest repeat the first (or block 0 itself)
        for k in ("k_codes", "v_codes", "k_scale", "v_scale"):
            pool = s[k].view(torch.uint8) if s[k].dtype == F8 else s[k]
            pool[to] = pool[of]
        refs += named(new) - named(torch.where(need, table, -1))
        table.copy_(torch.where(need, new, table))
    return dict({k: s[k] for k in ("table", "n_tok", "weight", "refs", "k_codes", "v_codes", "k_scale", "v_scale")}, granted=granted)


def _compact(s):
    to = s["to"]
    if own:
        s["cache"].compact(s["into"])
        return to
    live = s["refs"] > 0
    n = torch.cumsum(live.to(torch.int32), 0) - 1
    n_to = to["refs"].shape[0]
    order = torch.argsort((~live).to(torch.uint8), stable=True)[:n_to]
    count = live.sum()
    used = torch.arange(n_to, device="cuda") < count
    for k in ("k_codes", "v_codes", "k_scale", "v_scale"):
        a, z = (x.view(torch.uint8) if x.dtype == F8 else x for x in (s[k], to[k]))
        z.copy_(torch.where(used.view(-1, *[1] * (z.dim() - 1)), a[order], z))
    to["refs"].copy_(torch.where(used, s["refs"][order], 0))
    to["table"].copy_(torch.where(s["table"] >= 0, n.to(torch.int32)[s["table"].clamp(min=0).long()], -1))
    to["n_tok"].copy_(s["n_tok"])
    to["weight"].copy_(s["weight"])
    return to


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    e = 4 if c.get("dtype") == "f32" else 2
    if op == "attend":
        mean = 0.5 if c["ragged"] and c["b"] > 1 else 1.0                # a ragged batch has about half
        s, held = max(1, int(c["s"] * mean)), c["held"] * mean
        n = held + (s if c["causal"] else 1)                               # tokens in the cache
        seen = held + (s + 1) / 2 if c["causal"] else n                   # tokens a query sees, in the mean
        tokens = c["b"] * c["h_kv"] * n
        return dict(bytes=int(tokens * (2 * c["d"] + 12 / c["block"]) + c["b"] * s * c["h_q"] * (2 * c["d"] * e + 4)),
                    flops=int(4 * c["d"] * c["h_q"] * c["b"] * s * seen))
    if op == "verify":
        mean = 0.5 if c["ragged"] and c["b"] > 1 else 1.0
        rows = c["b"] * (c["s"] * mean + 1)
        n = rows * c["vocab"]
        return dict(bytes=int(n * e + (c["b"] * c["vocab"] * 4 if c["probs"] else 0) + c["b"] * (c["s"] + 1) * 16), flops=int(4 * n))
    blocks = c["b"] * c["h_kv"] * max(1, int(0.75 * c["held"] / c["block"]))
    page = 2 * c["block"] * c["d"] + 8
    if op == "pages":
        # tables, weights and references read and written once; a partly filled block copied for every sequence of a fork
        return dict(bytes=int(blocks * 24 + min(c["b"], 2 * c["forks"]) * c["h_kv"] * 2 * page), flops=int(10 * blocks))
    live = blocks * (0.5 + 0.5 / c["fan"])
    return dict(bytes=int(live * 2 * page + blocks * 24), flops=int(4 * blocks))


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    if case["op"] in ("pages", "compact"):        # ids, counts and copies: nothing is computed in a floating type
        return None
    if case["op"] == "attend" and work(case)["flops"] > 3e12:
        return None
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return _exact_attend(s) if case["op"] == "attend" else _exact_verify(s)


def _exact_attend(s):
    c = s["case"]
    h, g, d = c["h_kv"], c["h_q"] // c["h_kv"], c["d"]
    out, lse = s["out"].double(), s["lse"].double()
    for i in range(c["b"]):
        m = int(s["lens"][i])
        for j in range(h):
            n = int(s["n_tok"][i, j])
            ids = s["table"][i, j, :-(-n // c["block"])].long()
            k = (_rows_k(_take(s["k_codes"], ids)).double() * s["k_scale"][ids].double()[:, None, None]).reshape(-1, d)[:n]
            v = (_rows_v(_take(s["v_codes"], ids)).double() * s["v_scale"][ids].double()[:, None, None]).reshape(-1, d)[:n]
            step = max(1, (1 << 28) // (g * n))
            for a in range(0, m, step):
                e = min(m, a + step)
                z = s["q"][i, j * g:(j + 1) * g, a:e].double() @ k.T * d ** -0.5
                if c["causal"]:
                    late = torch.arange(n, device="cuda")[None] > (n - m + torch.arange(a, e, device="cuda"))[:, None]
                    z.masked_fill_(late, -math.inf)
                lse[i, j * g:(j + 1) * g, a:e] = torch.logsumexp(z, -1)
                out[i, j * g:(j + 1) * g, a:e] = torch.softmax(z, -1) @ v
    return dict(out=out, lse=lse)


def _exact_verify(s):
    c = s["case"]
    n, t = c["s"], c["temperature"]
    tokens = torch.full((c["b"], n + 1), -1, dtype=torch.int32, device="cuda")
    accepted = torch.zeros(c["b"], dtype=torch.int32, device="cuda")
    for i in range(c["b"]):
        m = int(s["lens"][i])
        for j in range(m + 1):
            x = s["logits"][i, j].double()
            if t > 0:
                p = torch.softmax(x / t, 0)
            else:
                p = torch.zeros_like(x)
                p[x.argmax()] = 1
            if j == m:
                break
            y = int(s["drafts"][i, j])
            q = s["probs"][i, j].double() if s["probs"] is not None else torch.zeros_like(p)
            if s["probs"] is None:
                q[y] = 1
            if float(s["accept"][i, j]) * float(q[y]) < float(p[y]):
                tokens[i, j] = y
                continue
            if s["probs"] is None:
                p[y] = 0
            else:
                p = torch.relu(p - q)
            break
        line = torch.cumsum(p, 0)
        tokens[i, j] = torch.searchsorted(line, s["sample"][i].double() * line[-1], right=True).to(torch.int32)
        accepted[i] = j
    return dict(tokens=tokens, accepted=accepted)
