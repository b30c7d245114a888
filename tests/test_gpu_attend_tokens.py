"""Attention of several tokens per sequence over the block cache, against its
definition in 64 bits on the same codes.

Tolerance, for a result out = sum p v with M = sum p |v| (the magnitudes it is made of):
  its own rounding: half a step, bf16 2^-8, fp32 2^-24 of the value;
  p times its V scale as an fp16 operand: half a step is 2^-11 of itself (11 bits: steps of 2^-10 of
    the power of two below a value); beside fp32 two terms, the second half a step of what the first
    leaves: 2^-11 of 2^-11 = 2^-22; and 2^-36 of the largest p times the largest V scale at
    least (fp16's subnormals: half a step is 2^-25, and the largest product is 2^11 or more);
  the logit: exact products of fp16 operands (fp32 queries, two terms: to 2^-22), summed in fp32 with
    errors of at most 2^-21 of the sum of magnitudes L, three roundings more;
  2^x by the hardware: 2^-22, its argument's rounding 2^-23 of the logit in base 2;
  the sum of p: fp32, in partial sums: (64 + tiles) roundings of 2^-24;
  the accumulation of p v in fp32: 2^-21 of M, as for the logits, and a rounding for each tile.
A relative error e of p moves out by at most 2 e M (p and the sum)."""
import math

import numpy as np
import pytest
import torch

from helpers import np64
from sparse_rank_kv_gb300 import binding, build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(b, h, d, block, lens, seed, spare=1, wide=0, top=0x77):
    """A cache of random codes (up to e4m3 code `top`) in a pool of an order of its own; lens: tokens per
    sequence, or per pair.  All bytes and scales that no token lies in are NaN.  wide: scales from 2^-wide to 2^wide."""
    g = gen(seed)
    n = torch.tensor(lens)
    n = (n[:, None].expand(b, h) if n.dim() == 1 else n).contiguous()
    mb = max(1, -(-int(n.max()) // block) + spare)
    pool = b * h * mb + 3
    rnd = lambda *s: (torch.randint(0, top + 1, s, generator=g, device="cuda", dtype=torch.uint8) |  # noqa: E731
                      (torch.randint(0, 2, s, generator=g, device="cuda", dtype=torch.uint8) << 7))
    k, v = rnd(pool, block, d), rnd(pool, block, d)
    table = torch.randperm(pool, generator=g, device="cuda")[:b * h * mb].view(b, h, mb)
    scale = lambda: torch.exp2(torch.randint(-wide, wide + 1, (pool,), generator=g, device="cuda").float() - 7)  # noqa: E731
    ks, vs = scale(), scale()
    held = torch.zeros(pool, block, dtype=torch.bool, device="cuda")
    at = torch.arange(mb * block, device="cuda").view(mb, block)
    held[table] = at < n.cuda()[..., None, None]
    k[~held], v[~held] = 0x7f, 0x7f
    ks[~held.any(1)], vs[~held.any(1)] = math.nan, math.nan
    kc = k.view(pool, block // 8, 8, d // 16, 16).transpose(2, 3).contiguous()
    vc = v.view(pool, block // 16, 16, d).transpose(2, 3).contiguous()
    return binding.BlockCache(kc, vc, ks, vs, table.to(torch.int32).contiguous(), n.to(torch.int32).cuda())


def values(c, i, g):
    """Keys and values of a pair, n x d, in 64 bits, and the V scale of each token."""
    n = int(c.n_tok[i, g])
    ids = c.table[i, g, :-(-n // c.block)].long()
    f8 = lambda t: t.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()  # noqa: E731
    k = f8(c.k_codes).transpose(2, 3).reshape(-1, c.block, c.d).double() * c.k_scale[ids].double()[:, None, None]
    v = f8(c.v_codes).transpose(2, 3).reshape(-1, c.block, c.d).double() * c.v_scale[ids].double()[:, None, None]
    return k.reshape(-1, c.d)[:n], v.reshape(-1, c.d)[:n], c.v_scale[ids].double().abs().repeat_interleave(c.block)[:n]


def close(got, lse, c, q, lens=None, causal=True, scale=None, before=None):
    """Every row of `got` (and of lse) against the definition; rows past lens must be as they were."""
    b, hq, s, d = q.shape
    G, scale, bf = hq // c.h_kv, d ** -0.5 if scale is None else scale, q.dtype == torch.bfloat16
    worst = 0.0
    for i in range(b):
        m = s if lens is None else min(max(int(lens[i]), 0), s)
        if before is not None:
            assert torch.equal(got[i, :, m:], before[0][i, :, m:]) and torch.equal(lse[i, :, m:], before[1][i, :, m:])
        for g in range(c.h_kv):
            if m == 0:
                continue
            k, v, vs = values(c, i, g)
            n = len(k)
            x = q[i, g * G:(g + 1) * G, :m].double()
            o, z = got[i, g * G:(g + 1) * G, :m].double(), None if lse is None else lse[i, g * G:(g + 1) * G, :m].double()
            if n == 0:
                assert bool((o == 0).all()) and (z is None or bool((z == -math.inf).all()))
                continue
            seen = (n - m + torch.arange(m, device="cuda") + 1).clamp(min=0) if causal else torch.full((m,), n, device="cuda")
            y = scale * (x @ k.T)
            hide = torch.arange(n, device="cuda") >= seen[:, None]
            y.masked_fill_(hide, -math.inf)
            top = y.amax(-1, keepdim=True)
            empty = top == -math.inf
            e = torch.exp(y - torch.where(empty, 0.0, top))
            total = e.sum(-1, keepdim=True)
            p = e / torch.where(empty, 1.0, total)
            ref, mag = p @ v, p @ v.abs()
            L = abs(scale) * (x.abs() @ k.abs().T).masked_fill(hide, 0).amax(-1, keepdim=True)
            tiles = -(-n // 128)
            dp = (2.0 ** -21 + 3 * U + 2 * U * 1.45) * L + 2.0 ** -22 + 2 * U * top.abs().masked_fill(empty, 0) * 1.45 + (64 + tiles) * U
            dp = dp + (0 if bf else 2.0 ** -22 * L)
            floor = n * 2.0 ** -36 * 448 * (p.amax(-1, keepdim=True)) * vs.max()
            tol = (2.0 ** -8 if bf else U) * ref.abs() + (2 * dp + (2.0 ** -11 if bf else 2.0 ** -22) + 2.0 ** -21 + tiles * U) * mag + floor
            err = (o - ref).abs()
            assert bool((err <= tol + 1e-38).all()), (i, g, float((err / (tol + 1e-38)).max()))
            worst = max(worst, float((err / (tol + 1e-38)).max()))
            if z is not None:
                want = torch.where(empty, -math.inf, top + torch.log(total))[..., 0]
                fin = ~empty[..., 0]
                assert bool((z[~fin] == -math.inf).all())
                zt = (dp[..., 0] + 3 * U * (want.abs() + 1))[fin]
                assert bool(((z - want).abs()[fin] <= zt).all()), float(((z - want).abs()[fin] / zt).max())
    return worst


def run(c, q, lens=None, causal=True, scale=None):
    out = torch.randn(q.shape, generator=gen(5), device="cuda").to(q.dtype)
    lse = torch.randn(q.shape[:3], generator=gen(6), device="cuda")
    before = out.clone(), lse.clone()
    got = c.attend_tokens(q, lens=None if lens is None else ints(lens), causal=causal, scale=scale, out=out, lse=lse)
    assert got is out
    w = close(out, lse, c, q, lens, causal, scale, before)
    c.check()
    return w


def queries(b, hq, s, d, dtype, seed):
    return torch.randn(b, s, hq, d, generator=gen(seed), device="cuda").to(DT[dtype]).transpose(1, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,G,d,block,s,lens,held", [
    (1, 1, 64, 16, 1, [1], [0]), (1, 1, 128, 128, 1, [1, 1], [127, 128]), (2, 4, 128, 64, 5, [5, 1, 0], [700, 0, 90]),
    (2, 3, 64, 32, 17, [17, 16], [111, 129]), (1, 8, 128, 16, 33, [33, 7, 0, 32], [0, 5000, 40, 95]),
    (3, 1, 128, 64, 130, [130, 129, 2], [0, 127, 1000]), (2, 16, 64, 64, 9, [9], [300]), (1, 128, 128, 64, 3, [3, 2], [77, 600]),
    (2, 5, 128, 32, 300, [300, 11], [17, 2000]), (8, 4, 128, 64, 64, [64], [0]), (1, 2, 64, 16, 1000, [1000], [24])])
def test_causal(dtype, h, G, d, block, s, lens, held):
    b = len(lens)
    c = cache(b, h, d, block, [x + y for x, y in zip(lens, held)], s + d)
    run(c, queries(b, h * G, s, d, dtype, 1), lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,G,d,block,s,lens,n", [
    (1, 1, 64, 16, 1, [1], [1]), (2, 2, 64, 16, 33, [33, 20, 5], [100, 1, 0]), (4, 4, 128, 64, 3, [3, 3], [4097, 128]),
    (2, 7, 128, 32, 100, [100, 0], [640, 900]), (1, 4, 64, 128, 500, [500], [257])])
def test_every_token_seen(dtype, h, G, d, block, s, lens, n):
    c = cache(len(n), h, d, block, n, s + 3)
    run(c, queries(len(n), h * G, s, d, dtype, 2), lens, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_heads_of_different_lengths_and_more_queries_than_tokens(dtype, causal):
    """Per-head counts (as eviction leaves them), some below the queries' number: rows that see nothing."""
    c = cache(2, 3, 128, 32, [[0, 5, 300], [40, 129, 1]], 7, spare=3)
    run(c, queries(2, 6, 40, 128, dtype, 3), [40, 30], causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s", [3, 150])
def test_wide_scales_scale_argument_and_strides(dtype, s):
    c = cache(2, 2, 128, 16, [900, 400], 8, wide=20, top=0x40)
    wide = torch.randn(2, s, 3, 4, 136, generator=gen(9), device="cuda").to(DT[dtype])
    q = wide[:, :, 1, :, 3:131].transpose(1, 2)                       # neither pointer nor strides of 16 bytes
    run(c, q, [s, s - 1], scale=0.002)
    run(c, q, [s, s - 1], scale=-0.002)
    run(c, q.contiguous(), None, scale=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,G", [(2, 1), (40, 4)])
def test_a_callers_own_scales(dtype, s, G):
    """Scales that are no powers of two, negative or zero."""
    c = cache(1, 2, 64, 16, [500], 10)
    r = torch.rand(c.k_scale.shape, generator=gen(11), device="cuda") / 64 + 0.001
    c.k_scale.copy_(r)
    c.v_scale.copy_(torch.where(r > 0.01, -r, r))
    c.v_scale[c.table[0, 0, 3].long()] = 0.0
    run(c, queries(1, 2 * G, s, 64, dtype, 12))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s", [4, 200])
def test_token_with_all_the_weight_and_no_value(dtype, s):
    """A first token that takes nearly all the weight in a block of tiny V scale; the others' values count."""
    c = cache(1, 1, 128, 16, [700], 13)
    first = int(c.table[0, 0, 0])
    c.k_codes.view(torch.uint8)[first] = 0x38                        # keys of ones
    c.k_scale[first], c.v_scale[first] = 0.5, 2.0 ** -100
    q = (torch.rand(1, 2, s, 128, generator=gen(14), device="cuda") * 2).to(DT[dtype])
    run(c, q, scale=0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s", [5, 140])
def test_maxima_that_grow_and_fall(dtype, s):
    """Keys whose logits grow by far from tile to tile, then fall: the running maximum's rescaling."""
    for sign in (1, -1):
        c = cache(1, 1, 64, 16, [1500], 15)
        ids = c.table[0, 0].long()
        c.k_codes.view(torch.uint8)[ids] = 0x38
        ramp = torch.arange(len(ids), device="cuda").float()
        c.k_scale[ids] = sign * torch.where(ramp < 50, ramp, 100 - ramp) / 8
        q = torch.full((1, 1, s, 64), 0.25, device="cuda").to(DT[dtype]) * (1 + torch.arange(s, device="cuda")[:, None] % 7).to(DT[dtype])
        run(c, q, scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4, 40])
def test_nan_tokens_reach_the_queries_that_see_them(dtype, G):
    """One NaN key and one NaN value (a single dimension's code) among the last tokens: queries before them are
    untouched; from the value on that dimension is NaN, from the key on the whole row."""
    s, d, n = 9, 128, 200
    c = cache(2, 1, d, 16, [n, n], 16)
    clean = binding.BlockCache(c.k_codes.clone(), c.v_codes.clone(), c.k_scale, c.v_scale, c.table, c.n_tok)
    tv, tk, dim = n - 6, n - 3, 77                                    # query s - 6 is the first to see tv
    c.v_codes[int(c.table[0, 0, tv // 16]), 0, dim, tv % 16] = 0xff
    c.k_codes[int(c.table[0, 0, tk // 16]), (tk % 16) // 8, 3, tk % 8, 5] = 0x7f
    q = queries(2, G, s, d, dtype, 17)
    want, lw = torch.empty(2, G, s, d, dtype=q.dtype, device="cuda"), torch.empty(2, G, s, device="cuda")
    clean.attend_tokens(q, out=want, lse=lw)
    close(want, lw, clean, q)
    lse = torch.empty(2, G, s, device="cuda")
    got = c.attend_tokens(q, lse=lse)
    a, e = s - (n - tv), s - (n - tk)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, :, :a], want[0, :, :a]) and torch.equal(lse[0, :, :e], lw[0, :, :e])
    other = torch.arange(d, device="cuda") != dim
    assert bool(got[0, :, a:e, dim].isnan().all()) and torch.equal(got[0, :, a:e][..., other], want[0, :, a:e][..., other])
    assert bool(got[0, :, e:].isnan().all()) and bool(lse[0, :, e:].isnan().all())
    assert bool(c.attend_tokens(q, causal=False)[0].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_that_are_not_finite_and_queries_with_an_outlier(dtype):
    s = 12
    c = cache(1, 2, 64, 32, [333], 18)
    q = queries(1, 4, s, 64, dtype, 19).contiguous()
    q[0, 0, 3, 5], q[0, 2, 7, 0], q[0, 3, 1] = math.nan, math.inf, 0.0
    q[0, 1, 4, 9] = 2.0 ** 20                                          # the others' products still count
    c.k_codes.view(torch.uint8)[c.table[0, 0].long(), :, 0, :, 9] &= 0x80     # except where the outlier meets zeros
    got = c.attend_tokens(q)
    assert bool(got[0, 0, 3].isnan().all()) and bool(got[0, 2, 7].isnan().all())
    q2 = q.clone()
    q2[0, 0, 3], q2[0, 2, 7] = 0, 0
    out = got.clone()
    out[0, 0, 3], out[0, 2, 7] = c.attend_tokens(q2)[0, 0, 3], c.attend_tokens(q2)[0, 2, 7]
    close(out, None, c, q2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_is_what_attend_gives(dtype):
    c = cache(3, 2, 128, 64, [1, 700, 128], 20)
    q = queries(3, 8, 1, 128, dtype, 21)
    lse, l1 = torch.empty(3, 8, 1, device="cuda"), torch.empty(3, 8, device="cuda")
    got, one = c.attend_tokens(q, lse=lse), c.attend(q[:, :, 0], lse=l1)
    close(one[:, :, None], l1[..., None], c, q)
    close(got, lse, c, q)


def test_offsets_past_32_bits():
    """A pool of more than 4 GB, the blocks in use at its end, and rows that lie as far apart."""
    n_pool, block, d = 560000, 64, 128
    k = torch.zeros(n_pool, block // 8, d // 16, 8, 16, dtype=torch.uint8, device="cuda")
    v = torch.zeros(n_pool, block // 16, d, 16, dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones(n_pool, device="cuda"), torch.ones(n_pool, device="cuda")
    small = cache(2, 1, d, block, [200, 130], 22)
    table = (n_pool - 1 - torch.arange(8, dtype=torch.int32, device="cuda")).view(2, 1, 4).contiguous()
    for i in range(2):
        for e in range(4):
            a, z = int(small.table[i, 0, e]), int(table[i, 0, e])
            k[z], v[z], ks[z], vs[z] = small.k_codes[a], small.v_codes[a], small.k_scale[a], small.v_scale[a]
    c = binding.BlockCache(k, v, ks, vs, table, small.n_tok)
    q = queries(2, 2, 6, d, "bf16", 23)
    far = torch.zeros(2, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")
    out = far[:, :2 * 6 * d].view(2, 2, 6, d)
    out2 = torch.empty_like(out)
    c.attend_tokens(q, out=out)
    small.attend_tokens(q, out=out2)
    assert torch.equal(out, out2)
    close(out2, None, small, q)


def test_bad_block_ids_lengths_and_counts_are_recorded():
    c = cache(2, 1, 64, 16, [100, 100], 24)
    q = queries(2, 2, 8, 64, "bf16", 25)
    want = c.attend_tokens(q)
    assert torch.equal(c.attend_tokens(q, lens=ints([9, -1]))[0], want[0])       # clamped to 8 and 0
    with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
        c.check()
    c = cache(2, 1, 64, 16, [100, 100], 24)
    zero = int(c.table[0, 0, 2])
    c.table[0, 0, 2] = 1 << 20
    got = c.attend_tokens(q)
    assert torch.equal(got[1], want[1])
    c.table[0, 0, 2] = 0                                                # read as block 0
    again = c.attend_tokens(q)
    assert torch.equal(torch.nan_to_num(got[0]), torch.nan_to_num(again[0])) and zero != 0
    with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
        c.check()


@pytest.mark.parametrize("s", [3, 200])
def test_in_place_streams_graphs_and_repeats(s):
    c = cache(3, 2, 128, 64, [900, 250, 4000], 26)
    q = queries(3, 8, s, 128, "bf16", 27)
    want = c.attend_tokens(q)
    close(want, None, c, q)
    for _ in range(3):
        assert torch.equal(c.attend_tokens(q), want)                   # the same bits each time
    own = q.clone()
    c.attend_tokens(own, out=own)                                      # over its own queries
    assert torch.equal(own, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.attend_tokens(q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c.attend_tokens(q))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [c.attend_tokens(q, stream=st) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    c.check()


def test_refusals_and_empty_calls():
    c = cache(2, 2, 64, 16, [40, 40], 28)
    q = queries(2, 4, 3, 64, "f32", 29)
    for call in (lambda: c.attend_tokens(q[0]), lambda: c.attend_tokens(q.half()), lambda: c.attend_tokens(q[:1]),
                 lambda: c.attend_tokens(q, lens=ints([1])), lambda: c.attend_tokens(q, lse=torch.empty(2, 4, 4, device="cuda")),
                 lambda: c.attend_tokens(q, out=q.bfloat16()), lambda: c.attend_tokens(q.transpose(2, 3)),
                 lambda: c.attend_tokens(q.cpu()), lambda: c.attend_tokens(q, lens=torch.tensor([1, 1], device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.attend_tokens(q[:, :3]), lambda: c.attend_tokens(q, scale=math.inf),
                 lambda: c.attend_tokens(q, out=q[:, :, :1].expand(2, 4, 3, 64))):
        with pytest.raises(binding.ShadowKVError):
            call()
    assert c.attend_tokens(q[:, :, :0]).shape == (2, 4, 0, 64)
    none = cache(2, 2, 64, 16, [0, 0], 30)
    assert bool((none.attend_tokens(q) == 0).all())
    none.check()
    got = c.attend_tokens(q, lens=ints([2, 0]))
    assert bool((got[0, :, 2:] == 0).all()) and bool((got[1] == 0).all())
    run(c, q[:, :, :1].expand(2, 4, 3, 64))                             # one row read by all queries


def test_a_speculative_decode_loop():
    """Drafts appended, attended and verified, the rejected ones taken off again: the cache then holds, bit for bit in
    what it gives, the tokens that a cache fed only the accepted ones holds (blocks whose scale the rejected ones
    raised excepted: values here share a scale), over a pool with forks."""
    g = gen(40)
    b, h, G, d, block, v = 3, 2, 4, 64, 16, 97
    c = binding.BlockCache.pooled(b, h, d, 20, 90, block=block)
    ref = binding.BlockCache.empty(b, h, d, 20, block=block)
    emb = (torch.randint(-6, 7, (2, v, h, d), generator=g, device="cuda") / 4).bfloat16()      # K and V of a token
    emb[:, :, :, 0] = 1.75                                             # every block's largest value: one scale for all
    qs = torch.randn(v, h * G, d, generator=g, device="cuda").bfloat16()
    head = 0.3 * torch.randn(h * G * d, v, generator=g, device="cuda")
    rows = lambda kind, t: emb[kind][t.long()].permute(0, 2, 1, 3).contiguous()       # noqa: E731 (b, s) -> b h s d
    prompt = torch.randint(0, v, (b, 21), generator=g, device="cuda", dtype=torch.int32)
    prompt[1:] = prompt[0]
    lens = c.reserve(21, ints([21, 0, 0]))
    c.append(rows(0, prompt), rows(1, prompt), lens)
    c.share(ints([0, 0]), ints([1, 2]))
    ref.append(rows(0, prompt), rows(1, prompt))
    last = ints([5, 6, 7])
    stood = 0
    for step in range(12):
        s = 1 + step % 4
        drafts = torch.randint(0, v, (b, s), generator=g, device="cuda", dtype=torch.int32)
        t = torch.cat([last[:, None], drafts], 1)
        room = c.reserve(s + 1)
        assert room.tolist() == [s + 1] * b
        c.append(rows(0, t), rows(1, t), room)
        x = c.attend_tokens(qs[t.long()].transpose(1, 2), lens=room)
        logits = x.transpose(1, 2).reshape(b, s + 1, -1).float() @ head
        probs = torch.full((b, s, v), 1.0 / v, device="cuda")
        tokens, n = binding.verify_drafts(logits, drafts, probs, torch.rand(b, s, generator=g, device="cuda"),
                                          torch.rand(b, generator=g, device="cuda"))
        c.truncate(s - n)
        ref.append(rows(0, t), rows(1, t), n + 1)
        q = qs[t[:, 0].long()].view(b, h * G, d)
        assert torch.equal(c.n_tok, ref.n_tok)
        assert torch.equal(c.attend(q), ref.attend(q))
        last = tokens.gather(1, n[:, None].long())[:, 0].contiguous()
        stood += int(n.sum())
    assert stood > 5
    named = torch.bincount(c.table[c.table >= 0].long(), minlength=90)
    assert torch.equal(named.int(), c.refs)
    c.check()
    ref.check()


@pytest.mark.parametrize("dtype,d,G,s", [("bf16", 128, 4, 6), ("bf16", 64, 1, 32), ("bf16", 128, 4, 25), ("bf16", 64, 3, 40), ("bf16", 128, 4, 70),
                                         ("bf16", 64, 8, 33), ("f32", 128, 4, 5), ("f32", 64, 2, 60), ("f32", 128, 1, 300)])
def test_rings_turned_many_times(dtype, d, G, s):
    """More than 40 tiles to a CTA, its run over several pairs of different lengths: every ring's turn, parts that several
    CTAs hold, whole row tiles, in each of the kernel's forms."""
    lens = [9000, 1, 130, 8704, 4097, 77, 12000, 300]
    c = cache(8, 8, d, 64, lens, 31)
    q = queries(8, 8 * G, s, d, dtype, 32)
    n = [min(s, x) for x in lens]
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    c.attend_tokens(q, lens=ints(n), out=out, lse=lse)
    close(out, lse, c, q, n)
    c.check()


def test_threads_on_their_own_streams():
    """Four host threads at a time, one cache: each call's kernels and workspace are its own."""
    import threading
    c = cache(4, 2, 128, 64, [700, 3000, 64, 1500], 33)
    qs = [queries(4, 8, s, 128, "bf16", 34 + s) for s in (1, 7, 40, 150)]
    want = [c.attend_tokens(q) for q in qs]
    torch.cuda.synchronize()
    got, faults = [None] * 4, []

    def work(i):
        try:
            st = torch.cuda.Stream()
            for _ in range(20):
                got[i] = c.attend_tokens(qs[i], stream=st)
            st.synchronize()
        except Exception as e:      # noqa: BLE001 (shown below)
            faults.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s", [4, 40, 200])
def test_v_scales_far_apart(dtype, s):
    """Blocks of all-zero values (a scale of 2^-100) and scales over 40 binades beside ordinary ones."""
    c = cache(1, 2, 64, 16, [640], 35, wide=20, top=0x40)
    c.v_codes.view(torch.uint8)[c.table[0, :, 5].long()] = 0
    c.v_scale[c.table[0, :, 5].long()] = 2.0 ** -100
    run(c, queries(1, 4, s, 64, dtype, 36), scale=0.002)


@pytest.mark.parametrize("s,G", [(1, 1), (5, 4), (40, 1), (30, 4), (300, 1), (70, 8)])
@pytest.mark.parametrize("wide", [0, 3])
def test_values_that_cancel(s, G, wide):
    """bf16, one row for all queries, and values chosen for its p so that sum p v is next to nothing beside
    M = sum p |v|: p's own error shows, whatever bf16 keeps of the result.

    The allowance is the one above with p (and its V scale) held to 2^-20 in place of 2^-11, and 2^-19 for its exponent,
    which the scale's 11 binades take to 32 (two roundings of 2^-24 32, log2 of the scale 2^-22): 2^-15.7 M in
    all at the logits here (at most 6).  2^-12, as one fp16 of p is off by, is 10 times that."""
    d, block, n = 128, 16, 200
    c = cache(1, 1, d, block, [n], 50, wide=wide)
    r = gen(51)
    ids = c.table[0, 0, :-(-n // block)].long()
    # keys: one code in all dimensions, so that |q . k| is the sum of its magnitudes, too; logits over +-6
    row = torch.randint(0x28, 0x40, (len(ids), 1, 1, block, 1), generator=r, device="cuda", dtype=torch.uint8)
    row |= torch.randint(0, 2, row.shape, generator=r, device="cuda", dtype=torch.uint8) << 7
    c.k_codes.view(torch.uint8)[ids] = row.view(len(ids), block // 8, 1, 8, 1).expand(-1, -1, d // 16, 8, 16)
    c.k_scale[ids] = 1.0
    q = torch.full((1, 1, 1, d), 0.75, device="cuda").bfloat16()
    scale = 6 / (0.75 * d * 1.875)
    k, v, vs = values(c, 0, 0)
    x = scale * (q[0, 0].double() @ k.T)[0]
    p = torch.softmax(x, 0)
    # values of random magnitude, each of the sign that takes the sum so far towards 0, the largest p first
    code = torch.randint(0x30, 0x40, (n, d), generator=r, device="cuda", dtype=torch.uint8)
    size = code.view(torch.float8_e4m3fn).double() * vs[:, None]
    total, sign = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(n, d, dtype=torch.uint8, device="cuda")
    for t in (p[:, None] * size).amax(1).argsort(descending=True).tolist():
        sign[t] = (total > 0).to(torch.uint8)
        total += torch.where(total > 0, -1.0, 1.0) * p[t] * size[t]
    full = torch.zeros(len(ids) * block, d, dtype=torch.uint8, device="cuda")
    full[:n] = code | sign << 7
    c.v_codes.view(torch.uint8)[ids] = full.view(len(ids), block // 16, 16, d).transpose(2, 3)
    k, v, vs = values(c, 0, 0)
    ref, mag = p @ v, p @ v.abs()
    assert float((ref.abs() / mag).max()) < 2.0 ** -8
    got = c.attend_tokens(q.expand(1, G, s, d), causal=False, scale=scale)
    dp = (2.0 ** -21 + 3 * U + 2 * U * 1.45) * 6 + 2.0 ** -22 + 2 * U * 6 * 1.45 + 66 * U
    floor = n * 2.0 ** -36 * 448 * p.max() * vs.max()
    tol = 2.0 ** -8 * ref.abs() + (2 * (dp + 2.0 ** -20 + 2.0 ** -19) + 2.0 ** -21 + 2 * U) * mag + floor
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,G", [(20, 1), (20, 4), (20, 8), (100, 4), (300, 1)])
@pytest.mark.parametrize("up", [30, 40, 100])
def test_a_hidden_block_of_large_values_leaves_earlier_queries_alone(dtype, s, G, up):
    """The last block's V scale is 2^up times the others'.  The queries that do not see it are those of a cache without it:
    the same definition, with the allowance of the scales that they see (`close` knows no others there)."""
    n, block = 330 + s, 16
    c = cache(2, 2, 128, block, [n, n], 60)
    last = c.table[:, :, (n - 1) // block].long().flatten()
    c.v_scale[last] = 2.0 ** (up - 7)
    m = s - ((n - 1) % block + 1)                                     # queries before the last block's first token
    assert 0 < m < s
    q = queries(2, 2 * G, s, 128, dtype, 61)
    lse = torch.empty(2, 2 * G, s, device="cuda")
    got = c.attend_tokens(q, lse=lse)
    short = binding.BlockCache(c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.table, c.n_tok - (s - m))
    close(got[:, :, :m], lse[:, :, :m], short, q[:, :, :m])
    close(got, lse, c, q)                                              # and those that see it
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,G", [(1, 1), (7, 4), (30, 4), (300, 1)])
@pytest.mark.parametrize("kexp,qexp", [(6, 0), (14, 6), (16, 8), (30, 0), (0, 40), (60, 50), (-90, 100)])
@pytest.mark.parametrize("causal", [True, False])
def test_logits_of_any_size(dtype, s, G, kexp, qexp, causal):
    """Finite logits from 2^8 to 2^112, the largest ones of a row apart by a sixteenth of themselves or the same: the
    softmax is the mean over the same ones (e^-16 beside it at the smallest), which products of e4m3 and powers of two
    give exactly; the tolerance is that of the other tests with a logit's error 0."""
    d, block, n = 64, 16, 700
    c = cache(2, 1, d, block, [n, n - 30], 70)
    g = gen(71)
    row = torch.randint(0x20, 0x40, (len(c.k_scale), 1, 1, block, 1), generator=g, device="cuda", dtype=torch.uint8)
    row |= torch.randint(0, 2, row.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    c.k_codes.view(torch.uint8).copy_(row.view(len(c.k_scale), block // 8, 1, 8, 1).expand(-1, -1, d // 16, 8, 16))
    c.k_scale.fill_(2.0 ** kexp)
    c.v_scale.fill_(2.0 ** -7)                                         # (scales without tokens, too: there they are not read)
    sign = torch.where(torch.arange(s, device="cuda") % 3 == 1, -1.0, 1.0)
    q = (sign[:, None] * 2.0 ** qexp).expand(2, G, s, d).to(DT[dtype]).contiguous()
    lse = torch.empty(2, G, s, device="cuda")
    got = c.attend_tokens(q, causal=causal, scale=0.125, lse=lse)
    for i in range(2):
        k, v, _ = values(c, i, 0)
        y = 0.125 * (q[i].double() @ k.T)
        m = len(k)
        if causal:
            y.masked_fill_(torch.arange(m, device="cuda") >= (m - s + torch.arange(s, device="cuda") + 1)[:, None], -math.inf)
        p = torch.softmax(y, -1)
        ref, mag = p @ v, p @ v.abs()
        e = 2.0 ** -20 + 2.0 ** -19 + 2.0 ** -22 + 70 * U              # p's terms and exponent, 2^x, the sums
        assert bool(((got[i].double() - ref).abs() <= (2.0 ** -8 if dtype == "bf16" else U) * ref.abs() + (2 * e + 2.0 ** -21) * mag).all())
        want = torch.logsumexp(y, -1)
        assert bool(((lse[i].double() - want).abs() <= 6 * U * want.abs() + 2.0 ** -19).all())
    c.check()
