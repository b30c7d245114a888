"""The dense decode path where its arithmetic and its contracts are tightest.

A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by U = 2^-24."""
import threading

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import dense_oracle as D
from sparse_rank_kv_gb300 import binding
from test_gpu_dense import DT, STEP, U, _built, filled, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ bits kept
@pytest.mark.parametrize("spare", [0, 20])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 8), (128, 1), (128, 2), (128, 4), (128, 8)])
def test_attend_weights_keep_16_bits_in_bf16(d, G, spare):
    """Two tokens with values 1 and -1 and logits 0 and x: out = (1 - e^x) / (1 + e^x), small
    where x is, so that what the output loses is what the weights lose: 2^-16 of each, which
    sum to 1 (a weight of 11 bits misses by up to 2^-13).  The exponential's 2^-21 and the
    logit's rounding stand beside it."""
    b, h = 16, 2
    c = binding.BlockCache.empty(b, h, d, 1 + spare, block=64)
    k = torch.zeros(b, h, 2, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 1, 0] = 1
    v = torch.ones_like(k)
    v[:, :, 1] = -1
    c.append(k, v)
    g = gen(G)
    x = torch.exp2(-6 - 3 * torch.rand(b, h * G, generator=g, device="cuda")) * torch.sign(randn(g, b, h * G))
    q = torch.zeros(b, h * G, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = x
    out = np64(c.attend(q, scale=1.0))
    want = -np.tanh(np64(q[:, :, :1]) / 2)
    tol = STEP[torch.bfloat16] * np.abs(want) + 2.0 ** -16 + 2.0 ** -20
    err = np.abs(out - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("dtype,exact,floor", [("bf16", 2.0 ** -21, 2.0 ** -29), ("f32", 0.0, 2.0 ** -37)])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 2), (128, 4), (128, 8)])
def test_attend_queries_with_an_outlier(dtype, exact, floor, d, G):
    """A query entry far below its row's largest, whose keys are zero, makes the logit alone:
    lse of the one token is q_1 k_1.  A bf16 entry is exact down to 2^-21 of the row's largest and
    within 2^-29 of that one below (fp32: 2^-24 of itself, 2^-37 of the largest); the product
    itself takes the roundings of the scaling and of log2 to ln."""
    b, h, dt = 32, 2, DT[dtype]
    c = binding.BlockCache.empty(b, h, d, 1, block=16)
    k = torch.zeros(b, h, 1, d, dtype=dt, device="cuda")
    k[..., 1] = 1
    c.append(k, k)
    g = gen(d + G)
    q = torch.zeros(b, h * G, d, dtype=dt, device="cuda")
    q[..., 0] = 9984                                          # 312 under the row's scale of 32
    q[..., 1] = torch.exp2(-26 * torch.rand(b, h * G, generator=g, device="cuda")) * 5000 * torch.sign(randn(g, b, h * G))
    lse = torch.empty(b, h * G, device="cuda")
    c.attend(q, scale=1.0, lse=lse)
    want = np64(q[..., 1])
    tol = 16 * U * np.abs(want) + np.where(np.abs(want) >= exact * 9984, 0 if exact else U * np.abs(want), floor * 9984)
    if not exact:
        tol += floor * 9984
    err = np.abs(np64(lse) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spare", [0, 60])
def test_attend_token_with_the_weight_and_no_value(dtype, spare):
    """A token of no value takes all the weight; another one of its 128, in a block of its own
    with a V scale up to 2^8 smaller or larger, makes the output with a weight of 2^-8 to 2^-24.
    It is off by at most 2^-16 of itself and 2^-30 of (largest weight) (largest V scale) times its
    code of 448 (fp32: 2^-23 and 2^-38), beside logits and exponentials in fp32."""
    b, h, G, d, dt = 32, 2, 4, 64, DT[dtype]
    c = binding.BlockCache.empty(b, h, d, 8 + spare, block=16)
    g = gen(7)
    x = -8 - 16 * torch.rand(b, h, 1, generator=g, device="cuda")
    k = torch.zeros(b, h, 128, d, device="cuda")
    k[..., 0] = -256                                         # the others: out of the picture
    k[:, :, 0, 0] = 0
    k[:, :, 100, 0] = x[..., 0]
    v = torch.zeros(b, h, 128, d, device="cuda")
    v[:, :, 1] = 1                                           # the first block's V scale
    v[:, :, 100] = 448 / 256 * torch.exp2(torch.randint(-8, 9, (b, h, 1), generator=g, device="cuda").float())
    c.append(k.to(dt), v.to(dt))
    q = torch.zeros(b, h * G, d, dtype=dt, device="cuda")
    q[..., 0] = 1
    scale = 0.6931471805599453
    out = np64(c.attend(q, scale=scale))
    # the definition on what the cache holds
    id_ = c.table[:, :, 6].long()
    kc = c.k_codes.view(torch.float8_e4m3fn).float()[id_][:, :, 0, 0, 4, 0].double() * c.k_scale[id_].double()
    val = 448 * np64(c.v_scale[id_])
    p = np.exp(np64(kc) * scale)
    want = (p * val / (1 + p))[:, :, None]
    big = np.maximum(2.0 ** -8, np64(c.v_scale[id_]))[:, :, None]
    bf = dt == torch.bfloat16
    rel = STEP[dt] + (2.0 ** -16 if bf else 2.0 ** -23) + 2.0 ** -20 + 2 * (d + 8) * U * 24 * scale
    tol = rel * np.abs(want) + (2.0 ** -30 if bf else 2.0 ** -38) * 448 * big
    err = np.abs(out.reshape(b, h, G * d) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance"


# ------------------------------------------------------------ table entries out of the pool
def known_cache(g, b, h, d, block, max_blocks, lens):
    """A cache of finite codes and scales, pool block 0 nobody's, lens[i] tokens held of sequence i."""
    n = b * h * max_blocks + 1
    codes = lambda *s: torch.randint(0, 0x70, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    scale = lambda: torch.exp2(torch.randint(-9, -6, (n,), generator=g, device="cuda").float())  # noqa: E731
    table = (1 + torch.randperm(n - 1, generator=g, device="cuda")).to(torch.int32).view(b, h, max_blocks)
    n_tok = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(b, h).contiguous()
    return binding.BlockCache(codes(n, block // 8, d // 16, 8, 16), codes(n, block // 16, d, 16), scale(), scale(), table,
                              n_tok, torch.full((b, h, max_blocks), 5.0, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("s", [1, 2, 300])
def test_append_through_a_bad_id_writes_nothing(dtype, d, block, s):
    """The blocks whose ids are out of the pool, a held one that would be rescaled and a new one
    among them, are dropped and recorded; every other block gets what it gets without them."""
    b, h, mb, dt = 2, 2, 40, DT[dtype]
    g = gen(s + d)
    held = [block + 5, 2 * block]                             # one pair goes on in a block, one begins one
    bad = known_cache(g, b, h, d, block, mb, held)
    good = binding.BlockCache(*(t.clone() for t in (bad.k_codes, bad.v_codes, bad.k_scale, bad.v_scale, bad.table,
                                                    bad.n_tok, bad.weight)))
    lost = []
    for i, g_, j, x in ((0, 0, 1, -1), (0, 1, 2, bad.k_scale.numel()), (1, 0, 2, 2**31 - 1), (1, 1, 3, -2**31)):
        lost.append(int(bad.table[i, g_, j]))
        bad.table[i, g_, j] = x
    before = [t.clone() for t in (bad.k_codes, bad.v_codes, bad.k_scale, bad.v_scale)]
    k, v = 100 * randn(g, b, h, s, d).to(dt), 100 * randn(g, b, h, s, d).to(dt)
    bad.append(k, v)
    good.append(k, v)
    good.check()
    keep = torch.ones(bad.k_scale.numel(), dtype=torch.bool, device="cuda")
    keep[lost] = False
    for name, was in zip(("k_codes", "v_codes", "k_scale", "v_scale"), before):
        x, y = getattr(bad, name), getattr(good, name)
        assert torch.equal(x[0], was[0]), f"{name}: block 0"
        assert torch.equal(x[keep], y[keep]) and torch.equal(x[lost], was[lost]), name
    assert torch.equal(bad.n_tok, good.n_tok) and torch.equal(bad.weight, good.weight)
    with pytest.raises(binding.ShadowKVError) as e:
        bad.check()
    assert e.value.code == 4


@pytest.mark.parametrize("d,block,lens", [(64, 16, [64]), (128, 64, [1500])])
def test_attend_reads_block_0_in_a_bad_ids_place(d, block, lens):
    """By value: what a bad id gives is what block 0 gives, and neither is what the pair's own block gives."""
    c = known_cache(gen(3), 1, 2, d, block, 40, lens)
    q = randn(gen(4), 1, 8, d)
    t = c.table.clone()
    own = c.attend(q, decay=0.0)
    c.table[0, :, 1:3] = torch.tensor([0, 0], device="cuda")
    want, w = c.attend(q, decay=0.0), c.weight.clone()
    c.check()
    c.table[0, :, 1:3] = torch.tensor([-1, 10**9], device="cuda")
    got = c.attend(q, decay=0.0)
    assert torch.isfinite(want).all() and not torch.equal(want, own)
    assert torch.equal(got, want) and torch.equal(c.weight, w)
    with pytest.raises(binding.ShadowKVError):
        c.check()
    c.table.copy_(t)
    c.status.zero_()
    assert torch.equal(c.attend(q, decay=0.0), own)
    c.check()


# ------------------------------------------------------------ threads
def in_threads(n, work):
    """work(i) in n threads that begin together; the first exception is raised here."""
    go, got = threading.Barrier(n), [None] * n

    def one(i):
        try:
            go.wait()
            got[i] = work(i)
        except Exception as e:  # noqa: BLE001
            got[i] = e

    ts = [threading.Thread(target=one, args=(i,)) for i in range(n)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for x in got:
        if isinstance(x, Exception):
            raise x
    torch.cuda.synchronize()
    return got


def test_threads_attend_on_one_stream():
    """Threads share the current stream and with it the workspace; a call of two
    kernels gets the rows of its own query whatever the other threads enqueue."""
    c, _ = filled(2, 2, 128, 64, [3000, 100], torch.bfloat16, seed=31)
    n, calls = 4, 300
    qs = [randn(gen(i), 2, 8, 128).bfloat16() for i in range(n)]
    want = [c.attend(q) for q in qs]
    torch.cuda.synchronize()
    got = in_threads(n, lambda i: [c.attend(qs[i]) for _ in range(calls)])
    for i in range(n):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_threads_attend_on_many_streams():
    """More streams than workspaces kept: none is taken from a call in flight."""
    c, _ = filled(2, 2, 128, 64, [3000, 100], torch.bfloat16, seed=31)
    n = 3
    qs = [randn(gen(i), 2, 8, 128).bfloat16() for i in range(n)]
    want = [c.attend(q) for q in qs]
    streams = [[torch.cuda.Stream() for _ in range(5)] for _ in range(n)]
    torch.cuda.synchronize()
    got = in_threads(n, lambda i: [c.attend(qs[i], stream=streams[i][t % 5]) for t in range(60)])
    for i in range(n):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_threads_append_on_one_stream():
    """An append of several tokens writes its counts by a second kernel: none may be
    lost to another thread's append in between.  All tokens are alike, so that their order does not show."""
    n, calls, s = 4, 50, 3
    c = binding.BlockCache.empty(2, 2, 64, 40, block=16)
    row = randn(gen(1), 1, 1, 1, 64).bfloat16()
    k = row.expand(2, 2, s, 64)
    in_threads(n, lambda i: [c.append(k, k) for _ in range(calls)])
    c.check()
    assert torch.all(c.n_tok == n * calls * s)
    one = binding.BlockCache.empty(2, 2, 64, 40, block=16)
    one.append(row.expand(2, 2, n * calls * s, 64), row.expand(2, 2, n * calls * s, 64))
    for x in ("k_codes", "v_codes", "k_scale", "v_scale", "n_tok"):
        assert torch.equal(getattr(c, x), getattr(one, x)), x


# ------------------------------------------------------------ streams
def test_outputs_belong_to_the_stream_that_writes_them():
    """With stream=..., what a call allocates comes from that stream's memory: the current
    stream's pending work may still use what was freed there, and may be handed the output's
    memory again before the other stream has written it."""
    s = torch.cuda.Stream()
    x = randn(gen(1), 1, 2, 700, 128).bfloat16()
    c = binding.BlockCache.empty(1, 2, 128, 12)
    s.wait_stream(torch.cuda.current_stream())
    c.append(x, x, stream=s)
    for stream in (s, s.cuda_stream):
        q, k = binding.qk_norm_rope(x, x, stream=stream)
        out = c.attend(x[:, :, 0], stream=stream)
        torch.cuda.synchronize()
        for t in (q, k, out):
            seg = [m for m in torch.cuda.memory_snapshot()
                   if m["address"] <= t.data_ptr() < m["address"] + m["total_size"]]
            assert [m["stream"] for m in seg] == [s.cuda_stream]
        a, b = binding.qk_norm_rope(x, x)
        assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(out, c.attend(x[:, :, 0]))


# ------------------------------------------------------------ the attention's ring and its two forms
def cache_of_codes(g, lens, h, d, block):
    """A cache of random codes under scales of 2^-9 to 2^-7, blocks in any order, lens[i] tokens of each head of sequence i."""
    b, mb = len(lens), -(-max(lens) // block)
    n = sum(-(-x // block) for x in lens) * h + 1
    codes = lambda *s: torch.randint(0, 0x70, s, generator=g, device="cuda", dtype=torch.uint8) | (  # noqa: E731
        torch.randint(0, 2, s, generator=g, device="cuda", dtype=torch.uint8) << 7)
    scale = lambda: torch.exp2(torch.randint(-9, -6, (n,), generator=g, device="cuda").float())  # noqa: E731
    ids, at = (torch.randperm(n - 1, generator=g, device="cuda") + 1).to(torch.int32), 0
    table = torch.zeros(b, h, mb, dtype=torch.int32, device="cuda")
    for i, x in enumerate(lens):
        nb = -(-x // block)
        table[i, :, :nb] = ids[at:at + h * nb].view(h, nb)
        at += h * nb
    n_tok = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(b, h).contiguous()
    return binding.BlockCache(codes(n, block // 8, d // 16, 8, 16), codes(n, block // 16, d, 16), scale(), scale(), table, n_tok,
                              torch.full((b, h, mb), 3.0, device="cuda"))


def attend_pair(c, q, scale, i, j):
    """The definition in 64 bits, on the GPU, for query heads q (G, d) of pair (i, j): out, lse, block weights, sum p |v|,
    the largest logit's sum of magnitudes, and the sum over 128-token tiles of the largest p times the largest 448 V scale."""
    n = int(c.n_tok[i, j])
    nb = -(-n // c.block)
    ids = c.table[i, j, :nb].long()
    f8 = lambda t: t.view(torch.float8_e4m3fn).float().double()  # noqa: E731
    k = (f8(c.k_codes[ids]).permute(0, 1, 3, 2, 4).reshape(nb, c.block, c.d) * c.k_scale[ids].double()[:, None, None]).reshape(-1, c.d)[:n]
    v = (f8(c.v_codes[ids]).permute(0, 1, 3, 2).reshape(nb, c.block, c.d) * c.v_scale[ids].double()[:, None, None]).reshape(-1, c.d)[:n]
    q = q.double()
    z = scale * (q @ k.T)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    pad = lambda x, m: torch.nn.functional.pad(x, (0, -(-x.shape[-1] // m) * m - x.shape[-1]))  # noqa: E731
    w = pad(p, c.block).view(len(q), nb, c.block).sum((0, 2))
    tile = pad(p, 128).view(len(q), -1, 128).amax(-1)
    vs = pad(c.v_scale[ids].double()[None], 128 // c.block).view(-1, 128 // c.block).amax(-1)
    return p @ v, lse, w, p @ v.abs(), abs(scale) * (q.abs() @ k.abs().T).amax(-1), (tile * 448 * vs).sum(-1)


def attend_as_defined(c, q, scale, tiles_per_share, parts):
    """One call with its weights against the definition.  A logit takes d roundings of its sum and 8 of
    its scaling, p as much twice and an exponential's 2^-21; a share's sum takes per tile two
    roundings and, where the maximum moves, an exponential (2^-22), the join one per part.  p itself:
    2^-16 (bf16) or 2^-22 and the floor of its tile."""
    bf = q.dtype == torch.bfloat16
    lse = torch.empty(q.shape[:2], device="cuda")
    out = c.attend(q, scale=scale, decay=0.0, lse=lse)
    w = c.weight.clone()
    G = q.shape[1] // c.h_kv
    run = 2.0 ** -20 + tiles_per_share * (2.0 ** -22 + 2 * U) + (64 + parts) * U
    for i in range(c.b):
        for j in range(c.h_kv):
            n, hs = int(c.n_tok[i, j]), slice(j * G, (j + 1) * G)
            nb = -(-n // c.block)
            assert torch.all(w[i, j, nb:] == 3.0)
            if n == 0:
                assert not out[i, hs].any() and torch.all(lse[i, hs] == -float("inf"))
                continue
            o, l, wb, mag, lm, top = attend_pair(c, q[i, hs], scale, i, j)
            dl = (c.d + 8) * U * lm
            p = 2 * dl + run + (2.0 ** -16 if bf else 2.0 ** -22)
            tol = STEP[q.dtype] * o.abs() + p[:, None] * mag + (128 * 2.0 ** (-30 if bf else -38) * top)[:, None] + 1e-30
            err = (out[i, hs].double() - o).abs()
            assert torch.all(err <= tol), f"out {i, j}: worst {float((err / tol).max()):.3g} of the tolerance"
            assert torch.all((lse[i, hs].double() - l).abs() <= dl + run + 8 * U * l.abs()), f"lse {i, j}"
            err = (w[i, j, :nb].double() - wb).abs()
            assert torch.all(err <= (2 * dl.max() + run + 128 * U) * wb + 1e-30), f"weights {i, j}"
    return out, w


@pytest.mark.parametrize("dtype,d,G,block", [
    ("bf16", 64, 1, 32), ("bf16", 64, 4, 64), ("bf16", 64, 8, 64), ("bf16", 128, 1, 128), ("bf16", 128, 2, 32),
    ("bf16", 128, 4, 64), ("bf16", 128, 8, 32), ("f32", 64, 1, 64), ("f32", 64, 4, 32), ("f32", 64, 8, 128),
    ("f32", 128, 1, 32), ("f32", 128, 4, 128), ("f32", 128, 8, 64)])
def test_attend_turns_its_ring_many_times(dtype, d, G, block):
    """A CTA's share is three times its stages or more (2 to 6 stages, two or three CTAs per SM),
    and pairs of no, one and a few tiles end and begin inside shares; twice the same bits."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = (36 if d == 64 else 18) * sms                    # 18 per CTA at two CTAs per SM, 12 at three; half for d = 128
    few = [1, 0, 127, 128, 129, 300, 64, 5, 1000, 2, 640, 0, 17]
    rest = tiles * 128 - 2 * sum(few)
    lens = [rest // 2 + 1, *few, rest // 3, *few[::-1], rest - rest // 2 - rest // 3 + 77]
    g = gen(d + G)
    c = cache_of_codes(g, lens, 1, d, block)
    q = randn(g, len(lens), G, d).to(DT[dtype])
    out, w = attend_as_defined(c, q, 0.5, 40, 3 * sms)
    assert torch.equal(c.attend(q, scale=0.5, decay=0.0), out) and torch.equal(c.weight, w)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,G,block,lens", [
    (64, 2, 8, 16, [496, 183]), (64, 1, 1, 32, [512, 0, 1]), (128, 2, 4, 128, [512, 129, 385]), (128, 3, 2, 64, [300, 448]),
    (64, 4, 4, 64, [64, 65, 511]), (128, 1, 8, 16, [481])])
def test_attend_in_one_launch_and_in_two(dtype, d, h, G, block, lens):
    """The same tokens under a table of four tiles per pair, which one CTA finishes, and under one of many, whose
    shares a second launch joins."""
    g = gen(d + G)
    c = cache_of_codes(g, lens, h, d, block)
    q = randn(g, len(lens), h * G, d).to(DT[dtype])
    for mb in (512 // block, 4096 // block):
        table = torch.zeros(len(lens), h, mb, dtype=torch.int32, device="cuda")
        table[:, :, :c.max_blocks] = c.table
        x = binding.BlockCache(c.k_codes, c.v_codes, c.k_scale, c.v_scale, table, c.n_tok, torch.full_like(table, 3, dtype=torch.float32))
        attend_as_defined(x, q, 0.5, 4, 4)
        x.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_wide_queries_and_scales(dtype):
    """Query entries over 2^20 and V scales over 2^16 inside a tile, some of them zero: beside the
    usual roundings the row's floor (2^-29 or 2^-37 of the largest entry, times sum |k|) moves the logits."""
    d, h, G, dt = 128, 2, 4, DT[dtype]
    g = gen(5)
    c = cache_of_codes(g, [900, 128, 77], h, d, 16)
    c.v_scale.copy_(torch.exp2(torch.randint(-16, 1, c.v_scale.shape, generator=g, device="cuda").float()) * (torch.rand(c.v_scale.shape, generator=g, device="cuda") > 0.1))
    q = (randn(g, 3, h * G, d) * torch.exp2(-20 * torch.rand(3, h * G, d, generator=g, device="cuda"))).to(dt)
    lse = torch.empty(3, h * G, device="cuda")
    out = c.attend(q, scale=0.5, lse=lse)
    bf = dt == torch.bfloat16
    for i in range(3):
        for j in range(h):
            hs = slice(j * G, (j + 1) * G)
            o, l, _, mag, lm, top = attend_pair(c, q[i, hs], 0.5, i, j)
            ones = attend_pair(c, q[i, hs].abs().amax(-1, keepdim=True).expand(G, d), 0.5, i, j)[4]   # largest entry x sum |k|
            dl = (d + 8) * U * lm + 2.0 ** (-29 if bf else -37) * ones
            p = 2 * dl + 2.0 ** -19 + 128 * U + (2.0 ** -16 if bf else 2.0 ** -22)
            tol = STEP[dt] * o.abs() + p[:, None] * mag + (128 * 2.0 ** (-30 if bf else -38) * top)[:, None] + 1e-30
            err = (out[i, hs].double() - o).abs()
            assert torch.all(err <= tol), f"out {i, j}: worst {float((err / tol).max()):.3g} of the tolerance"
            assert torch.all((lse[i, hs].double() - l).abs() <= dl + 2.0 ** -20 + 8 * U * l.abs())


# ------------------------------------------------------------ calls the interface allows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_of_single_sequences_heads_and_tokens_do_not_matter(dtype):
    """One token of one sequence cut from a row of odd length: the odd strides belong to extents of 1."""
    dt = DT[dtype]
    n = 6 * 64 + 1
    qkv = randn(gen(1), n).to(dt).as_strided((1, 6, 1, 64), (n, 64, n, 1))
    same = qkv.contiguous()
    q, k = binding.qk_norm_rope(qkv[:, :4], qkv[:, 4:5])
    a, b = binding.qk_norm_rope(same[:, :4], same[:, 4:5])
    assert torch.equal(q, a) and torch.equal(k, b)
    caches = [binding.BlockCache.empty(1, 1, 64, 2, block=16) for _ in range(2)]
    for c, y in zip(caches, (qkv, same)):
        c.append(y[:, 4:5], y[:, 5:])
    c, e = caches
    assert torch.equal(c.k_codes, e.k_codes) and torch.equal(c.v_codes, e.v_codes) and torch.equal(c.n_tok, e.n_tok)
    assert torch.equal(c.attend(qkv[:, :4, 0]), e.attend(same[:, :4, 0]))
    odd = torch.zeros(n, dtype=dt, device="cuda").as_strided((1, 4, 1, 64), (n, 64, n, 1))
    binding.qk_norm_rope(qkv[:, :4], None, q_out=odd)
    assert torch.equal(odd, q)


def test_norm_rope_on_a_stream_with_outputs_given():
    """With nothing to allocate the call goes to the stream as it is: handles of any kind, one output given and one made."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    x = randn(gen(1), 2, 3, 50, 128).bfloat16()
    want, _ = binding.qk_norm_rope(x, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(x) for _ in range(4)]
    s.wait_stream(torch.cuda.current_stream())
    binding.qk_norm_rope(x, None, q_out=outs[0], stream=s)
    binding.qk_norm_rope(x, x, q_out=outs[1], k_out=outs[2], stream=s.cuda_stream)
    a, b = binding.qk_norm_rope(x, x, q_out=outs[3], stream=Handle(s))
    s.synchronize()
    assert a is outs[3]
    for t in (*outs, b):
        assert torch.equal(t, want)


def test_rotation_keeps_fp32_factors_in_bf16():
    """Where the two products cancel, the result's own rounding is small and shows the factors: sine and
    cosine within 2 ulp of the reduced angle (2^-23) and the angle to 2^-25, two products and a
    sum in fp32 (2 U of the terms)."""
    g = gen(2)
    b, s, h, d = 4, 2048, 4, 128
    x = randn(g, b, h, s, d).bfloat16()
    pos = torch.randint(0, 2**31 - 1, (b, s), generator=g, device="cuda", dtype=torch.int32)
    got, _ = binding.qk_norm_rope(x, None, norm=False, theta=5e5, pos=pos)
    ref, mag = D.norm_rope(np64(x), None, 0, False, 5e5, d, pos.cpu().numpy().astype(np.float64))
    tol = STEP[torch.bfloat16] * np.abs(ref) + (2.0 ** -23 + 2.0 ** -25 + 2 * U) * mag
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("spare", [0, 60])
def test_attend_output_over_its_own_query(spare):
    c = cache_of_codes(gen(1), [500, 77], 2, 64, 64)
    table = torch.zeros(2, 2, 8 + spare, dtype=torch.int32, device="cuda")
    table[:, :, :8] = c.table
    c = binding.BlockCache(c.k_codes, c.v_codes, c.k_scale, c.v_scale, table, c.n_tok)
    q = randn(gen(2), 2, 8, 64).bfloat16()
    want = c.attend(q)
    assert c.attend(q, out=q) is q and torch.equal(q, want)
