"""The dense decode path on the GPU against 64-bit definitions: norm and
rotation of query and key heads, the e4m3 block cache's append, attention and
eviction, each alone and as a decode loop runs them together.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by
2^-24 (U below).  fp32 work before it is bounded term by term at each test."""
import math

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import dense_oracle as D
from sparse_rank_kv_gb300 import binding, build, synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ------------------------------------------------------------ norm and rotation
def norm_rope_close(got, x, weight, eps, norm, theta, rot, pos):
    """|error| <= half a step of the result + fp32 work on the terms: the sum of squares
    of 128 terms in a lane-wise tree (8 + 4 roundings, halved by the root), the root (2 ulp = 4 U), the
    products (3 U), the rotation (2 products and a sum: 3 U) and its factors, within 2^-20
    (hardware sine and cosine, bf16) or 2^-22 (fp32) of the exact ones."""
    ref, mag = D.norm_rope(np64(x), None if weight is None else np64(weight), eps, norm, theta, rot, pos)
    trig = 2.0 ** -20 if x.dtype == torch.bfloat16 else 2.0 ** -22
    tol = STEP[x.dtype] * np.abs(ref) + (16 * U + (trig if rot else 0.0)) * mag + 1e-37
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,s,hq,h,d,rot,norm,pos", [
    (1, 1, 1, 1, 64, 64, True, None), (3, 1, 32, 8, 128, 128, True, "first"), (2, 7, 4, 2, 64, 32, True, "each"),
    (1, 300, 32, 8, 128, 128, False, "first"), (2, 33, 17, 3, 128, 72, True, "each"), (1, 5, 64, 1, 64, 0, True, None),
    (5, 2, 3, 40, 128, 8, False, "each"), (1, 1000, 1, 1, 128, 120, True, "first"), (70, 9, 2, 2, 64, 64, True, "first")])
def test_norm_rope(dtype, b, s, hq, h, d, rot, norm, pos):
    g = gen(b * 131 + s)
    dt = DT[dtype]
    qkv = (randn(g, b, s, hq + 2 * h, d) * torch.exp2(3 * randn(g, b, s, 1, 1))).to(dt)
    q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + h].transpose(1, 2)
    w = (1 + 0.3 * randn(g, 2, d)).to(dt)
    if pos == "first":
        p = torch.randint(0, 1 << 20, (b,), generator=g, device="cuda", dtype=torch.int32)
        at = np64(p)[:, None] + np.arange(s)
    elif pos == "each":
        p = torch.randint(-5000, 2**31 - 1, (b, s), generator=g, device="cuda", dtype=torch.int32)
        at = p.cpu().numpy().astype(np.float64)
    else:
        p, at = None, np.broadcast_to(np.arange(s, dtype=np.float64), (b, s))
    k_out = torch.empty(b, h, s, d, dtype=dt, device="cuda")
    q0 = q.clone()
    qo, ko = binding.qk_norm_rope(q, k, w[0], w[1], norm=norm, theta=5e5, rot=rot, pos=p, k_out=k_out)
    assert ko is k_out and torch.equal(q, q0)
    norm_rope_close(qo, q, w[0], 1e-6, norm, 5e5, rot, at)
    norm_rope_close(ko, k, w[1], 1e-6, norm, 5e5, rot, at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_forms(dtype):
    """One of q and k alone, no weights, in place, zero rows, untouched neighbours, another stream."""
    g, dt = gen(3), DT[dtype]
    buf = randn(g, 2, 6, 5, 128).to(dt)                      # b, s, h + 2 rows around, d
    x = buf[:, :, 1:4].transpose(1, 2)
    x[0, 1, 2] = 0
    before, at = buf.clone(), np.broadcast_to(np.arange(6.0), (2, 6))
    keep = x.clone()
    qo, ko = binding.qk_norm_rope(x, None)
    assert ko is None
    norm_rope_close(qo, keep, None, 1e-6, True, 1e4, 128, at)
    _, ko = binding.qk_norm_rope(None, x, theta=1e4, rot=64)
    norm_rope_close(ko, keep, None, 1e-6, True, 1e4, 64, at)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    binding.qk_norm_rope(x, None, q_out=x, stream=st)        # in place
    st.synchronize()
    assert torch.equal(x, qo)
    assert torch.equal(buf[:, :, 0], before[:, :, 0]) and torch.equal(buf[:, :, 4], before[:, :, 4])


def test_norm_rope_makes_the_keys_prefill_rotates():
    """rot = 0 gives the pre-RoPE keys shadowkv_prefill takes; its own rotation
    of the last w of them (the exported local window) is this operator's."""
    cfg = synth.CONFIGS["tiny_f32_s1k"]
    inp = synth.make_inputs(cfg, device="cuda")
    k = inp["k_pre"]
    w = 1 + 0.1 * randn(gen(1), cfg.d)
    _, k_pre = binding.qk_norm_rope(None, k, None, w, rot=0)
    ctx = binding.prefill(binding.make_params(cfg), k_pre, inp["v"])
    b, h, d, cap = cfg.b, cfg.h_kv, cfg.d, cfg.w + cfg.max_new
    loc = ctx.export("K_LOC").view(b, h, cap, d)[:, :, :cfg.w]
    _, k_rot = binding.qk_norm_rope(None, k, None, w, theta=cfg.theta)
    ref, mag = D.norm_rope(np64(k_pre), None, 0, False, cfg.theta, d, np.broadcast_to(np.arange(float(cfg.s)), (b, cfg.s)))
    # both sides round k_pre's rotation once and k_pre itself once more on one of them
    tol = 8 * 2.0 ** -22 * mag[:, :, -cfg.w:]
    assert np.all(np.abs(np64(loc) - np64(k_rot[:, :, -cfg.w:])) <= tol)
    ctx.close()


# ------------------------------------------------------------ the cache
def shuffled(b, h, d, max_blocks, block, seed, spare=3):
    """An empty cache whose pairs' blocks lie in the pool in an order of their own; its
    codes start as NaN and its scales too, so that nothing unwritten may count."""
    n = b * h * max_blocks + spare
    c = binding.BlockCache.empty(b, h, d, max_blocks, block=block)
    perm = torch.randperm(n, generator=gen(seed), device="cuda")[:b * h * max_blocks].to(torch.int32)
    mk = lambda *s: torch.full(s, 0x7f, dtype=torch.uint8, device="cuda")  # noqa: E731
    nan = lambda: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
    return binding.BlockCache(mk(n, block // 8, d // 16, 8, 16), mk(n, block // 16, d, 16), nan(), nan(),
                              perm.view(b, h, max_blocks), c.n_tok, c.weight)


def codes_of(c, i, g, blk):
    """(K codes (block, d), K scale, V codes, V scale) of one block as numbers."""
    id_ = int(c.table[i, g, blk])
    f8 = lambda t: t.view(torch.float8_e4m3fn).float()  # noqa: E731
    kc = np64(f8(c.k_codes[id_]).permute(0, 2, 1, 3).reshape(c.block, c.d))
    vc = np64(f8(c.v_codes[id_]).permute(0, 2, 1).reshape(c.block, c.d))
    return kc, float(c.k_scale[id_]), vc, float(c.v_scale[id_])


def same_cache(c, ref):
    for (i, g), bl in ref.blocks.items():
        n = ref.n[i, g]
        assert int(c.n_tok[i, g]) == n
        for j, want in enumerate(bl):
            got = codes_of(c, i, g, j)
            m = min(c.block, n - j * c.block)
            assert got[1] == want[1] and got[3] == want[3], (i, g, j)
            assert np.array_equal(got[0][:m], want[0][:m]) and np.array_equal(got[2][:m], want[2][:m]), (i, g, j)


def tokens(g, b, h, s, d, dt, grow=0.0):
    """k and v whose size changes along the sequence, some rows zero."""
    amp = torch.exp2(grow * torch.arange(s, device="cuda")[:, None] + 4 * randn(g, b, h, s, 1))
    k, v = (randn(g, b, h, s, d) * amp).to(dt), (randn(g, b, h, s, d) * amp).to(dt)
    if s > 4:
        k[:, :, 3] = 0
        v[:, :, 2] = 0
    return k, v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,h,d,block,pieces", [
    (1, 1, 64, 16, [1, 1, 1, 14, 16, 17, 1]), (2, 3, 128, 64, [63, 1, 1, 130, 5, 64]), (2, 2, 64, 32, [200, 1, 31, 33]),
    (1, 2, 128, 128, [127, 2, 300, 1]), (3, 1, 128, 16, [500, 3, 16])])
def test_append_in_pieces(dtype, b, h, d, block, pieces):
    """Single tokens, pieces inside a block, across one and over many, ragged:
    every code and scale equal to the definition's, bytes past the tokens untouched."""
    dt, total = DT[dtype], sum(pieces)
    mb = -(-total // block) + 1
    c, ref = shuffled(b, h, d, mb, block, seed=total), D.Cache(b, h, d, block, mb)
    g = gen(total)
    c.weight.fill_(7.0)
    for i, s in enumerate(pieces):
        k, v = tokens(g, b, h, s, d, dt, grow=0.02 if i % 2 else 0.0)
        lens = None if i % 2 else torch.tensor([max(0, s - 2 * j) for j in range(b)], dtype=torch.int32, device="cuda")
        n0 = c.n_tok.clone()
        c.append(k, v, lens)
        ref.append(np64(k), np64(v), [s] * b if lens is None else lens.tolist())
        same_cache(c, ref)
        for p in ref.n:                                       # blocks begun by this piece
            first = -(-int(n0[p]) // block)
            assert torch.all(c.weight[p][first:len(ref.blocks[p])] == 0)
            c.weight[p] = 7.0
    for p in ref.n:                                           # past the tokens: still NaN
        n = ref.n[p]
        if n % block:
            kc, _, vc, _ = codes_of(c, *p, n // block)
            assert np.isnan(kc[n % block:]).all() and np.isnan(vc[n % block:]).all()
        for j in range(len(ref.blocks[p]), mb):
            kc, ks, vc, vs = codes_of(c, *p, j)
            assert np.isnan(kc).all() and np.isnan(vc).all() and math.isnan(ks) and math.isnan(vs)
    c.check()


def test_append_strided_and_from_norm_rope_layout():
    """Rows of a fused projection (b, s, heads, d) and head-major rows give the same cache."""
    g = gen(9)
    qkv = randn(g, 2, 100, 8, 128).bfloat16()
    k, v = qkv[:, :, 2:5].transpose(1, 2), qkv[:, :, 5:].transpose(1, 2)
    a, b = (binding.BlockCache.empty(2, 3, 128, 4, block=32) for _ in range(2))
    a.append(k, v)
    b.append(k.contiguous(), v.contiguous())
    for x in ("k_codes", "v_codes", "k_scale", "v_scale", "n_tok"):
        assert torch.equal(getattr(a, x), getattr(b, x)), x


def test_append_special_values():
    """Infinities saturate at the scale of the finite entries, NaN stays NaN, zeros get the least scale."""
    c = binding.BlockCache.empty(1, 1, 64, 2, block=16)
    k = torch.ones(1, 1, 3, 64, device="cuda")
    k[0, 0, 0, 0], k[0, 0, 1, 1], k[0, 0, 2, 2] = float("inf"), float("-inf"), float("nan")
    c.append(k, torch.zeros_like(k))
    kc, ks, vc, vs = codes_of(c, 0, 0, 0)
    assert ks == 2.0 ** -8 and vs == 2.0 ** -100 and not vc[:3].any()
    assert kc[0, 0] == 448 and kc[1, 1] == -448 and math.isnan(kc[2, 2]) and kc[0, 1] == 256
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s", [1, 4])
def test_append_onto_a_callers_own_scales(dtype, s):
    """A partly filled block whose scale the caller chose (no power of two, larger
    than the new tokens need or smaller, negative, zero) keeps its values up to one
    rounding of its codes; new tokens are quantised by the scale that results."""
    scales = [0.3, 1000.0, -1000.0, -0.01, 0.0, 3e-5]
    c, ref = filled(1, len(scales), 64, 16, [21], DT[dtype], seed=44)
    for h, x in enumerate(scales):
        id_ = int(c.table[0, h, 1])
        c.k_scale[id_], c.v_scale[id_] = x, -x
        ref.blocks[0, h][1][1], ref.blocks[0, h][1][3] = np.float32(x).astype(np.float64), -np.float32(x).astype(np.float64)
    k, v = tokens(gen(4), 1, len(scales), s, 64, DT[dtype])
    c.append(k, v)
    ref.append(np64(k), np64(v), [s])
    for h in range(len(scales)):
        kc, ks, vc, vs = codes_of(c, 0, h, 1)
        want = ref.blocks[0, h][1]
        assert ks == want[1] and vs == want[3]
        for got, exp in ((kc, want[0]), (vc, want[2])):
            # quotients here are fp32 divisions: a tie may fall to the other neighbour (a step: 2^-3 of the value, 2^-9 at least)
            err = np.abs(got[:5 + s] - exp[:5 + s])
            assert np.all(err <= np.maximum(2.0 ** -3 * np.abs(exp[:5 + s]), 2.0 ** -9) * 1.001)
            assert np.mean(err > 0) < 0.02
    c.check()


def test_append_past_the_end_is_dropped_and_reported():
    c = binding.BlockCache.empty(1, 2, 64, 2, block=16)
    k = randn(gen(1), 1, 2, 30, 64)
    c.append(k, k)
    c.check()
    c.append(k[:, :, :7], k[:, :, :7])
    assert c.n_tok.tolist() == [[32, 32]]
    with pytest.raises(binding.ShadowKVError) as e:
        c.check()
    assert e.value.code == 4
    ref = D.Cache(1, 2, 64, 16, 2)
    ref.append(np64(k), np64(k), [30])
    ref.append(np64(k[:, :, :7]), np64(k[:, :, :7]), [7])
    same_cache(c, ref)
    for bad in (-3, 9):                                       # a length outside 0..s is clamped
        c.status.zero_()
        c.reset()
        c.append(k[:, :, :7], k[:, :, :7], torch.tensor([bad], dtype=torch.int32, device="cuda"))
        assert int(c.n_tok[0, 0]) == max(0, min(7, bad))
        with pytest.raises(binding.ShadowKVError):
            c.check()


# ------------------------------------------------------------ attention
def attend_close(out, lse, q, ref, dtype):
    """|error| <= half a step of the result + what moves p: a logit is a sum of d exact products in
    fp32 (d roundings of its largest partial sum, and 8 of its own scaling), p moves by as much twice (its own and
    the sum's), the exponential is within 2^-21, p itself is held to 2^-11 (bf16: rounded to fp16, half a step of 2^-10) or 2^-23 (fp32), and
    sums over n tokens cost at most 64 roundings in tiles and partials.  Below that p has a
    floor: with its tile's largest p V-scale at 256, the last of T e4m3 terms ends at half the
    least step, 2^-10 16^(1-T) (T = 3: 2^-18, so 2^-26 of the largest; T = 6: 2^-38), times
    a code of at most 448, for each of the tile's 128 tokens."""
    o, l, mag, lm, top = ref
    bf = dtype == torch.bfloat16
    dl = (q.shape[-1] + 8) * U * lm
    p = 2 * dl + 2.0 ** -20 + 64 * U + (2.0 ** -11 if bf else 2.0 ** -22)
    tol = STEP[dtype] * np.abs(o) + p[..., None] * mag + (128 * 2.0 ** (-26 if bf else -38) * top)[..., None] + 1e-30
    err = np.abs(np64(out) - o)
    assert np.all(err <= tol), f"out: worst {np.max(err / tol):.3g} of the tolerance"
    if lse is not None:
        got = np64(lse)
        assert np.array_equal(np.isneginf(got), np.isneginf(l))
        f = np.isfinite(l)
        tol = dl + 2.0 ** -20 + 8 * U * np.abs(np.where(f, l, 0))
        assert np.all(np.abs(got[f] - l[f]) <= tol[f]), "lse"
    return dl


def weights_close(c, ref, dl):
    G = dl.shape[1] // c.h_kv
    for (i, g), w in ref.weight.items():
        if not w:
            continue
        tol = (2 * dl[i, g * G:(g + 1) * G].max() + 2.0 ** -19 + 128 * U) * np.abs(w) + 1e-30
        err = np.abs(np64(c.weight[i, g, :len(w)]) - np.asarray(w))
        assert np.all(err <= tol), f"weights {i, g}: {np.max(err / tol):.3g} of the tolerance"


def filled(b, h, d, block, lens, dt, seed, spare=1):
    mb = max(1, -(-max(lens) // block)) + spare
    c, ref = shuffled(b, h, d, mb, block, seed), D.Cache(b, h, d, block, mb)
    s = max(max(lens), 1)
    g = gen(seed)
    k, v = tokens(g, b, h, s, d, dt)
    k = (k.float() / k.float().abs().amax(-1, keepdim=True).clamp(min=1e-3) * (1 + 2 * torch.rand(b, h, s, 1, generator=g, device="cuda"))).to(dt)
    c.append(k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ref.append(np64(k), np64(v), lens)
    return c, ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,G,d,block,lens", [
    (1, 1, 64, 16, [1]), (2, 4, 128, 64, [128, 0, 1, 65]), (1, 8, 128, 128, [129, 127, 1000]), (3, 2, 64, 32, [500, 33, 0, 31]),
    (8, 4, 128, 64, [777]), (2, 1, 128, 16, [255, 257, 3000]), (1, 4, 64, 128, [0, 0, 5]), (4, 8, 64, 64, [640, 64, 63])])
def test_attend(dtype, h, G, d, block, lens):
    b, dt = len(lens), DT[dtype]
    c, ref = filled(b, h, d, block, lens, dt, seed=sum(lens) + G)
    g = gen(5)
    q = (randn(g, b, h * G, d) * torch.exp2(torch.randint(-2, 2, (b, h * G, d), generator=g, device="cuda").float())).to(dt)
    lse = torch.full((b, h * G), 9.0, device="cuda")
    c.weight.fill_(3.0)
    out = c.attend(q, lse=lse)
    want = ref.attend(np64(q), d ** -0.5)
    attend_close(out, lse, q, want, dt)
    assert torch.all(c.weight == 3.0)                          # not gathered
    # gathered: decay 0 does not read the old weights, 0.5 does; entries past the blocks stay
    c.weight.fill_(float("nan"))
    for p in ref.n:
        c.weight[p][len(ref.blocks[p]):] = 3.0
    assert torch.equal(c.attend(q, decay=0.0), out)
    dl = attend_close(out, None, q, ref.attend(np64(q), d ** -0.5, 0.0), dt)
    weights_close(c, ref, dl)
    ref.attend(np64(q), d ** -0.5, 0.5)
    c.attend(q, decay=0.5)
    weights_close(c, ref, 2 * dl)
    for p in ref.n:
        assert torch.all(c.weight[p][len(ref.blocks[p]):] == 3.0)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_many_splits_and_many_pairs(dtype):
    """One pair over every CTA, and more pairs than CTAs with lengths from 0 to 300."""
    dt = DT[dtype]
    c, ref = filled(1, 1, 128, 64, [50000], dt, seed=2)
    q = randn(gen(1), 1, 4, 128).to(dt)
    lse = torch.empty(1, 4, device="cuda")
    out = c.attend(q, lse=lse, decay=0.0)
    dl = attend_close(out, lse, q, ref.attend(np64(q), 128 ** -0.5, 0.0), dt)
    weights_close(c, ref, dl)
    lens = [(i * 37) % 301 for i in range(130)]
    c, ref = filled(130, 3, 64, 16, lens, dt, seed=3)
    q = randn(gen(2), 130, 6, 64).to(dt)
    out = c.attend(q, decay=0.0)
    dl = attend_close(out, None, q, ref.attend(np64(q), 0.125, 0.0), dt)
    weights_close(c, ref, dl)


@pytest.mark.parametrize("spare", [1, 60])
@pytest.mark.parametrize("dtype,b,h,G,d,block,lens", [
    ("bf16", 60, 3, 4, 128, 64, lambda i: (i * 173) % 961), ("f32", 2, 2, 8, 64, 16, lambda i: 500 - 313 * i),
    ("bf16", 3, 1, 2, 64, 128, lambda i: 128 * i + (i == 2)), ("f32", 80, 2, 1, 128, 32, lambda i: (i * 29) % 300)])
def test_attend_with_and_without_a_second_launch(spare, dtype, b, h, G, d, block, lens):
    """The same tokens in a cache of few tiles per pair (one CTA finishes a pair)
    and of many (shares joined by a second launch)."""
    dt = DT[dtype]
    c, ref = filled(b, h, d, block, [lens(i) for i in range(b)], dt, seed=b + spare, spare=spare)
    q = randn(gen(2), b, h * G, d).to(dt)
    lse = torch.empty(b, h * G, device="cuda")
    want = ref.attend(np64(q), 0.1, 0.0)
    dl = attend_close(c.attend(q, scale=0.1, decay=0.0, lse=lse), lse, q, want, dt)
    weights_close(c, ref, dl)
    c.check()


def test_attend_scale_strides_out_and_peaked_rows():
    """A scale of one's own (0 and negative too), q and out as strided views,
    and logits far apart: one token takes everything."""
    c, ref = filled(2, 2, 128, 64, [300, 77], torch.bfloat16, seed=8)
    buf = randn(gen(3), 2, 20, 128).bfloat16()
    q = buf[:, 3:19:2]                                        # b, 8 heads, d
    o = torch.zeros(2, 8, 3, 128, dtype=torch.bfloat16, device="cuda")
    for scale in (0.0, -0.3, 0.01, 40.0):
        got = c.attend(q, scale=scale, out=o[:, :, 1])
        assert got.data_ptr() == o[:, :, 1].data_ptr()
        attend_close(got, None, q, ref.attend(np64(q), scale), torch.bfloat16)
    assert not o[:, :, 0].any() and not o[:, :, 2].any()


def test_attend_caller_scales():
    """Scales that are no powers of two, negative and zero ones: the value is code times scale."""
    c, ref = filled(1, 2, 64, 16, [100], torch.float32, seed=12)
    f = torch.tensor([0.3, -1.7, 0.0, 2.5, 1.0, 0.9, 3.3], device="cuda")
    for i in range(2):
        for j in range(7):
            id_ = int(c.table[0, i, j])
            c.k_scale[id_] *= f[j]
            c.v_scale[id_] *= f[6 - j]
            ref.blocks[0, i][j][1] = float(c.k_scale[id_])
            ref.blocks[0, i][j][3] = float(c.v_scale[id_])
    q = randn(gen(3), 1, 4, 64)
    attend_close(c.attend(q), None, q, ref.attend(np64(q), 0.125), torch.float32)


def test_attend_nan_and_infinite_queries_stay_in_their_heads():
    c, ref = filled(1, 2, 128, 64, [200], torch.bfloat16, seed=4)
    q = randn(gen(6), 1, 8, 128).bfloat16()
    good = c.attend(q)
    bad = q.clone()
    bad[0, 1, 5], bad[0, 6, 0] = float("nan"), float("inf")
    out = c.attend(bad)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 6]).all()
    rest = [0, 2, 3, 4, 5, 7]
    assert torch.equal(out[0, rest], good[0, rest])
    # a NaN value row reaches exactly its dimension's outputs, of the heads that read it
    k = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    v[0, 0, 0, 9] = float("nan")
    c.append(k, v)
    out = c.attend(q)
    assert torch.isnan(out[0, :4, 9]).all()
    out[0, :4, 9] = 0
    assert torch.isfinite(out).all()


def test_attend_bad_block_ids_are_read_as_block_0_and_reported():
    c, _ = filled(1, 1, 64, 16, [64], torch.float32, seed=4)
    q = randn(gen(6), 1, 2, 64)
    t = c.table.clone()
    c.table[0, 0, 1], c.table[0, 0, 2] = -1, 10**9
    out = c.attend(q)
    with pytest.raises(binding.ShadowKVError) as e:
        c.check()
    assert e.value.code == 4
    c.table.copy_(t)
    c.table[0, 0, 1:3] = 0
    c.status.zero_()
    z = c.k_scale[0].clone()
    assert torch.equal(c.attend(q).isnan(), out.isnan()) and torch.equal(z.isnan(), c.k_scale[0].isnan())
    c.check()
    c.n_tok.fill_(10**6)
    c.attend(q)
    with pytest.raises(binding.ShadowKVError):
        c.check()


def test_attend_refuses_a_small_workspace():
    c = binding.BlockCache.empty(1, 2, 128, 4)
    need = binding.lib().shadowkv_cache_attend_workspace(c._desc, 8)
    assert need > 0
    w = torch.empty(need, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 8, 128, device="cuda")
    r = binding.Rows(q.data_ptr(), 1024, 128, 0)
    assert binding.lib().shadowkv_cache_attend(c._desc, 0, 8, r, 1.0, 0, 0.0, r, None, w.data_ptr(), need - 1, None) == 1
    with pytest.raises(binding.ShadowKVError):
        c.attend(torch.zeros(1, 6, 128, device="cuda"))


# ------------------------------------------------------------ eviction
def ids(c, i, g, n):
    return c.table[i, g, :n].tolist()


@pytest.mark.parametrize("block,lens,keep,sink,recent", [
    (16, [100], 3, 1, 1), (64, [64 * 40 + 5, 64 * 7, 0, 64 * 8], 8, 0, 2), (32, [32 * 300, 9000], 100, 2, 0),
    (128, [128 * 1500 + 1], 777, 4, 4), (16, [16 * 9000 + 3, 16 * 5000], 4096, 1, 64), (64, [6400], 1, 0, 0), (64, [6400], 1, 1, 0),
    (64, [6401], 1, 0, 1), (16, [33], 3, 0, 0)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(block, lens, keep, sink, recent, ties):
    b, h, mb = len(lens), 2, -(-max(lens) // block) + 2
    c = binding.BlockCache.empty(b, h, 64, mb, block=block)
    g = gen(keep)
    c.table.copy_(torch.stack([torch.randperm(b * h * mb, generator=g, device="cuda")[:mb] for _ in range(b * h)])
                  .view(b, h, mb).to(torch.int32))
    c.n_tok.copy_(torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(b, h))
    w = randn(g, b, h, mb).exp()
    if ties:
        w = (w * 2).round() / 2 - 0.5
        w[0, 0, ::5] = float("nan")
        w[0, 1, ::7] = float("-inf")
        w[0, 1, 1::9] = float("inf")
        w[0, 1, 2::9] = -0.0
    c.weight.copy_(w)
    t0, w0 = c.table.cpu().numpy(), np64(w)
    kept = torch.full((b, h, keep), 77, dtype=torch.int32, device="cuda")
    f = c.fork()
    c.evict(keep, sink=sink, recent=recent, into=f, kept=kept)
    assert np.array_equal(c.table.cpu().numpy(), t0)            # the source stays
    c.evict(keep, sink=sink, recent=recent)                     # in place
    for x in ("table", "n_tok", "weight"):
        assert torch.equal(getattr(c, x).nan_to_num(), getattr(f, x).nan_to_num()), x
    for i in range(b):
        n = -(-lens[i] // block)
        for j in range(h):
            want, tok = D.evict(w0[i, j], lens[i], block, keep, sink, recent)
            assert [x for x in kept[i, j].tolist() if x >= 0] == want and kept[i, j].tolist()[len(want):] == [-1] * (keep - len(want))
            assert int(c.n_tok[i, j]) == tok
            gone = [x for x in range(n) if x not in set(want)]
            order = want + gone + list(range(n, mb))
            assert np.array_equal(c.table[i, j].cpu().numpy(), t0[i, j][order])
            exp = np.zeros(mb)
            exp[:len(want)] = w0[i, j][want]
            assert np.array_equal(np64(c.weight[i, j]), exp, equal_nan=True)
    c.check()


# ------------------------------------------------------------ together
def test_decode_loop_with_eviction():
    """Norm and rotation, append, attention that gathers, eviction over budget:
    a ragged prompt and 64 steps against the 64-bit definitions fed with the same
    rounded q, k, v, through evictions and the reuse of freed blocks."""
    b, hq, h, d, block, keep, T = 3, 8, 2, 128, 16, 6, 64
    lens = [70, 16, 1]
    g = gen(11)
    wq, wk = (1 + 0.2 * randn(g, 2, d)).bfloat16()
    mb = keep + 2
    c, ref = shuffled(b, h, d, mb, block, 1), D.Cache(b, h, d, block, mb)
    qkv = randn(g, b, 70, hq + 2 * h, d).bfloat16()
    view = lambda x, a, n: x[:, :, a:a + n].transpose(1, 2)  # noqa: E731
    _, k = binding.qk_norm_rope(None, view(qkv, hq, h), None, wk, theta=5e5)
    c.append(k, view(qkv, hq + h, h), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ref.append(np64(k), np64(view(qkv, hq + h, h)), lens)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    evictions = 0
    for t in range(T):
        qkv = randn(g, b, 1, hq + 2 * h, d).bfloat16()
        q, k = binding.qk_norm_rope(view(qkv, 0, hq), view(qkv, hq, h), wq, wk, theta=5e5, pos=pos)
        v = view(qkv, hq + h, h)
        at = np.asarray(lens)[:, None] + t
        norm_rope_close(q, view(qkv, 0, hq), wq, 1e-6, True, 5e5, d, at)
        c.append(k, v)
        ref.append(np64(k), np64(v), [1] * b)
        q1 = q[:, :, 0]
        out = c.attend(q1, decay=0.9)
        dl = attend_close(out, None, q1, ref.attend(np64(q1), d ** -0.5, 0.9), torch.bfloat16)
        weights_close(c, ref, (t + 1) * dl + 2.0 ** -19)
        kept = torch.empty(b, h, keep, dtype=torch.int32, device="cuda")
        c.evict(keep, sink=1, recent=2, kept=kept)
        for p, w in ref.weight.items():
            want, tok = D.evict(np64(c.weight[p])[:len(w)] if len(w) <= keep else w, ref.n[p], block, keep, 1, 2)
            got = [x for x in kept[p].tolist() if x >= 0]
            evictions += len(w) > keep
            assert len(got) == len(want)
            # a different choice only between weights that the tolerance cannot tell apart
            for x, y in zip(sorted(set(got) - set(want)), sorted(set(want) - set(got))):
                assert abs(w[x] - w[y]) <= 1e-4 * abs(w[y])
            ref.weight[p] = [w[x] for x in got]
            ref.blocks[p] = [ref.blocks[p][x] for x in got]
            ref.n[p] = tok
        same_cache(c, ref)
        pos += 1
    # the first sequence exceeds 96 tokens at its 27th step and a block more 16 and 32 steps later, in both heads
    assert evictions == 6
    c.check()


def test_captured_steps_replay_and_streams():
    """A decode step captured twice into graphs of their own workspaces, replayed in
    turn and on another stream, equals the same calls made eagerly."""
    b, hq, h, d = 2, 8, 2, 64

    def step(c, qkv, pos, out):
        q, k = binding.qk_norm_rope(qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + h].transpose(1, 2), pos=pos)
        c.append(k, qkv[:, :, hq + h:].transpose(1, 2))
        c.attend(q[:, :, 0], decay=1.0, out=out)
        c.evict(5, recent=1)
        pos += 1

    g = gen(21)
    xs = randn(g, 60, b, 1, hq + 2 * h, d)
    eager, cap = (binding.BlockCache.empty(b, h, d, 7, block=16) for _ in range(2))
    pe, pc = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))
    oe = torch.empty(b, hq, d, device="cuda")
    want = []
    for x in xs:
        step(eager, x, pe, oe)
        want.append(oe.clone())
    buf, oc = torch.empty_like(xs[0]), torch.empty_like(oe)
    warm = binding.BlockCache.empty(b, h, d, 7, block=16)
    step(warm, xs[0], torch.zeros_like(pc), torch.empty_like(oe))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(cap, buf, pc, oc)
        graphs.append(gr)
    cap.reset(), cap.weight.zero_(), pc.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t, x in enumerate(xs):
            buf.copy_(x)
            graphs[t % 2].replay()
            assert torch.equal(oc, want[t]), t
    side.synchronize()
    assert torch.equal(cap.table, eager.table) and torch.equal(cap.n_tok, eager.n_tok) and torch.equal(cap.weight, eager.weight)
    cap.check()


def test_attend_calls_may_overlap_without_gathering():
    c, ref = filled(2, 2, 128, 64, [3000, 100], torch.bfloat16, seed=31)
    qs = [randn(gen(i), 2, 8, 128).bfloat16() for i in range(8)]
    want = [c.attend(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [c.attend(q, stream=streams[i % 4]) for i, q in enumerate(qs)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_new_token_made_by_norm_rope_feeds_the_sparse_decode_step():
    """qk_norm_rope's q and k straight into shadowkv_decode_step, nothing in between:
    the appended local-window rows and the outputs equal those of inputs made
    beforehand (the step's kernels may start early, never before their inputs are there)."""
    cfg = synth.CONFIGS["llama_b1_s32k"].with_(s=4096 + 64, k=32, o=16, steps=12, seed=7)
    st = synth.make_state(cfg, device="cuda")
    p = binding.make_params(cfg)
    b, hq, h, d = cfg.b, cfg.h_q, cfg.h_kv, cfg.d
    g = gen(17)
    qkv = randn(g, cfg.steps, b, 1, hq + 2 * h, d).bfloat16()
    pos = torch.full((b,), cfg.s, dtype=torch.int32, device="cuda")

    def run(ready):
        ctx = binding.load_state(p, st)
        outs = []
        made = []
        for t in range(cfg.steps):
            x = qkv[t]
            if ready:
                q, k = ready[t]
            else:
                q, k = torch.empty(b, hq, 1, d, dtype=x.dtype, device="cuda"), torch.zeros(b, h, 1, d, dtype=x.dtype, device="cuda")
                v = x[:, 0, hq + h:].contiguous()
                out = torch.empty(b, hq, d, dtype=x.dtype, device="cuda")
                torch.cuda.synchronize()
                binding.qk_norm_rope(x[:, :, :hq].transpose(1, 2), x[:, :, hq:hq + h].transpose(1, 2), theta=cfg.theta,
                                     pos=pos, q_out=q, k_out=k)
            if ready:
                v = x[:, 0, hq + h:].contiguous()
                out = torch.empty(b, hq, d, dtype=x.dtype, device="cuda")
                torch.cuda.synchronize()
            ctx.decode_step(q.view(b, hq, d), k.view(b, h, d), v, out)
            outs.append(out)
            made.append((q, k))
        torch.cuda.synchronize()
        loc = ctx.export("K_LOC")
        ctx.check()
        ctx.close()
        return outs, made, loc

    outs, made, loc = run(None)
    again, _, loc2 = run(made)
    assert torch.equal(loc, loc2)
    for a, c in zip(outs, again):
        assert torch.equal(a, c)


def test_blocks_shared_by_sequences():
    """Two sequences whose tables name the same blocks (a common prompt) attend
    over them as over copies of their own."""
    c, ref = filled(2, 2, 128, 16, [70, 70], torch.bfloat16, seed=3)
    c.table[1, :, :4] = c.table[0, :, :4]
    for h in range(2):
        ref.blocks[1, h][:4] = ref.blocks[0, h][:4]
    q = randn(gen(1), 2, 8, 128).bfloat16()
    dl = attend_close(c.attend(q, decay=0.0), None, q, ref.attend(np64(q), 128 ** -0.5, 0.0), torch.bfloat16)
    weights_close(c, ref, dl)


def test_offsets_past_32_bits():
    """Blocks and rows whose byte and element offsets pass 2^32: the last blocks of a
    pool of 4.6 GB a side, and rows 2^31 + 8 elements apart."""
    n = 560000                                                 # 8 KB each
    big = binding.BlockCache(torch.empty(n, 8, 8, 8, 16, dtype=torch.uint8, device="cuda"),
                             torch.empty(n, 4, 128, 16, dtype=torch.uint8, device="cuda"), torch.zeros(n, device="cuda"),
                             torch.zeros(n, device="cuda"), torch.arange(n - 8, n, dtype=torch.int32, device="cuda").view(2, 1, 4),
                             torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, 4, device="cuda"))
    small = binding.BlockCache.empty(2, 1, 128, 4)
    far = torch.empty(2**31 + 8 + 200 * 128, dtype=torch.bfloat16, device="cuda")
    k = far.as_strided((2, 1, 150, 128), (2**31 + 8, 150 * 128, 128, 1))
    k.copy_(randn(gen(2), 2, 1, 150, 128))
    for c in (big, small):
        c.append(k, k)
        c.append(k[:, :, :1], k[:, :, 1:2])
    q = randn(gen(3), 2, 4, 128).bfloat16()
    assert torch.equal(big.attend(q, decay=0.0), small.attend(q, decay=0.0))
    assert torch.equal(big.weight, small.weight)
    near = k.contiguous()
    a, _ = binding.qk_norm_rope(k, None)
    b, _ = binding.qk_norm_rope(near, None)
    assert torch.equal(a, b)
    binding.qk_norm_rope(near, None, q_out=k)
    assert torch.equal(k, b)
    big.check()


def test_empty_calls_and_reset():
    c = binding.BlockCache.empty(2, 2, 64, 3, block=16)
    e = torch.empty(2, 2, 0, 64, device="cuda")
    c.append(e, e)
    q, k = binding.qk_norm_rope(e, e)
    assert q.shape == k.shape == e.shape
    x = randn(gen(1), 2, 2, 40, 64)
    c.append(x, x, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert not c.n_tok.any()
    one = x[:, :, :1]
    c.append(one, one, torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert c.n_tok.tolist() == [[0, 0], [1, 1]]
    out = c.attend(one[:, :, 0])
    assert not out[0].any() and torch.isfinite(out).all()
    c.evict(1, recent=0)
    assert c.n_tok.tolist() == [[0, 0], [1, 1]]
    c.reset()
    assert not c.attend(one[:, :, 0]).any()
    c.check()


def test_stream_handles():
    """A raw cudaStream_t and a torch stream serve as the calls' stream."""
    c, ref = filled(1, 2, 64, 16, [100], torch.float32, seed=6)
    q = randn(gen(2), 1, 4, 64)
    want = c.attend(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.attend(q, stream=s.cuda_stream)
    k = randn(gen(3), 1, 2, 5, 64)
    s.wait_stream(torch.cuda.current_stream())
    c.append(k, k, stream=s)
    c.evict(4, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and c.n_tok.tolist() == [[3 * 16 + 9, 3 * 16 + 9]]
