"""Verification of drafted tokens on the GPU against its definition in 64 bits.

Whole numbers come out, so they have to be equal, unless a decision lies so near its
border that fp32 inputs carried through 2^-37 weights may fall on the other side:
2^-33 of the numbers compared, which one case in 2^20 of the sizes here meets; such a
case's inputs would be excluded by that bound alone (none is)."""
import numpy as np
import pytest
import torch

from oracle import pool_oracle as PO
from sparse_rank_kv_gb300 import binding, build

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -33
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def made(b, s, v, dtype, seed, spread=3.0, apart=0.5):
    """Logits, drafts sampled from a distribution near the target's, that distribution, random numbers."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = (spread * torch.randn(b, s + 1, v, generator=g, device="cuda")).to(DT[dtype])
    scores = logits[:, :s].float() + apart * torch.randn(b, s, v, generator=g, device="cuda")
    u = torch.rand(b, s, v, generator=g, device="cuda").clamp(1e-30, 1 - 1e-7)
    drafts = torch.argmax(scores - torch.log(-torch.log(u)), -1).to(torch.int32) if s else ints([[]] * b).view(b, 0)
    rnd = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    return logits, drafts, torch.softmax(scores, -1), rnd(b, s), rnd(b)


def agree(got, logits, drafts, probs, accept, sample, lens=None, temperature=1.0):
    tokens, accepted = (x.cpu().numpy() for x in got)
    f = lambda x: None if x is None else x.detach().cpu().to(torch.float64).numpy()  # noqa: E731
    l, q, u, r, d = f(logits), f(probs), f(accept), f(sample), drafts.cpu().numpy()
    t = np.broadcast_to(np.asarray(f(temperature) if isinstance(temperature, torch.Tensor) else temperature, np.float64), len(l))
    far = 0
    for i in range(len(l)):
        n = d.shape[1] if lens is None else min(max(int(lens[i]), 0), d.shape[1])
        a, token, near = PO.verify(l[i], d[i], None if q is None else q[i], u[i], r[i], n, t[i])
        if near < NEAR:
            continue
        far += 1
        want = d[i, :a].tolist() + [token] + [-1] * (d.shape[1] - a)
        assert (accepted[i], tokens[i].tolist()) == (a, want), f"sequence {i}"
    assert far >= len(l) - 1
    return accepted


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,s,v", [(1, 1, 1), (1, 4, 32000), (7, 3, 2), (5, 2, 33), (3, 6, 50257), (2, 1, 128256), (16, 7, 1000),
                                   (4, 0, 513), (1, 2, 1 << 19), (300, 3, 511), (2, 40, 4097)])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify(dtype, b, s, v, sampled):
    x = made(b, s, v, dtype, b * 31 + s)
    if not sampled:
        x = (x[0], x[1], None, *x[3:])
    lens = [(s * (i + 1)) // b for i in range(b)]
    lens[0] = s
    agree(binding.verify_drafts(*x), *x)
    agree(binding.verify_drafts(*x, lens=ints(lens), temperature=0.6), *x, lens=lens, temperature=0.6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_of_flat_and_peaked_rows(dtype):
    """Every border of a flat distribution is as near as it gets; a peaked one has most weights below 2^-43."""
    for spread, apart, temperature in ((0.0, 0.0, 1.0), (0.01, 0.0, 1.0), (0.3, 0.1, 2.0), (30.0, 1.0, 1.0), (3.0, 0.5, 0.05)):
        x = made(24, 3, 70001, dtype, 5, spread, apart)
        agree(binding.verify_drafts(*x, temperature=temperature), *x, temperature=temperature)


def test_verify_accepts_as_often_as_the_distributions_overlap():
    """Speculative sampling's acceptance rate is sum min(p, q): 4096 drafts of one pair of distributions."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    v, b = 50, 4096
    l = torch.randn(v, generator=g, device="cuda")
    q = torch.softmax(l + torch.randn(v, generator=g, device="cuda"), -1)
    p = torch.softmax(l, -1)
    d = torch.multinomial(q, b, True, generator=g).to(torch.int32).view(b, 1)
    rnd = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    tokens, acc = binding.verify_drafts(l.expand(b, 2, v), d, q.expand(b, 1, v), rnd(b, 1), rnd(b))
    rate = float(torch.minimum(p, q).sum())
    assert abs(float(acc.float().mean()) - rate) <= 5 * (rate * (1 - rate) / b) ** 0.5
    # and the first token is distributed as p, whether it was drafted or sampled: 5 standard deviations of each count
    n = torch.bincount(tokens[:, 0].long(), minlength=v).float()
    assert bool(((n - b * p).abs() <= 5 * (b * p * (1 - p)).sqrt() + 1).all())


def test_verify_greedy_and_temperatures_per_sequence():
    x = made(6, 3, 777, "f32", 9)
    l, d = x[0], x[1]
    l[0, 0, 500] = l[0, 0, 20] = l[0, 0].max() + 1              # ties: the first
    d[:, 0] = l[:, 0].argmax(-1).to(torch.int32)
    d[0, 0] = 20
    t = torch.tensor([0.0, 0.0, 1.0, 0.3, 1e-31, float("nan")], device="cuda")
    want = torch.tensor([0, 0, 1, 0.3, 0, 0], dtype=torch.float32, device="cuda")
    got = binding.verify_drafts(*x, temperature=t)
    acc = agree(got, *x, temperature=want)
    assert acc[0] >= 1 and acc[1] >= 1
    d[0, 0] = 500
    assert int(binding.verify_drafts(*x, temperature=0)[1][0]) == 0


def test_verify_special_values():
    """Masked, infinite and NaN logits; drafts out of the vocabulary; numbers at and past the ends of [0, 1);
    distributions that leave nothing, or are no distributions."""
    inf, nan, v = float("inf"), float("nan"), 600
    l, d, q, u, r = made(14, 2, v, "f32", 11)
    l[0, :, 5:] = -inf                                   # few tokens left
    l[1] = -inf                                          # none
    l[2, 0] = nan
    l[3, 0, 7] = inf                                     # one has all the weight
    l[3, 0, 9] = nan
    d[3, 0] = 7
    d[4, 0], d[5, 1] = v, -1
    u[6], r[6] = 0.0, 0.0
    u[7], r[7] = nan, nan
    r[8], r[9] = 1.0, -1.0
    q[10] = torch.softmax(l[10, :2], -1)                 # p - q is nothing, or rounding: u of 1 rejects
    u[10] = 1.0
    q[11] = 2.0                                          # p - q below 0 everywhere: p itself
    u[11] = 0.99
    q[12, :, ::2] = -1.0
    l[13, 0] = 0.0                                       # all equal
    r[8] = 1.0
    got = binding.verify_drafts(l, d, q, u, r)
    tokens, acc = got
    assert tokens[1].tolist() == [-1, -1, -1] and tokens[2].tolist() == [-1, -1, -1] and acc[1] == 0 == acc[2]
    assert tokens[3, 0] == 7 and acc[4] == 0 and acc[5] <= 1 and acc[7] == 0 and acc[11] == 0
    assert acc[6] == 2 and int(tokens[6, 2]) == 0
    l[2, 0] = -inf
    r[7], r[9], u[7] = 0.0, 0.0, 2.0
    r[8] = 1.0 - 2.0 ** -24
    q[12] = q[12].clamp(min=0)
    rows = [0, 3, 4, 5, 6, 7, 8, 9, 11, 12, 13]
    pick = lambda x: x[rows]  # noqa: E731
    agree(tuple(pick(x) for x in got), *(pick(x) for x in (l, d, q, u, r)))


def test_verify_decides_near_borders():
    """Acceptance numbers a few fp32 steps to either side of p / q."""
    l, d, q, u, r = made(64, 1, 5000, "f32", 21)
    p = torch.softmax(l[:, 0].double(), -1).gather(1, d.long())
    edge = (p / q[:, 0].double().gather(1, d.long())).clamp(max=0.999)
    for steps in (-4, -1, 1, 4):
        u = (edge * (1 + steps * 2.0 ** -23)).float()
        agree(binding.verify_drafts(l, d, q, u, r), l, d, q, u, r)


def test_verify_strides_streams_outputs_and_graphs():
    l, d, q, u, r = made(5, 3, 1001, "bf16", 31)
    wide = torch.full((5, 4, 1003), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, :, 1:1002] = l
    view = wide[:, :, 1:1002]                            # rows of odd alignment
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)  # positions before sequences
    want = binding.verify_drafts(l, d, q, u, r)
    agree(want, l, d, q, u, r)
    tokens, acc = torch.full((5, 4), 99, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.verify_drafts(view, d, qt, u, r, tokens=tokens, accepted=acc, stream=side)
    side.synchronize()
    assert got[0] is tokens and got[1] is acc
    assert torch.equal(tokens, want[0]) and torch.equal(acc, want[1])
    one = binding.verify_drafts(l[:1, :1].expand(5, 4, 1001), d, None, u, r)       # one row for all
    agree(one, l[:1, :1].expand(5, 4, 1001), d, None, u, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.verify_drafts(l, d, q, u, r)
    u.copy_(1 - u)
    graph.replay()
    agree(out, l, d, q, u, r)


def test_verify_refusals():
    l, d, q, u, r = made(2, 2, 64, "f32", 41)
    bad = [(l.half(), d, q, u, r), (l, d.long(), q, u, r), (l, d, q.double(), u, r), (l, d, q[:, :1], u, r), (l, d, q, u[:, :1], r),
           (l, d, q, u, r[:1]), (l.transpose(1, 2), d, q, u, r), (l.cpu(), d, q, u, r), (l[:, :2], d, q, u, r), (l[:, :0], d, q, u, r)]
    for x in bad:
        with pytest.raises(ValueError):
            binding.verify_drafts(*x)
    with pytest.raises(ValueError):
        binding.verify_drafts(l, d, q, u, r, lens=ints([1]))
    for t in (-1.0, float("nan"), float("inf")):
        with pytest.raises(binding.ShadowKVError):
            binding.verify_drafts(l, d, q, u, r, temperature=t)
    x = made(1, 1, (1 << 19) + 1, "bf16", 1)
    with pytest.raises(binding.ShadowKVError, match="vocab"):
        binding.verify_drafts(*x)
    empty = made(0, 2, 64, "f32", 1)
    t, a = binding.verify_drafts(*empty)
    assert t.shape == (0, 3) and a.shape == (0,)


@pytest.mark.parametrize("sampled", [True, False])
def test_a_sample_of_one_or_more_is_the_largest_below(sampled):
    """A last token of weight e^-20, 2^-28.9: past 1 - 2^-24 of the total, where no number in [0, 1) falls."""
    l = torch.zeros(5, 2, 3, device="cuda")
    l[:, :, 0], l[:, :, 2] = -30.0, -20.0
    r = torch.tensor([1.0, 2.5, float("inf"), 1 - 2.0 ** -24, 0.0], device="cuda")
    d, u = ints([[0]] * 5), torch.full((5, 1), 0.5, device="cuda")
    q = torch.tensor([1.0, 0.0, 0.0], device="cuda").expand(5, 1, 3) if sampled else None
    tokens, acc = binding.verify_drafts(l, d, q, u, r)
    assert acc.tolist() == [0] * 5 and tokens[:, 0].tolist() == [1] * 5


@pytest.mark.parametrize("v", [5000, 1 << 17, 1 << 19])
@pytest.mark.parametrize("tail", [27.3, 28.0, 30.2, 30.6])
def test_verify_of_a_peak_over_a_flat_tail(v, tail):
    """Two likely tokens and v - 2 equal ones e^-tail as likely: weights of few units, or none, whose errors all have one
    sign.  A weight is off by 2^-37 of itself and by 2^-44, the total (at least 1) by 2^-37 of itself and v 2^-44: u q z < p
    is decided right where u q and p are farther apart than B = 2^-36 + v 2^-44 of them, and the sampled token's
    place is right to B of the total, twice (its own sum and the total)."""
    bound = 2.0 ** -36 + v * 2.0 ** -44
    b = 16
    l = torch.full((b, 2, v), -tail, device="cuda")
    at = 1234
    l[:, :, at] = l[:, :, at + 7] = 0.0
    z = 2 + (v - 2) * float(np.exp(-np.float64(np.float32(tail))))
    p = 1 / z
    # u q next to p, from both sides: products of two floats, whose last bits are as fine as 2^-48
    g = np.random.default_rng(7)
    uq = []
    while len(uq) < b:
        q = np.float32(g.uniform(0.6, 0.95))
        u = np.float32(p / float(q))
        if 1.01 * bound < abs(float(u) * float(q) - p) / p < 16 * bound:
            uq.append((u, q))
    u, q = torch.tensor([[x[0]] for x in uq], device="cuda"), torch.zeros(b, 1, v, device="cuda")
    q[:, 0, at] = torch.tensor([x[1] for x in uq], device="cuda")
    r = torch.tensor(1 - g.integers(1, 9, b) * 2.0 ** -24, dtype=torch.float32, device="cuda")
    r[::3] = torch.rand(len(r[::3]), device="cuda")
    d = torch.full((b, 1), at, dtype=torch.int32, device="cuda")
    want = [float(x) * float(y) < p for x, y in uq]
    tokens, acc = binding.verify_drafts(l, d, q, u, r)
    assert acc.tolist() == [int(x) for x in want] and 0 < sum(want) < b
    w = np.full(v, np.exp(-np.float64(np.float32(tail))))
    for i in range(b):
        rest = w.copy()
        rest[at] = rest[at + 7] = 1.0
        rest /= z
        if not want[i]:
            rest = np.maximum(rest - q[i, 0].double().cpu().numpy(), 0)
        cum = np.cumsum(rest)
        k, place = int(tokens[i, int(acc[i])]), float(r[i]) * cum[-1]
        assert (cum[k - 1] if k else 0.0) - 2 * bound <= place <= cum[k] + 2 * bound
