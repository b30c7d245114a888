"""The block cache's pool as one that sequences share, on the GPU: forks, room for
appends with copies of shared blocks, rollback and compaction, each against its
definition (whole numbers and copied bytes: equal), and a loop of them together."""
import numpy as np
import pytest
import torch

from oracle import pool_oracle as PO
from sparse_rank_kv_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def content(c):
    """What every pool block holds, as bytes and scales."""
    k, v = c.k_codes.view(torch.uint8).cpu().numpy(), c.v_codes.view(torch.uint8).cpu().numpy()
    ks, vs = c.k_scale.cpu().numpy().view(np.int32), c.v_scale.cpu().numpy().view(np.int32)
    return [(k[i].tobytes(), v[i].tobytes(), int(ks[i]), int(vs[i])) for i in range(len(ks))]


def model(c):
    return PO.Pool(c.table.cpu().numpy(), c.n_tok.cpu().numpy(), c.weight.cpu().numpy(), c.refs.cpu().numpy(), c.block, content(c))


def same(c, m):
    for name in ("table", "n_tok", "weight", "refs"):
        got, want = getattr(c, name).cpu().numpy(), getattr(m, name)
        assert np.array_equal(got, want), f"{name}: {np.argwhere(got != want)[:5].tolist()}"
    got = content(c)
    bad = [i for i in range(len(got)) if got[i] != m.content[i]]
    assert not bad, f"blocks {bad[:8]} differ"
    named = np.bincount(m.table[m.table >= 0].ravel(), minlength=len(m.refs))
    assert np.array_equal(named, m.refs), "references are not what the tables name"


def pooled(b, h, d, block, max_blocks, n_pool, lens, seed, per_head=False, fan=1):
    """A cache whose pool holds random bytes, its sequences `lens` tokens long (each head its own where
    per_head); groups of `fan` share the whole blocks of their shortest member's first half."""
    r = np.random.default_rng(seed)
    c = binding.BlockCache.pooled(b, h, d, max_blocks, n_pool, block=block)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.from_numpy(r.integers(0, 0x7e, t.shape, np.uint8)))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.from_numpy(2.0 ** r.integers(-9, 9, n_pool)).float())
    n = np.broadcast_to(np.array(lens)[:, None], (b, h)).copy()
    if per_head:
        n -= np.minimum(n, r.integers(0, 2 * block, (b, h)))
    table, free = np.full((b, h, max_blocks), -1), list(r.permutation(n_pool))
    for i, g in np.ndindex(b, h):
        first = i // fan * fan
        common = min(n[first:first + fan, g]) // (2 * block) if i != first else 0
        for e in range(-(-n[i, g] // block)):
            table[i, g, e] = table[first, g, e] if e < common else free.pop()
    c.table.copy_(torch.from_numpy(table))
    c.n_tok.copy_(torch.from_numpy(n))
    c.weight.copy_(torch.from_numpy(np.where(table >= 0, r.random(table.shape), 0)))
    c.refs.copy_(torch.from_numpy(np.bincount(table[table >= 0].ravel(), minlength=n_pool)))
    return c


SHAPES = [   # b, h, d, block, max_blocks, n_pool, lens, fan
    (1, 1, 64, 16, 1, 1, [0], 1), (1, 1, 64, 16, 4, 9, [33], 1), (4, 2, 64, 16, 9, 100, [17, 64, 0, 129], 1),
    (6, 3, 128, 32, 20, 333, [500, 300, 611, 64, 1, 32], 3), (3, 8, 128, 64, 5, 77, [100, 130, 1], 1),
    (40, 5, 64, 128, 7, 1500, [(37 * i) % 800 for i in range(40)], 4), (2, 2, 128, 16, 700, 9000, [11000, 5001], 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("per_head", [False, True])
def test_truncate(shape, per_head):
    b, h, d, block, mb, pool, lens, fan = shape
    c = pooled(b, h, d, block, mb, pool, lens, 1, per_head, fan)
    m = model(c)
    c.truncate()
    m.truncate()
    same(c, m)
    drop = [(0, 1, block, 2 * block + 3, 2**31 - 1)[(i + 1) % 5] for i in range(b)]
    c.truncate(ints(drop))
    m.truncate(drop)
    same(c, m)
    c.check()
    c.reset()
    assert int(c.refs.abs().sum()) == 0 and int(c.n_tok.sum()) == 0 and bool((c.table == -1).all())
    c.check()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_share_then_reserve(shape):
    """Forks, then room for appends of every length: none, one, to the block's end, past it, several blocks."""
    b, h, d, block, mb, pool, lens, fan = shape
    for s in (0, 1, block - lens[0] % block, block + 1, 5 * block + 2):
        c = pooled(b, h, d, block, mb, pool, lens, 2 + s, True, fan)
        m = model(c)
        r = np.random.default_rng(s)
        order = r.permutation(b)
        dst = order[:b // 2].tolist()
        src = [int(order[b // 2 + i % (b - b // 2)]) for i in range(len(dst))]
        c.share(ints(src), ints(dst))
        assert m.share(src, dst) == []
        same(c, m)
        n = [int(x) for x in r.integers(0, s + 1, b)]
        n[0] = s
        got = c.reserve(s, ints(n))
        want = m.reserve(n)
        assert np.array_equal(got.cpu().numpy(), want)
        same(c, m)
        # once more: only sequences left out may still get a block, for none of their tokens
        assert np.array_equal(c.reserve(s, got).cpu().numpy(), m.reserve(want))
        same(c, m)
        assert torch.equal(c.reserve(s, got), got)
        same(c, m)
        c.check()


def test_reserve_grants_whole_sequences_in_order():
    """A pool with too few blocks: sequences up to the first that does not fit, and those that need nothing."""
    for free in range(0, 14):
        c = pooled(5, 2, 64, 16, 6, 200, [16, 32, 40, 16, 8], 3)
        taken = [i for i in range(200) if int(c.refs[i]) == 0]
        hold = torch.zeros(200, dtype=torch.int32)
        hold[taken[free:]] = 1
        c.refs += hold.cuda()                              # blocks another owner holds
        m = model(c)
        lens = [20, 1, 3, 16, 40]                            # 2 x (2, 1, 0, 1, 2) blocks
        got, want = c.reserve(40, ints(lens)).cpu().numpy(), m.reserve(lens)
        assert np.array_equal(got, want), (free, got, want)
        assert want[2] == 3 and (want[0] > 0) == (free >= 4) and (want[4] > 0) == (free >= 12)
        assert np.array_equal(c.table.cpu().numpy(), m.table) and np.array_equal(c.refs.cpu().numpy(), m.refs)
        c.check()


def test_reserve_past_the_table_grants_nothing():
    c = pooled(2, 2, 64, 16, 3, 40, [40, 40], 4)
    m = model(c)
    assert c.reserve(9, ints([9, 8])).tolist() == [0, 8] == m.reserve([9, 8]).tolist()
    same(c, m)
    c.check()


def test_share_leaves_out_what_overlaps():
    c = pooled(5, 2, 64, 16, 4, 60, [20, 33, 64, 5, 17], 5)
    m = model(c)
    src, dst = [0, 1, 0, 4, 9], [1, 2, 2, -1, 3]
    c.share(ints(src), ints(dst))
    assert m.share(src, dst) == [0, 2, 3, 4]
    same(c, m)
    with pytest.raises(binding.ShadowKVError, match="sequence"):
        c.check()


def test_bad_entries_and_counts_are_recorded_and_touch_nothing():
    c = pooled(2, 1, 64, 16, 4, 20, [20, 20], 6)
    c.table[0, 0, 1] = 20                                   # the partly filled block's id is not one of the pool
    refs = c.refs.clone()
    assert c.reserve(3).tolist() == [0, 3]
    assert torch.equal(c.refs, refs)
    with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
        c.check()
    c = pooled(2, 1, 64, 16, 4, 20, [20, 20], 6)
    c.truncate(ints([-1, 0]))
    assert c.n_tok.tolist() == [[20], [20]]
    with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
        c.check()
    c = pooled(2, 1, 64, 16, 4, 20, [20, 20], 6)
    assert c.reserve(3, ints([7, -2])).tolist() == [3, 0]    # clamped
    with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
        c.check()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("room", [0, 5, -1])
def test_compact(shape, room):
    b, h, d, block, mb, pool, lens, fan = shape
    c = pooled(b, h, d, block, mb, pool, lens, 7, True, fan)
    m = model(c)
    live = m.compact()
    n = len(live) + room
    if n < 1:
        n = max(1, len(live))
    to = pooled(b, h, d, block, mb, n, [0] * b, 8)
    was = content(to)
    to.n_tok.fill_(5)
    c.compact(to)
    same(c, m)                                               # the source stays
    if n < len(live):
        assert int(to.n_tok.abs().sum()) == 0 and bool((to.table == -1).all()) and int(to.refs.sum()) == 0
        assert content(to) == was
        with pytest.raises(binding.ShadowKVError, match="pool"):
            to.check()
        return
    place = {old: new for new, old in enumerate(live)}
    table = np.vectorize(lambda x: place.get(x, -1))(m.table)
    assert np.array_equal(to.table.cpu().numpy(), table)
    assert np.array_equal(to.n_tok.cpu().numpy(), m.n_tok) and np.array_equal(to.weight.cpu().numpy(), m.weight)
    assert to.refs.tolist() == [int(m.refs[i]) for i in live] + [0] * (n - len(live))
    assert content(to) == [m.content[i] for i in live] + was[len(live):]
    c.check()
    to.check()


def test_large_pool():
    """More blocks than one walk of the cluster's warps takes, and a need of thousands."""
    c = pooled(1, 2, 64, 16, 16384, 300001, [9], 9)
    m = model(c)
    assert c.reserve(100000).tolist() == [100000] == m.reserve([100000]).tolist()
    same(c, m)
    c.check()


def test_append_and_attend_of_forks():
    """Two forks of a prompt that append tokens of their own: each reads what a cache of its own would hold, the
    parent's partly filled block is untouched, and evicted blocks go back with truncate()."""
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    b, h, d, block = 3, 2, 128, 16
    tok = lambda n: torch.randn(b, h, n, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    c = binding.BlockCache.pooled(b, h, d, 10, 60, block=block)
    own = binding.BlockCache.empty(b, h, d, 10, block=block)
    k, v = tok(40), tok(40)
    k, v = k[:1].expand(b, -1, -1, -1).contiguous(), v[:1].expand(b, -1, -1, -1).contiguous()
    lens = c.reserve(40, ints([40, 0, 0]))
    c.append(k, v, lens)
    c.share(ints([0, 0]), ints([1, 2]))
    own.append(k, v)
    assert int(c.refs.max()) == 3 and int((c.refs > 0).sum()) == 2 * 3
    for n in (1, 5, 20):
        k, v = tok(n), tok(n)
        c.append(k, v, c.reserve(n))
        own.append(k, v)
        q = torch.randn(b, 4, d, generator=g, device="cuda").bfloat16()
        assert torch.equal(c.attend(q, decay=0.5), own.attend(q, decay=0.5))
    m = model(c)
    same(c, m)
    c.evict(3, sink=1, recent=1)
    own.evict(3, sink=1, recent=1)
    c.truncate()
    assert int((c.refs > 0).sum()) <= 3 * 2 * 3
    q = torch.randn(b, 4, d, generator=g, device="cuda").bfloat16()
    assert torch.equal(c.attend(q), own.attend(q))
    same(c, model(c))
    small = binding.BlockCache.pooled(b, h, d, 10, 18, block=block)
    c.compact(small)
    assert torch.equal(small.attend(q), own.attend(q))
    c.check()
    small.check()


def test_calls_on_another_stream_and_captured():
    c = pooled(4, 2, 64, 16, 9, 100, [17, 64, 3, 100], 11)
    start = {n: getattr(c, n).clone() for n in ("table", "n_tok", "weight", "refs")}
    m = model(c)
    src, dst, lens, drop = ints([0]), ints([2]), ints([30, 1, 2, 17]), ints([1, 0, 0, 40])
    to = pooled(4, 2, 64, 16, 9, 100, [0] * 4, 12)

    def step(stream=None):
        c.truncate(drop, stream=stream)
        c.share(src, dst, stream=stream)
        got = c.reserve(30, lens, stream=stream)
        c.compact(to, stream=stream)
        return got

    m.truncate([1, 0, 0, 40])
    m.share([0], [2])
    want = m.reserve([30, 1, 2, 17])

    def check(got):
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), want)
        same(c, m)
        assert int((to.refs > 0).sum()) == int((c.refs > 0).sum())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(step(side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for n, t in start.items():
            getattr(c, n).copy_(t)
        graph.replay()
        check(got)
    c.check()


def test_refusals():
    c, plain = pooled(2, 1, 64, 16, 4, 20, [20, 20], 6), binding.BlockCache.empty(2, 1, 64, 4, block=16)
    for call in (lambda: plain.reserve(1), lambda: plain.share(ints([0]), ints([1])), lambda: plain.compact(c),
                 lambda: c.compact(plain), c.fork, lambda: c.evict(2, into=pooled(2, 1, 64, 16, 4, 20, [20, 20], 6)),
                 lambda: c.reserve(1, ints([1])), lambda: c.share(ints([0]), ints([1, 0])), lambda: c.truncate(ints([0])),
                 lambda: c.reserve(1, torch.ones(2, device="cuda")), lambda: c.share(ints([0]).cpu(), ints([1]))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.compact(c), lambda: c.share(ints([0, 1, 0]), ints([1, 0, 1])), lambda: c.reserve(-1),
                 lambda: c.compact(pooled(2, 1, 64, 16, 5, 20, [20, 20], 6))):
        with pytest.raises(binding.ShadowKVError):
            call()
    c.share(ints([]), ints([]))                              # nothing to do
    plain.append(torch.ones(2, 1, 20, 64, device="cuda"), torch.ones(2, 1, 20, 64, device="cuda"))
    table = plain.table.clone()
    plain.truncate(ints([3, 30]))                            # a cache of its own pool: counts and weights alone
    assert plain.n_tok.tolist() == [[17], [0]] and torch.equal(plain.table, table)
    plain.check()


def held(c, i):
    """Keys and values of sequence i in 64 bits, each (h, n, d), and the scale of each token's block (h, n, 1)."""
    n, out = int(c.n_tok[i, 0]), []
    ids = c.table[i, :, :-(-n // c.block)].long()
    for codes, scale, shape in ((c.k_codes, c.k_scale, (0, 1, 2, 4, 3, 5)), (c.v_codes, c.v_scale, (0, 1, 2, 4, 3))):
        x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double().permute(*shape)
        x = x.reshape(c.h_kv, -1, c.d)[:, :n]
        s = scale[ids].double().repeat_interleave(c.block, 1)[:, :n, None]
        out += [x * s, s]
    return out


def test_a_rejected_draft_leaves_no_more_than_its_scale():
    """A draft 2^12 times as large as the tokens beside it in a block, taken off again.  The scale stays: the smallest power
    of two with which 448 covers the draft; the other entries are off by half a step of e4m3 below its normal range, 2^-10
    of that scale, at most, and exact where the block was not touched.  Then the same with a fork before the
    drafts: every bit is as it was."""
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    h, d, block = 2, 128, 16
    tok = lambda n, up=1.0: (up * torch.randn(2, h, n, d, generator=g, device="cuda")).bfloat16()  # noqa: E731
    c = binding.BlockCache.pooled(2, h, d, 6, 30, block=block)
    only = lambda n: ints([n, 0])  # noqa: E731
    c.append(tok(21), tok(21), c.reserve(21, only(21)))
    c.weight[0, :, :2] = 0.5
    before = [x.clone() for x in held(c, 0)]
    k, v = tok(2, 4096.0), tok(2, 4096.0)
    start = {n: getattr(c, n).clone() for n in ("table", "n_tok", "weight", "refs", "k_codes", "v_codes", "k_scale", "v_scale")}

    c.append(k, v, c.reserve(2, only(2)))
    c.truncate(only(2))
    after = held(c, 0)
    for x, new, s_old, s_new, big in ((before[0], after[0], before[1], after[1], k), (before[2], after[2], before[3], after[3], v)):
        assert torch.equal(x[:, :block], new[:, :block]) and torch.equal(s_old[:, :block], s_new[:, :block])
        most = big[0].double().abs().amax((1, 2))[:, None, None]
        s = s_new[:, block:]
        assert bool((s > s_old[:, block:]).all()) and bool((most <= 448 * s).all()) and bool((most > 224 * s).all())
        err = (new[:, block:] - x[:, block:]).abs()
        assert bool((err <= 2.0 ** -10 * s).all()) and bool((err > 0).any())
    c.append(k * 0 + 1, v * 0 + 1, c.reserve(2, only(2)))          # later tokens are held by that scale
    assert bool((held(c, 0)[1][:, -1] == after[1][:, -1]).all())

    for n, t in start.items():
        getattr(c, n).copy_(t)
    there, back = ints([0]), ints([1])
    c.share(there, back)
    c.append(k, v, c.reserve(2, only(2)))
    c.share(back, there)                                           # the drafts are rejected
    c.truncate(ints([0, 21]))
    for x, y in zip(before, held(c, 0)):
        assert torch.equal(x, y)
    assert torch.equal(c.weight[0], start["weight"][0]) and c.n_tok.tolist() == [[21, 21], [0, 0]]
    same(c, model(c))
    c.check()


def test_reserve_may_write_what_it_grants_over_the_lengths():
    """granted is lens itself: what one of its own gets, sequences without room, past the table and clamped ones among them."""
    for n_pool in (20, 23, 80):
        lens = [20, 300, 3, 16, 40]
        got = []
        for own in (False, True):
            c = pooled(5, 2, 64, 16, 6, n_pool, [16, 32, 40, 16, 8], 3)
            x = ints(lens)
            got.append((c.reserve(200, x, granted=None if own else x).tolist(), c.table.tolist(), c.refs.tolist()))
            with pytest.raises(binding.ShadowKVError, match="DEVICE_CHECK"):
                c.check()
        assert got[0] == got[1]
        assert got[0][0][1] == 0 and got[0][0][2] == 3
