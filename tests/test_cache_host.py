"""Host-side checks of the dense decode path's entry points: every refusal is
answered before any CUDA call (no pointer here is dereferenced), and the
oracle's quantisation agrees with worked values."""
import ctypes

import numpy as np
import pytest

from oracle import dense_oracle as D
from sparse_rank_kv_gb300 import binding, build

P = 0x100000     # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def desc(**kw):
    f = dict(b=2, h_kv=8, d=128, block=64, max_blocks=10, n_pool=160, k_codes=P, v_codes=P, k_scale=P, v_scale=P,
             table=P, n_tok=P, weight=P, status=P)
    f.update(kw)
    return binding.CacheDesc(**f)


def rows(ptr=P, sb=8192, sh=1024, ss=128):
    return binding.Rows(ptr, sb, sh, ss)


@pytest.mark.parametrize("change,code", [
    (dict(b=0), 1), (dict(h_kv=0), 1), (dict(max_blocks=0), 1), (dict(n_pool=0), 1), (dict(n_pool=-4), 1),
    (dict(k_codes=None), 1), (dict(v_codes=P + 8), 1), (dict(k_codes=P + 16), 1), (dict(k_scale=None), 1), (dict(table=P + 2), 1),
    (dict(n_tok=None), 1), (dict(status=None), 1), (dict(weight=P + 1), 1),
    (dict(d=96), 7), (dict(block=48), 7), (dict(block=256), 7), (dict(max_blocks=16385), 7),
    (dict(b=1 << 20, h_kv=64, max_blocks=64), 7),
])
def test_cache_descriptor_is_checked(lib, change, code):
    assert lib.shadowkv_cache_validate(desc(**change)) == code
    assert lib.shadowkv_last_error().decode()
    # every call that takes the cache checks it
    c = desc(**change)
    assert lib.shadowkv_cache_append(c, 1, rows(), rows(), 1, None, None) == code
    assert lib.shadowkv_cache_attend(c, 1, 32, rows(), 1.0, 0, 0.0, rows(), None, P, 1 << 30, None) == code
    assert lib.shadowkv_cache_evict(c, None, 4, 0, 1, None, None) == code
    assert lib.shadowkv_cache_check(c) == code
    assert lib.shadowkv_cache_attend_workspace(c, 32) == 0


def test_cache_descriptor_accepts(lib):
    assert lib.shadowkv_cache_validate(desc()) == 0
    assert lib.shadowkv_cache_validate(desc(weight=None)) == 0
    assert lib.shadowkv_cache_validate(None) == 1


@pytest.mark.parametrize("args,code", [
    (dict(dtype=2), 1), (dict(s=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=rows(None)), 1),
    (dict(k=rows(P + 8)), 1), (dict(v=rows(ss=132)), 1), (dict(v=rows(sb=-8)), 1), (dict(lens=P + 2), 1),
])
def test_append_refuses(lib, args, code):
    a = dict(dtype=1, k=rows(), v=rows(), s=3, lens=None)
    a.update(args)
    assert lib.shadowkv_cache_append(desc(), a["dtype"], a["k"], a["v"], a["s"], a["lens"], None) == code


def test_append_of_nothing_is_no_call(lib):
    assert lib.shadowkv_cache_append(desc(), 1, rows(), rows(), 0, None, None) == 0


@pytest.mark.parametrize("args,code", [
    (dict(dtype=7), 1), (dict(hq=12), 7), (dict(hq=24), 7), (dict(hq=128), 7), (dict(hq=0), 7), (dict(q=None), 1),
    (dict(out=rows(None)), 1), (dict(q=rows(P + 1)), 1), (dict(out=rows(sh=-128)), 1), (dict(out=rows(sh=0)), 1),
    (dict(lse=P + 2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(gather=2), 1),
    (dict(gather=1, decay=float("nan")), 1), (dict(gather=1, c=dict(weight=None)), 1), (dict(work=None), 1),
    (dict(work=P + 64), 1),
])
def test_attend_refuses(lib, args, code):
    a = dict(dtype=1, hq=32, q=rows(), scale=0.1, gather=0, decay=0.0, out=rows(), lse=None, work=P, c={})
    a.update(args)
    assert lib.shadowkv_cache_attend(desc(**a["c"]), a["dtype"], a["hq"], a["q"], a["scale"], a["gather"], a["decay"],
                                     a["out"], a["lse"], a["work"], 1 << 40, None) == code


@pytest.mark.parametrize("args", [
    dict(keep=0), dict(keep=11), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=2), dict(sink=2**31 - 1, recent=2**31 - 1),
    dict(kept=P + 2), dict(src=dict(weight=None)), dict(dst=dict(weight=None)), dict(dst=dict(b=1)),
    dict(dst=dict(block=32)), dict(dst=dict(max_blocks=9)),
])
def test_evict_refuses(lib, args):
    a = dict(keep=4, sink=0, recent=1, kept=None, src={}, dst=None)
    a.update(args)
    dst = None if a["dst"] is None else desc(**a["dst"])
    assert lib.shadowkv_cache_evict(desc(**a["src"]), dst, a["keep"], a["sink"], a["recent"], a["kept"], None) == 1


def nr(**kw):
    f = dict(b=1, s=2, h_q=4, h_kv=2, d=64, rot=64, dtype=1, norm=1, pos_per_token=0, eps=1e-6, theta=1e4)
    f.update(kw)
    return binding.NormRopeParams(**f)


@pytest.mark.parametrize("p,args,code", [
    (dict(b=-1), {}, 1), (dict(s=-1), {}, 1), (dict(h_q=0), {}, 1), (dict(h_kv=0), {}, 1), (dict(d=80), {}, 7),
    (dict(rot=72), {}, 1), (dict(rot=12), {}, 1), (dict(rot=-8), {}, 1), (dict(dtype=3), {}, 1), (dict(norm=2), {}, 1),
    (dict(pos_per_token=2), {}, 1), (dict(eps=0.0), {}, 1), (dict(eps=float("nan")), {}, 1), (dict(theta=0.0), {}, 1),
    (dict(theta=float("inf")), {}, 1), (dict(b=1 << 16, s=1 << 15), {}, 7), (dict(h_q=1 << 20), {}, 7),
    ({}, dict(q=None), 1), ({}, dict(q=None, k=None, q_out=None, k_out=None), 1), ({}, dict(k_out=None), 1),
    ({}, dict(q=None, q_out=None, qw=P), 1), ({}, dict(q=rows(P + 2)), 1), ({}, dict(k=rows(ss=66)), 1),
    ({}, dict(k_out=rows(sh=-64)), 1), ({}, dict(q_out=rows(ss=0)), 1), ({}, dict(kw=P + 2), 1), ({}, dict(pos=P + 1), 1),
    ({}, dict(q=rows(None)), 1),
])
def test_norm_rope_refuses(lib, p, args, code):
    a = dict(q=rows(), k=rows(), qw=None, kw=None, pos=None, q_out=rows(), k_out=rows())
    a.update(args)
    assert lib.shadowkv_qk_norm_rope(nr(**p), a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["q_out"], a["k_out"], None) == code
    assert lib.shadowkv_last_error().decode()


def test_norm_rope_of_nothing_is_no_call(lib):
    for p in (dict(b=0), dict(s=0)):
        assert lib.shadowkv_qk_norm_rope(nr(**p), rows(), rows(), None, None, None, rows(), rows(), None) == 0
    assert lib.shadowkv_qk_norm_rope(None, rows(), rows(), None, None, None, rows(), rows(), None) == 1


def test_packed_arguments_have_the_structures_layout():
    r = binding.Rows.from_buffer_copy(binding._PACK_ROWS(P, 1, 2, 3))
    assert (r.ptr, r.sb, r.sh, r.ss) == (P, 1, 2, 3) and ctypes.sizeof(binding.Rows) == 32
    n = binding.NormRopeParams.from_buffer_copy(binding._PACK_NORM_ROPE(1, 2, 3, 4, 5, 6, 7, True, False, 0.5, 2.0))
    got = [getattr(n, f) for f, _ in binding.NormRopeParams._fields_]
    assert got == [1, 2, 3, 4, 5, 6, 7, 1, 0, 0.5, 2.0]


def test_binding_refuses_wrong_tensors():
    import torch
    cpu = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.qk_norm_rope(cpu, None)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        binding.qk_norm_rope(cpu.half(), None)
    with pytest.raises(ValueError, match="both None"):
        binding.qk_norm_rope(None, None)
    with pytest.raises(ValueError, match="contiguous"):
        binding.qk_norm_rope(torch.zeros(1, 2, 3, 128)[..., ::2], None)
    with pytest.raises(ValueError, match="pos"):
        binding.qk_norm_rope(cpu, None, pos=torch.zeros(1, dtype=torch.int64))
    c = binding.BlockCache.empty(1, 2, 64, 3, block=16, device="cpu")   # names the tensors, runs nothing
    assert (c.b, c.h_kv, c.d, c.block, c.max_blocks) == (1, 2, 64, 16, 3)
    with pytest.raises(ValueError, match="CUDA"):
        c.append(cpu, cpu)
    with pytest.raises(ValueError, match="shape"):
        c.append(cpu[:, :1], cpu)
    with pytest.raises(ValueError, match="expected"):
        c.append(cpu, cpu.bfloat16())
    with pytest.raises(ValueError, match="lens"):
        c.append(cpu, cpu, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="kept"):
        c.evict(2, kept=torch.zeros(1, 2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="8-bit"):
        binding.BlockCache(torch.zeros(6, 2, 4, 8, 16), c.v_codes, c.k_scale, c.v_scale, c.table, c.n_tok)
    with pytest.raises(ValueError, match="table"):
        binding.BlockCache(c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.table.long(), c.n_tok)
    with pytest.raises(binding.ShadowKVError):
        binding.BlockCache.empty(1, 2, 64, 3, block=48, device="cpu")


def test_oracle_e4m3_matches_every_code():
    """The oracle's rounding against the format's definition: every finite code's value
    is kept, midpoints go to the even neighbour, values above 448 saturate."""
    vals = []
    for c in range(127):
        e, m = c >> 3, c & 7
        vals.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    vals = np.array(vals)
    assert vals[-1] == 448.0
    assert np.array_equal(D.e4m3(vals), vals) and np.array_equal(D.e4m3(-vals), -vals)
    mid = (vals[1:] + vals[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(D.e4m3(mid), even)
    assert D.e4m3(1e6) == 448.0


def test_oracle_scale_is_the_smallest_power_of_two():
    assert D.block_scale([448.0]) == 1.0
    assert D.block_scale([448.0001]) == 2.0
    assert D.block_scale([1.0, -3.5, np.inf, np.nan]) == 2.0 ** -7
    assert D.block_scale([0.0]) == 2.0 ** -100


def test_oracle_eviction_by_hand():
    # 5 blocks of 16, 70 tokens: the first and last stay, then the largest; ties to the lower index
    assert D.evict([0, 3, 5, 3, 9], 70, 16, 3, 1, 1) == ([0, 2, 4], 2 * 16 + 6)
    assert D.evict([0, 3, 3, 3, 9], 70, 16, 3, 1, 1) == ([0, 1, 4], 2 * 16 + 6)
    assert D.evict([0, 3, 5, 3, 1], 70, 16, 2, 0, 0) == ([1, 2], 32)
    assert D.evict([0, float("nan"), float("-inf"), 3, 1], 70, 16, 4, 0, 0) == ([0, 2, 3, 4], 3 * 16 + 6)
    assert D.evict([1, 1], 20, 16, 2, 0, 1) == ([0, 1], 20)


def test_cache_tensors_cannot_be_exchanged():
    """The calls hold the tensors' addresses: another tensor under the attribute would leave them
    on memory that nobody owns. In-place changes are the cache's own."""
    c = binding.BlockCache.empty(1, 2, 64, 3, block=16, device="cpu")
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "table", "n_tok", "weight", "status"):
        t = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, t.clone())
        assert getattr(c, name) is t
    c.weight += 1
    c.table[0, 0] = c.table[0, 0].flip(0)
    assert c.weight.sum() == 6 and c.fork().table is not c.table
    bare = binding.BlockCache(c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.table, c.n_tok)
    with pytest.raises(AttributeError, match="weight"):
        bare.weight = c.weight


def test_torch_short_cuts_have_public_stand_ins():
    import torch
    assert binding._torch_fn("_no_such_function", torch.cuda.current_device) is torch.cuda.current_device
    for f in (binding._current_device, binding._current_stream, binding._capturing):
        assert callable(f)
