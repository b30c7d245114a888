"""The step of several tokens as the front page writes it, run: drafts of different lengths, sequences that get no
room, one that ends and makes room for others."""
import os
import re

import pytest
import torch

from sparse_rank_kv_gb300 import binding, build

pytestmark = pytest.mark.gpu
PAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.lib()


def the_step():
    """The cache and the step of its block on several tokens, as two pieces of code."""
    with open(PAGE) as f:
        blocks = re.findall(r"```(?:python)?\n(.*?)```", f.read(), flags=re.S)
    made, step = [x for x in blocks if "BlockCache.pooled" in x and "verify_drafts" in x][0].split("\n", 1)
    return compile(made, PAGE, "exec"), compile(step, PAGE, "exec")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_front_pages_step_keeps_what_stood():
    """After every step the cache holds what one that was only ever given the tokens that stood holds (values share
    a scale, so that rejected ones leave no trace), whatever the drafts' lengths and the room."""
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    b, h, G, d, v, s = 3, 2, 4, 64, 97, 5
    emb = (torch.randint(-6, 7, (2, v, h, d), generator=g, device="cuda") / 4).bfloat16()      # K and V of a token
    emb[:, :, :, 0] = 1.75                                             # every block's largest value
    qs = torch.randn(v, h * G, d, generator=g, device="cuda").bfloat16()
    out = 0.3 * torch.randn(h * G * d, v, generator=g, device="cuda")
    rows = lambda kind, t: emb[kind][t.long()].permute(0, 2, 1, 3).contiguous()       # noqa: E731 (b, s) -> b h s d
    made, step = the_step()
    env = dict(binding=binding, b=b, h_kv=h, d=d, max_blocks=8, n_pool=9, s=s)                  # 3 x 2 blocks of 64 at the start, and 3 more
    env["head"] = lambda x: x.transpose(1, 2).reshape(b, s + 1, -1).float() @ out
    exec(made, env)
    c, ref = env["cache"], binding.BlockCache.empty(b, h, d, 8)
    prompt = torch.randint(0, v, (b, 58), generator=g, device="cuda", dtype=torch.int32)
    c.append(rows(0, prompt), rows(1, prompt), c.reserve(58))
    ref.append(rows(0, prompt), rows(1, prompt))
    last = ints([5, 6, 7])
    seen = dict(none=0, short=0, again=0, stood=0)
    waiting = [False] * b
    for k in range(24):
        lens = torch.randint(1, s + 2, (b,), generator=g, device="cuda", dtype=torch.int32)
        if k >= 12:
            lens[0] = 0
        if k == 12:                                                    # the first sequence has ended
            end = ints([2**31 - 1, 0, 0])
            c.truncate(end)
            ref.truncate(end)
        drafts = torch.randint(0, v, (b, s), generator=g, device="cuda", dtype=torch.int32)
        t = torch.cat([last[:, None], drafts], 1)
        env.update(lens=lens, k=rows(0, t), v=rows(1, t), q=qs[t.long()].transpose(1, 2), drafts=drafts,
                   probs=torch.full((b, s, v), 1.0 / v, device="cuda"), u=torch.rand(b, s, generator=g, device="cuda"),
                   r=torch.rand(b, generator=g, device="cuda"))
        exec(step, env)
        room, tokens, stood = env["room"], env["tokens"], env["stood"]
        given = room > 0
        assert bool((stood <= (room - 1).clamp(min=0)).all())
        ref.append(env["k"], env["v"], torch.where(given, stood + 1, 0).to(torch.int32))
        assert torch.equal(c.n_tok, ref.n_tok), k
        q = qs[t[:, 0].long()].view(b, h * G, d)
        assert torch.equal(c.attend(q), ref.attend(q)), k
        last = torch.where(given, tokens.gather(1, stood[:, None].long())[:, 0], last).contiguous()
        for i in range(b):
            none = int(lens[i]) > 0 and int(room[i]) == 0
            seen["none"] += none
            seen["again"] += waiting[i] and int(room[i]) > 0
            waiting[i] = none
            seen["short"] += 0 < int(room[i]) <= s
        seen["stood"] += int(stood.sum())
    assert min(seen.values()) >= 1 and seen["none"] > 2, seen
    named = torch.bincount(c.table[c.table >= 0].long(), minlength=9)
    assert torch.equal(named.int(), c.refs)
    c.check()
    ref.check()
