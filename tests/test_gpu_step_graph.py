"""Page tables, rotation and attention of many decode steps in one captured graph, replayed without a wait: every
kernel starts while the one before it, whose results it reads, still runs. The same steps call by call, each waited
for, have to give the same bits."""
import random

import pytest
import torch

from plain64 import gen, randn

pytestmark = pytest.mark.gpu
STEPS, REPLAYS = 10, 4


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


class Step:
    """The buffers of a serving loop over one pool."""

    def __init__(self, hs2, B, Hq, Hk, d, page, f8, long):
        g, r = gen(7), random.Random(3)
        lens = [r.choice([0, page - 1, page, 3 * page + 2, r.randrange(long)]) for _ in range(B)]
        width = -(-(long + STEPS * REPLAYS + 5) // page)
        n = B * width
        table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        at = 0
        for b, m in enumerate(-(-x // page) for x in lens):
            table[b, :m] = perm[at:at + m]
            at += m
        ring = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        ring[:n - at] = perm[at:]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        pool = (lambda: (torch.randn(n, page, Hk, d, generator=g, device="cuda") * 16).to(torch.float8_e4m3fn).view(torch.uint8)) \
            if f8 else (lambda: randn(g, n, page, Hk, d))
        self.hs2, self.B, self.page, self.shape = hs2, B, page, (Hq, Hk, d)
        self.state = dict(table=table, lens=i32(lens), ring=ring, free=i32([0, n - at]), k=pool(), v=pool())
        self.delta = i32([1] * B)
        self.qkv = [randn(g, B, Hq + 2 * Hk, d) for _ in range(STEPS)]
        self.freq, _ = hs2.rope_frequencies(d)
        self.w = [1 + randn(g, d, dtype=torch.float32, std=0.2) for _ in range(2)]
        self.scales = dict(k_scale=2.0 ** -4, v_scale=0.07) if f8 else {}
        nbytes = hs2.paged_attn_workspace_bytes(B, Hq, Hk, d)
        self.ws = [torch.zeros(x, dtype=torch.uint8, device="cuda") for x in (256, 256, nbytes)]

    def run(self, s, step, wait):
        h, (Hq, Hk, d) = self.hs2, self.shape
        pause = torch.cuda.synchronize if wait else (lambda: None)
        _, _, _, pos, slots = h.page_table_update(s["table"], s["lens"], self.delta, s["ring"], s["free"], self.page, self.B,
                                                  lens_out=s["lens"], free_state_out=s["free"], workspace=self.ws[0])
        pause()
        q, k, v = self.qkv[step].split([Hq, Hk, Hk], 1)
        yq = h.qk_norm_rope_paged(q, k, v, pos, slots, s["k"], s["v"], self.freq, q_weight=self.w[0], k_weight=self.w[1],
                                  workspace=self.ws[1], **self.scales)
        pause()
        out, lse = h.paged_attn(yq[:, None], s["k"], s["v"], s["table"], s["lens"], workspace=self.ws[2], **self.scales)
        pause()
        return pos, slots, yq, out, lse


@pytest.mark.parametrize("B,Hq,Hk,d,page,f8,long", [(8, 64, 1, 128, 128, False, 3000), (3, 8, 2, 64, 16, False, 200), (40, 16, 8, 128, 16, False, 900),
                                                    (5, 64, 1, 128, 32, True, 20000), (33, 6, 2, 128, 16, True, 100), (300, 4, 1, 64, 16, False, 60)])
def test_captured_steps_replayed_without_waits(hs2, B, Hq, Hk, d, page, f8, long):
    loop = Step(hs2, B, Hq, Hk, d, page, f8, long)
    mine = {k: v.clone() for k, v in loop.state.items()}
    want = [loop.run(mine, i % STEPS, True) for i in range(STEPS * REPLAYS)][-STEPS:]
    assert all(hs2.read_device_status(w) == 0 for w in loop.ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [loop.run(loop.state, i, False) for i in range(STEPS)]
    for _ in range(REPLAYS):
        graph.replay()
    torch.cuda.synchronize()
    assert all(hs2.read_device_status(w) == 0 for w in loop.ws)
    for k in mine:
        assert torch.equal(mine[k], loop.state[k]), k
    for i, (a, b) in enumerate(zip(want, got)):
        for x, y, name in zip(a, b, ("positions", "slots", "q", "out", "lse")):
            assert torch.equal(x, y), (i, name)
    assert not bool(want[-1][3].isnan().any())
