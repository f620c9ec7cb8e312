"""page_table_update against one request after the other on the host (whole numbers: equal)."""
import random

import pytest
import torch

import plain64 as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """A pool's page table, lengths and free ring on the host, and the same on the device."""

    def __init__(self, B, width, page, n_pages, lens, seed=0):
        r = random.Random(seed)
        ids = list(range(n_pages))
        r.shuffle(ids)
        self.page, self.lens = page, list(lens)
        self.table = [[-1] * width for _ in range(B)]
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                self.table[b][j] = ids.pop()
        self.head, self.count = r.randrange(n_pages), len(ids)
        self.ring = [-1] * n_pages
        for i, g in enumerate(ids):
            self.ring[(self.head + i) % n_pages] = g
        self.t, self.r, self.l, self.s = dev(self.table), dev(self.ring), dev(self.lens), dev([self.head, self.count])

    def step(self, hs2, delta, max_tokens, **kw):
        got = hs2.page_table_update(self.t, self.l, dev(delta), self.r, self.s, self.page, max_tokens, lens_out=self.l,
                                    free_state_out=self.s, **kw)
        new, h, c, cu, pos, slots = P.page_table_step(self.table, self.lens, delta, self.ring, self.head, self.count, self.page,
                                                      max_tokens)
        self.lens, self.head, self.count = new, h, c
        assert got[0].tolist() == new and got[1].tolist() == [h, c] and got[2].tolist() == cu
        assert got[3].tolist() == pos and got[4].tolist() == slots
        assert self.t.tolist() == self.table and self.r.tolist() == self.ring


@pytest.mark.parametrize("B,page,most,seed", [(1, 16, 40, 0), (3, 1, 9, 1), (33, 128, 3000, 2), (512, 16, 60, 3),
                                              (513, 48, 200, 4), (4096, 16, 5, 5), (300, 64, 1500, 6)])
def test_steps_of_mixed_requests(hs2, B, page, most, seed):
    """Several steps in place: requests grow by nothing, one token and chunks, are cut back, end and begin again."""
    r = random.Random(seed)
    width = -(-4 * most // page) + 1
    p = Pool(B, width, page, B * width + 3, [r.randrange(most + 1) for _ in range(B)], seed)
    for step in range(5):
        d = [r.choice([0, 1, 1, r.randrange(most + 1), -p.lens[b], -(p.lens[b] // 2)]) for b in range(B)]
        d = [min(x, width * page - p.lens[b]) for b, x in enumerate(d)]
        p.step(hs2, d, sum(max(x, 0) for x in d) + step)
    assert hs2.read_device_status(hs2.cached_workspace("page_table")) == 0


def test_borders(hs2):
    """A page filled to its last row, one row more, the whole table, and nothing at all."""
    p = Pool(4, 4, 16, 16, [15, 16, 0, 64])
    p.step(hs2, [1, 1, 64, 0], 66)
    p.step(hs2, [-16, -1, -64, -64], 0)
    p.step(hs2, [0, 0, 0, 0], 3)


def test_outputs_apart_and_no_tokens(hs2):
    p = Pool(2, 4, 16, 8, [20, 3])
    lens, delta = p.l.clone(), dev([5, 0])
    lo, so, cu, pos, slots = hs2.page_table_update(p.t, p.l, delta, p.r, p.s, 16, 5)
    assert torch.equal(p.l, lens) and lo.tolist() == [25, 3] and so.tolist() == [p.head, p.count]
    assert cu.tolist() == [0, 5, 5] and pos.tolist() == [20, 21, 22, 23, 24]
    assert slots.tolist() == [p.table[0][1] * 16 + 4 + i for i in range(5)]
    lo, _, cu, pos, slots = hs2.page_table_update(p.t, p.l, dev([0, 0]), p.r, p.s, 16, 0)
    assert lo.tolist() == [20, 3] and cu.tolist() == [0, 0, 0] and pos.numel() == 0


def test_free_list_runs_out(hs2):
    """Requests are served in order while pages last (none overtakes one that is not); the others keep their
    length, their rows have no slot; one that needs no page is served."""
    p = Pool(4, 8, 16, 8, [16, 16, 16, 16])  # four pages are left
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    p.step(hs2, [32, 48, 16, -1], 96, workspace=ws)
    assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
    assert p.lens == [48, 16, 16, 15]


def test_bad_numbers_are_recorded(hs2):
    """A length or an end outside the table: the request stays as it is, the others are served."""
    p = Pool(5, 4, 16, 20, [10, 10, 10, 10, 10])
    bad = p.l.clone()
    bad[1], bad[2] = -3, 65
    before = p.t.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lo, so, cu, pos, slots = hs2.page_table_update(p.t, bad, dev([10, 5, 5, -11, 55]), p.r, p.s, 16, 75, workspace=ws)
    assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
    assert lo.tolist() == [20, -3, 65, 10, 10] and cu.tolist() == [0, 10, 15, 20, 20, 75]
    assert slots[:10].min() >= 0 and bool((slots[10:] == -1).all())
    assert torch.equal(p.t[1:], before[1:])
    # more new tokens than rows: what lies past them is not written
    ws.zero_()
    p = Pool(2, 4, 16, 20, [10, 10])
    full = torch.full((9,), 77, dtype=torch.int32, device="cuda")
    _, _, cu, pos, slots = hs2.page_table_update(p.t, p.l, dev([4, 4]), p.r, p.s, 16, 6, positions=full[:6].clone(), workspace=ws)
    assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
    assert cu.tolist() == [0, 4, 8] and pos.tolist() == [10, 11, 12, 13, 10, 11]
    # a ring that is too small for the pages given back: none is
    ws.zero_()
    p = Pool(2, 4, 16, 8, [64, 64])
    small = p.r[:3].clone()
    _, so, *_ = hs2.page_table_update(p.t, p.l, dev([-64, 0]), small, dev([0, 0]), 16, 0, workspace=ws)
    assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS and so.tolist() == [0, 0]
    for state in ([-1, 2], [8, 2], [0, 9], [0, -1]):
        ws.zero_()
        p = Pool(1, 4, 16, 8, [10])
        lo, so, *_ = hs2.page_table_update(p.t, p.l, dev([20]), p.r, dev(state), 16, 20, workspace=ws)
        assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
        assert lo.tolist() == [10] and so.tolist() == state


def test_captured_steps_in_place(hs2):
    """One captured step (several blocks: the last to read the lengths writes them) replayed many times."""
    p = Pool(64, 60, 16, 64 * 60, [0] * 64)
    delta = dev([40] * 64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = hs2.page_table_update(p.t, p.l, delta, p.r, p.s, 16, 2560, lens_out=p.l, free_state_out=p.s, workspace=ws)
    for i in range(20):
        gr.replay()
        torch.cuda.synchronize()
        new, p.head, p.count, cu, pos, slots = P.page_table_step(p.table, p.lens, [40] * 64, p.ring, p.head, p.count, 16, 2560)
        p.lens = new
        assert p.l.tolist() == new and out[3].tolist() == pos and out[4].tolist() == slots
    assert hs2.read_device_status(ws) == 0 and p.t.tolist() == p.table
