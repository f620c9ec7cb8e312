"""page_table_update where a step does not fit: more new tokens than rows, a ring too small for what comes back,
page ids that are none. Every request is either served whole or left as it was, and no page is lost or owned
twice. Whole numbers, against one request after the other on the host."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host_step(table, lens, delta, ring, head, count, page, rows):
    """One request after the other (lists, updated): (lens, head, count, cu, positions, slots, fits)."""
    cap, taken, short, fits = len(ring), 0, False, True
    new, back, cu, pos, slots = [], [], [0], [], []
    gone = sum(max(-(-n // page) - -(-(n + x) // page), 0) for n, x in zip(lens, delta))
    room = count + gone <= cap
    for b, (n, x) in enumerate(zip(lens, delta)):
        held, want = -(-n // page), -(-(n + x) // page)
        ok = True
        if x > 0:
            ok = cu[-1] + x <= rows  # all of its rows, or none
            short = short or want - held > count - taken
            ok = ok and (want <= held or not short)
        elif want < held:
            ok = room
        if ok and want > held:
            for j in range(held, want):
                table[b][j] = ring[(head + taken) % cap]
                taken += 1
        elif ok and want < held:
            back += [table[b][j] for j in range(want, held)]
        for i in range(max(x, 0)):
            pos.append(n + i)
            slots.append(table[b][(n + i) // page] * page + (n + i) % page if ok else -1)
        cu.append(cu[-1] + max(x, 0))
        new.append(n + x if ok else n)
        fits = fits and ok
    for i, g in enumerate(back):
        ring[(head + count + i) % cap] = g
    pad = [-1] * (rows - len(pos))
    return new, (head + taken) % cap, count - taken + len(back), cu, (pos + pad)[:rows], (slots + pad)[:rows], fits


class Pool:
    """A pool on the host and on the device; `stale`: what a table entry holds that no request owns."""

    def __init__(self, B, width, page, n_pages, lens, cap=None, stale=None, seed=0):
        r = random.Random(seed)
        ids = list(range(n_pages))
        r.shuffle(ids)
        self.page, self.lens, self.n_pages = page, list(lens), n_pages
        self.table = [[ids[0] if stale is None else stale] * width for _ in range(B)]
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                self.table[b][j] = ids.pop()
        cap = n_pages if cap is None else cap
        self.ring, self.head = [-1] * cap, r.randrange(cap)
        free = ids[:cap]
        self.count = len(free)
        for i, g in enumerate(free):
            self.ring[(self.head + i) % cap] = g
        self.t, self.r, self.l, self.s = dev(self.table), dev(self.ring), dev(self.lens), dev([self.head, self.count])
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step(self, hs2, delta, rows):
        got = hs2.page_table_update(self.t, self.l, dev(delta), self.r, self.s, self.page, rows, lens_out=self.l,
                                    free_state_out=self.s, workspace=self.ws)
        status = hs2.read_device_status(self.ws)
        self.ws.zero_()
        *want, fits = host_step(self.table, self.lens, delta, self.ring, self.head, self.count, self.page, rows)
        self.lens, self.head, self.count = want[0], want[1], want[2]
        assert got[0].tolist() == want[0], "lengths"
        assert got[1].tolist() == want[1:3], "the ring's state"
        assert got[2].tolist() == want[3] and got[3].tolist() == want[4] and got[4].tolist() == want[5]
        assert self.t.tolist() == self.table and self.r.tolist() == self.ring
        assert status == (0 if fits else hs2.ERR_DEVICE_BOUNDS)
        return fits

    def owners(self):
        """Every page id held by a request or in the free list, from the device's own arrays."""
        t, l, ring, (head, count) = self.t.tolist(), self.l.tolist(), self.r.tolist(), self.s.tolist()
        held = [t[b][j] for b, n in enumerate(l) for j in range(-(-n // self.page))]
        return sorted(held + [ring[(head + i) % len(ring)] for i in range(count)])


@pytest.mark.parametrize("rows", [0, 1, 9, 10, 39, 40, 41, 63])
def test_a_request_past_the_rows_is_left_as_it_was(hs2, rows):
    """40 new tokens from a full page on: with fewer rows no page leaves the ring, and the length stays."""
    p = Pool(1, 8, 16, 9, [16])
    before = p.owners()
    assert p.step(hs2, [40], rows) == (rows >= 40)
    assert p.owners() == before == list(range(9))
    p.step(hs2, [-p.lens[0]], 0)  # what it holds comes back: every page has one owner
    assert p.count == 9 and p.owners() == list(range(9))


def test_the_others_are_served(hs2):
    """A request that starts before the last row and ends behind it, one that needs no page and lies behind, single
    tokens, cut-backs and requests that stand still."""
    p = Pool(7, 6, 16, 40, [10, 16, 30, 20, 33, 5, 0])
    before = p.owners()
    assert not p.step(hs2, [30, -3, 20, 3, -33, 0, 1], 49)
    assert p.lens == [40, 13, 30, 20, 0, 5, 0] and p.owners() == before
    assert p.step(hs2, [0, 0, 20, 3, 0, 0, 1], 24)
    assert p.lens == [40, 13, 50, 23, 0, 5, 1] and p.owners() == before


@pytest.mark.parametrize("B,page,most,seed", [(5, 16, 60, 0), (40, 48, 300, 1), (600, 16, 50, 2), (130, 128, 900, 3)])
def test_many_steps_keep_every_page(hs2, B, page, most, seed):
    """Steps whose rows, pages or ring do not suffice now and then (several blocks, one and many requests a thread),
    lengths and state updated in place."""
    r = random.Random(seed)
    width = -(-3 * most // page) + 1
    p = Pool(B, width, page, B * width // 3 + 2, [0] * B, seed=seed)
    before, some = p.owners(), 0
    for _ in range(12):
        d = [r.choice([0, 1, r.randrange(most + 1), -p.lens[b], -(p.lens[b] // 2)]) for b in range(B)]
        d = [min(x, width * page - p.lens[b]) for b, x in enumerate(d)]
        total = sum(max(x, 0) for x in d)
        some += not p.step(hs2, d, r.choice([total, total + 5, total // 2, max(total - 1, 0)]))
        assert p.owners() == before
    assert some > 2


def test_a_ring_too_small_for_what_comes_back(hs2):
    """Nothing is given back, and the requests that would have given pages keep their lengths; the others are served."""
    p = Pool(4, 5, 16, 20, [64, 40, 20, 16], cap=6)
    kept = p.owners()
    # (the ring of six is full)
    assert not p.step(hs2, [-64, -33, -2, 0], 0)
    assert p.lens == [64, 40, 18, 16] and p.owners() == kept
    assert not p.step(hs2, [-64, 0, 20, 1], 21)
    assert p.lens == [64, 40, 38, 17] and p.owners() == kept
    assert p.step(hs2, [0, -33, 0, 0], 0)  # (two fit now)
    assert p.lens == [64, 7, 38, 17] and p.owners() == kept


@pytest.mark.parametrize("state", [[-1, 2], [9, 2], [0, 10], [0, -1]])
def test_a_state_that_is_none(hs2, state):
    """A head or count outside the ring: no page is taken or given back, and no length changes that would."""
    p = Pool(4, 5, 16, 9, [16, 33, 20, 5])
    t, ring = p.t.clone(), p.r.clone()
    lo, so, _, _, slots = hs2.page_table_update(p.t, p.l, dev([20, -20, 3, -1]), p.r, dev(state), 16, 23, workspace=p.ws)
    assert hs2.read_device_status(p.ws) == hs2.ERR_DEVICE_BOUNDS
    assert lo.tolist() == [16, 33, 23, 4] and so.tolist() == state
    assert torch.equal(p.t, t) and torch.equal(p.r, ring)
    assert slots.tolist() == [-1] * 20 + [p.table[2][1] * 16 + 4 + i for i in range(3)]


def test_page_ids_that_are_none_are_recorded(hs2):
    """A negative id, or one whose slot passes 32 bits: in the table under a new token, at the ring's head, and in what is
    given back."""
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        for where in ("table", "ring"):
            p = Pool(2, 4, 16, 8, [10, 16])
            if where == "table":
                p.t[0, 0] = bad
            else:
                p.r[p.head] = bad
            _, _, _, pos, slots = hs2.page_table_update(p.t, p.l, dev([3, 2]), p.r, p.s, 16, 5, workspace=p.ws)
            assert hs2.read_device_status(p.ws) == hs2.ERR_DEVICE_BOUNDS, (bad, where)
            assert pos.tolist() == [10, 11, 12, 16, 17]
            good = slots[3:] if where == "table" else slots[:3]
            none = slots[:3] if where == "table" else slots[3:]
            assert int(good.min()) >= 0 and bool((none == -1).all())
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        p = Pool(2, 4, 16, 8, [40, 16])
        p.t[0, 1] = bad
        hs2.page_table_update(p.t, p.l, dev([-40, 0]), p.r, p.s, 16, 0, workspace=p.ws)
        assert hs2.read_device_status(p.ws) == hs2.ERR_DEVICE_BOUNDS, bad
    # a request that stands still, or one whose tokens lie elsewhere: its other entries are not read
    p = Pool(2, 4, 16, 8, [40, 16])
    p.t[0, 0] = -1
    hs2.page_table_update(p.t, p.l, dev([1, 0]), p.r, p.s, 16, 1, workspace=p.ws)
    assert hs2.read_device_status(p.ws) == 0
