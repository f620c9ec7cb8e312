"""paged_attn against softmax attention in 64 bits (plain64), over pools whose unused rows hold NaN."""
import math

import pytest
import torch

import plain64 as P
from plain64 import gen, near, randn

pytestmark = pytest.mark.gpu
NAN8 = 0x7F  # an e4m3 NaN


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


class Cache:
    """Random sequences in a pool of shuffled pages; every row that no sequence uses is NaN, every table
    entry that none needs is out of range."""

    def __init__(self, lens, Hq, Hk, d, page, f8=False, layout="plain", seed=1, qstd=1.5, first=0, width=None):
        g = gen(seed)
        self.lens, self.page, self.Hk, self.d, self.f8 = lens, page, Hk, d, f8
        B, need = len(lens), [-(-n // page) for n in lens]
        n = sum(need) + 3
        new = (lambda *s: torch.full(s, NAN8, dtype=torch.uint8, device="cuda")) if f8 else \
            (lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda"))
        if layout == "joined":
            x = new(n, 2, page, Hk, d)
            self.k, self.v = x[:, 0], x[:, 1]
        elif layout == "heads first":
            self.k, self.v = (new(n, Hk, page, d).transpose(1, 2) for _ in range(2))
        else:
            self.k, self.v = new(n, page, Hk, d), new(n, page, Hk, d)
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((B, width or max(need + [1]) + 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
            rows = torch.arange(lens[b], device="cuda")
            pg, r = self.table[b, rows // page].long(), rows % page
            for pool, std in ((self.k, 1.0), (self.v, 1.0)):
                x = torch.randn(lens[b], Hk, d, generator=g, device="cuda") * std
                pool[pg, r] = (x * 16).to(torch.float8_e4m3fn).view(torch.uint8) if f8 else x.to(torch.bfloat16)
        self.q = randn(g, B, 1, Hq, d, std=qstd)
        self.l = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.scales = dict(k_scale=2.0 ** -4, v_scale=0.07) if f8 else {}

    def run(self, hs2, **kw):
        return hs2.paged_attn(self.q, self.k, self.v, self.table, self.l, **self.scales, **kw)

    def check(self, got, window=0, scale=None):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        out, lse, bo, bl = P.paged_attn(self.q, self.k, self.v, self.table, self.lens, scale, window,
                                        self.scales.get("k_scale"), self.scales.get("v_scale"))
        near(got[0], out, bo, "out")
        near(got[1], lse, bl, "lse")


SHAPES = [(1, 1, 64, 16, False), (64, 1, 128, 128, False), (8, 2, 128, 16, False), (33, 1, 64, 48, False), (12, 4, 64, 32, False),
          (16, 16, 128, 64, False), (17, 1, 128, 112, False), (64, 1, 128, 128, True), (1, 1, 128, 16, True), (21, 3, 128, 48, True),
          (16, 8, 128, 32, True)]


@pytest.mark.parametrize("window", [0, 1, 100, 130])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [63, 64, 65, 127, 128, 129], [1000, 1, 0, 2049, 300]], ids=str)
@pytest.mark.parametrize("Hq,Hk,d,page,f8", SHAPES)
def test_lengths_pages_and_windows(hs2, Hq, Hk, d, page, f8, lens, window):
    c = Cache(lens, Hq, Hk, d, page, f8)
    got = c.run(hs2, window=window)
    c.check(got, window)
    again = c.run(hs2, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert hs2.read_device_status(hs2.cached_workspace("paged_attn")) == 0


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("layout", ["joined", "heads first"])
def test_pool_strides(hs2, layout, f8):
    c = Cache([300, 7, 161], 12, 3, 128, 32, f8, layout)
    c.check(c.run(hs2))
    if not f8:
        c = Cache([300, 7, 161], 12, 3, 64, 32, f8, layout)
        c.check(c.run(hs2, window=77), 77)


@pytest.mark.parametrize("f8", [False, True])
def test_pool_without_a_head_dimension(hs2, f8):
    c = Cache([140, 33], 16, 1, 128, 16, f8)
    got = hs2.paged_attn(c.q, c.k[:, :, 0], c.v[:, :, 0], c.table, c.l, **c.scales)
    c.check(got)


@pytest.mark.parametrize("B,n,Hq,Hk,f8", [(1, 40000, 64, 1, False), (2, 70001, 8, 1, True), (200, 300, 16, 2, False),
                                          (1025, 40, 4, 4, True), (150, 200, 4, 1, False), (280, 100, 3, 1, True)])
def test_long_and_many(hs2, B, n, Hq, Hk, f8):
    """Pairs cut into many ranges, many pairs in one range, more sequences than threads, and a block a pair."""
    c = Cache([n - (37 * b) % n for b in range(B)], Hq, Hk, 128, 64, f8)
    c.check(c.run(hs2))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("boost", [8.0, 40.0])
def test_one_key_outweighs_the_rest(hs2, boost, f8):
    """A key whose score lies far above the others, and values that make the others count: each tile is
    rounded relative to its own maximum."""
    c = Cache([5000], 4, 1, 128, 128, f8, qstd=0.3)
    q = c.q[0, 0, 0].float()
    row = q / q.norm() * boost
    pg, r = int(c.table[0, 2345 // 128]), 2345 % 128
    if f8:
        c.k[pg, r, 0] = (row * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c.v[pg, r, 0] = 0
    else:
        c.k[pg, r, 0] = row.to(torch.bfloat16)
        c.v[pg, r, 0] = 0
    c.check(c.run(hs2, scale=1.0), scale=1.0)


def test_infinities_and_nan(hs2):
    """Infinite and NaN keys and values inside a sequence change the rows that the formula says, and outside its
    window none."""
    for f8 in (False, True):
        c = Cache([200, 90], 3, 1, 128, 16, f8)
        pg = int(c.table[0, 1])
        bad = NAN8 if f8 else float("nan")
        c.k[pg, 3], c.v[pg, 5] = bad, bad  # tokens 19 and 21 of the first sequence
        c.check(c.run(hs2, window=100), 100)
        out, lse = c.run(hs2)
        assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all()) and not bool(out[1].isnan().any())
    c = Cache([200], 2, 1, 64, 16)
    c.v[int(c.table[0, 0]), 0, 0, 7] = float("inf")
    out, lse = c.run(hs2)
    assert bool(torch.isinf(out[0, 0, :, 7]).all()) and bool(torch.isfinite(lse).all())
    assert bool(torch.isfinite(out[0, 0, :, :7]).all()) and bool(torch.isfinite(out[0, 0, :, 8:]).all())


@pytest.mark.parametrize("Hq,Hk,d,page", [(1, 1, 128, 16), (3, 3, 64, 48), (64, 1, 128, 128), (16, 2, 64, 16)])
def test_few_keys_keep_their_weights(hs2, Hq, Hk, d, page):
    """Short sequences and windows hold probabilities in two bf16 terms: one cut off (2^-7), the rest rounded by half a
    step of its own (2^-8 of it), 2^-15 together."""
    c = Cache([2, 3, 7, 64, 65, 256, 1], Hq, Hk, d, page)
    for window in (0, 2, 5):
        out, lse = c.run(hs2, window=window)
        want = P.paged_attn(c.q, c.k, c.v, c.table, c.lens, 1 / math.sqrt(d), window, p_round=2.0 ** -15)
        near(out, want[0], want[2], "out")
    c = Cache([2000, 900], Hq, Hk, d, page)  # (few of many keys are visible)
    out, _ = c.run(hs2, window=130)
    want = P.paged_attn(c.q, c.k, c.v, c.table, c.lens, 1 / math.sqrt(d), 130, p_round=2.0 ** -15)
    near(out, want[0], want[2], "out")


@pytest.mark.parametrize("f8", [False, True])
def test_query_magnitudes(hs2, f8):
    """Query rows of zeros, of tiny, of large and of one large element among tiny ones."""
    c = Cache([333], 4, 1, 128, 64, f8)
    c.q[0, 0, 0] = 0
    c.q[0, 0, 1] *= 2.0 ** -60
    c.q[0, 0, 2] *= 16
    c.q[0, 0, 3] *= 2.0 ** -9
    c.q[0, 0, 3, 77] = 9.0
    c.check(c.run(hs2))


def test_bad_pages_and_lengths_are_recorded(hs2):
    """An id outside the pool: its rows read as zero. A length outside the table counts as none."""
    for f8 in (False, True):
        c = Cache([100, 64, 30], 4, 2, 128, 16, f8)
        ws = torch.zeros(hs2.paged_attn_workspace_bytes(3, 4, 2, 128), dtype=torch.uint8, device="cuda")
        good = c.run(hs2, workspace=ws)
        assert hs2.read_device_status(ws) == 0
        k, v, table = c.k, c.v, c.table.clone()
        for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
            c.table[1, 2] = bad
            got = c.run(hs2, workspace=ws)
            assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
            assert torch.equal(got[0][0], good[0][0]) and torch.equal(got[0][2], good[0][2])
            c.table[1, 2] = table[1, 2]
            old = k[table[1, 2]].clone(), v[table[1, 2]].clone()
            k[table[1, 2]], v[table[1, 2]] = 0, 0
            c.check(got)
            k[table[1, 2]], v[table[1, 2]] = old
            ws.zero_()
        for n in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1):
            c.l[1] = n
            got = c.run(hs2, workspace=ws)
            assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
            assert not bool(got[0][1].any()) and bool((got[1][1] == -math.inf).all())
            assert torch.equal(got[0][0], good[0][0]) and torch.equal(got[0][2], good[0][2])
            ws.zero_()


@pytest.mark.parametrize("f8", [False, True])
def test_pages_before_the_window_may_be_gone(hs2, f8):
    """Table entries of pages that lie wholly before the window are not read."""
    c = Cache([700, 129, 40], 8, 2, 128, 16, f8)
    c.table[0, :(700 - 150) // 16] = -1
    c.check(c.run(hs2, window=150), 150)
    assert hs2.read_device_status(hs2.cached_workspace("paged_attn")) == 0


def test_without_logsumexp(hs2):
    """The C entry takes lse NULL."""
    import ctypes
    for lens in ([700, 0, 5], [30000, 0, 5]):
        c = Cache(lens, 6, 2, 64, 16)
        want = c.run(hs2)[0]
        out = torch.empty_like(want)
        ws = torch.zeros(hs2.paged_attn_workspace_bytes(3, 6, 2, 64), dtype=torch.uint8, device="cuda")
        st = (ctypes.c_longlong * 3)(*c.k.stride()[:3])
        code = hs2.lib.hs2_paged_attn(c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), st, st, c.k.shape[0], 16,
                                      c.table.data_ptr(), c.table.shape[1], c.l.data_ptr(), 3, 6, 2, 64, 0, 1.0, 1.0,
                                      1 / math.sqrt(64), 0, out.data_ptr(), None, ws.data_ptr(), ws.nbytes,
                                      torch.cuda.current_stream().cuda_stream)
        assert code == hs2.OK and hs2.read_device_status(ws) == 0
        assert torch.equal(out, want)


def test_offsets_past_32_bits(hs2):
    """Pages whose rows start beyond 2^31 elements of the pool."""
    n, page, d = 140000, 128, 128
    assert n * page * d > 2 ** 31
    k = torch.empty(n, page, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(n, page, 1, d, dtype=torch.bfloat16, device="cuda")
    c = Cache([300], 8, 1, d, page)
    far = torch.tensor([n - 1, 5, n - 7], device="cuda")
    k[far], v[far] = c.k[c.table[0, :3].long()], c.v[c.table[0, :3].long()]
    c.k, c.v = k, v
    c.table[0, :3] = far.to(torch.int32)
    c.check(c.run(hs2))


@pytest.mark.parametrize("times", [1, 12])  # (clusters; the line of tiles and its join)
def test_streams_graphs_and_new_lengths(hs2, times):
    """Two streams at once, and two captured calls replayed with other lengths and queries."""
    c = Cache([900 * times, 40, 0, 1500 * times], 16, 2, 128, 32)
    want = c.run(hs2)
    s = [torch.cuda.Stream() for _ in range(2)]
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    got = [c.run(hs2, stream=x) for x in s for _ in range(3)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    nbytes = hs2.paged_attn_workspace_bytes(4, 16, 2, 128)
    graphs = []
    for _ in range(2):
        ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = c.run(hs2, workspace=ws)
        graphs.append((gr, ws, out))
    for lens in ([900, 40, 0, 1500], [1, 0, 0, 1400], [0, 0, 0, 0], [899, 33, 0, 2]):
        lens = [n * times if n > 100 else n for n in lens]
        c.lens = lens
        c.l.copy_(torch.tensor(lens, dtype=torch.int32))
        c.q.mul_(-0.75)
        for gr, _, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for _, ws, out in graphs:
            c.check(out)
            assert hs2.read_device_status(ws) == 0


def test_no_sequences_and_small_workspace(hs2):
    c = Cache([20], 4, 1, 64, 16)
    out, lse = hs2.paged_attn(c.q[:0], c.k, c.v, c.table[:0], c.l[:0])
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    with pytest.raises(hs2.HS2Error) as e:
        c.run(hs2, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == hs2.ERR_WORKSPACE
    with pytest.raises(ValueError):
        hs2.paged_attn(c.q, c.k, c.v[:-1], c.table, c.l)
    with pytest.raises(ValueError):
        hs2.paged_attn(c.q, c.k, c.v, c.table, c.l.long())
    with pytest.raises(ValueError):
        hs2.paged_attn(c.q, c.k.view(torch.int16), c.v, c.table, c.l)
    with pytest.raises(ValueError):
        hs2.paged_attn(c.q.expand(2, 1, 4, 64), c.k, c.v, c.table, c.l)
