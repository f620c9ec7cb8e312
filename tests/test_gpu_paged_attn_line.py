"""paged_attn's two-kernel form (the line of tiles and its join) against softmax attention in 64 bits: heads of 64,
sliding windows, tables much wider than the sequences, few keys among many sequences."""
import ctypes
import math

import pytest
import torch

import plain64 as P
from plain64 import near
from test_gpu_paged_attn import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def joins(hs2, call):
    """The call's result, and how often it launched the second kernel."""
    lib, ms, n = hs2.lib, ctypes.c_double(), ctypes.c_longlong()
    lib.hs2_profile_enable(b"paged_join")
    try:
        got = call()
        assert lib.hs2_profile_read(b"paged_join", ctypes.byref(ms), ctypes.byref(n)) == 0
    finally:
        lib.hs2_profile_enable(None)
    return got, n.value


def check_line(hs2, c, window=0):
    got, n = joins(hs2, lambda: c.run(hs2, window=window))
    assert n == 1
    c.check(got, window)
    again = c.run(hs2, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert hs2.read_device_status(hs2.cached_workspace("paged_attn")) == 0


def ragged(B, n):
    return [n - (37 * b) % n for b in range(B)]


@pytest.mark.parametrize("lens,Hq,Hk,page", [([30000, 0, 5, 129], 6, 2, 16), ([20001], 64, 1, 128), ([9000, 8191, 1, 4097], 16, 4, 48),
                                             (ragged(320, 150), 1, 1, 16), (ragged(200, 700), 33 * 2, 2, 64),
                                             (ragged(1025, 40), 4, 4, 32)], ids=lambda x: str(x)[:24])
def test_heads_of_64(hs2, lens, Hq, Hk, page):
    check_line(hs2, Cache(lens, Hq, Hk, 64, page))


@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("window", [1, 100, 128, 1000])
@pytest.mark.parametrize("lens,Hq,Hk,page", [(ragged(64, 1500), 16, 8, 16), (ragged(310, 300), 7, 1, 48),
                                             ([5000, 0, 127, 128, 129, 1] * 30, 64 * 2, 2, 128)], ids=lambda x: str(x)[:24])
def test_windows(hs2, lens, Hq, Hk, page, window, d, f8):
    c = Cache(lens, Hq, Hk, d, page, f8)
    for b, n in enumerate(lens):  # pages that lie wholly before the window may be gone
        first = max(0, n - window) // page
        if first:
            c.table[b, :first] = -1
    check_line(hs2, c, window)


@pytest.mark.parametrize("window", [20000, 40000])
@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True)])
def test_long_windows(hs2, window, d, f8):
    """A window cut into many ranges, and one that is longer than the sequence."""
    check_line(hs2, Cache([30000, 17], 8, 1, d, 64, f8), window)


@pytest.mark.parametrize("d,f8", [(64, False), (128, False), (128, True)])
def test_short_sequences_in_a_wide_table(hs2, d, f8):
    """A table for the longest context, sequences of a few tokens: what a captured step of a serving loop has."""
    check_line(hs2, Cache([1000, 1, 0, 63, 130, 2], 64, 1, d, 128, f8, width=2047))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 2, 128])
def test_few_keys_among_many_sequences(hs2, d, window):
    """384 pairs: more than CTAs. Probabilities in one bf16 term (plain64's bound counts its rounding)."""
    c = Cache([2, 3, 7, 64, 65, 256, 1, 0] * 6, 16, 8, d, 16)
    check_line(hs2, c, window)


@pytest.mark.parametrize("f8", [False, True])
def test_infinities_outside_the_window(hs2, f8):
    """(the unused rows of Cache are NaN; here the rows before the window are too)"""
    lens, window = ragged(310, 400), 70
    c = Cache(lens, 4, 1, 128, 16, f8)
    want = P.paged_attn(c.q, c.k, c.v, c.table, lens, 1 / math.sqrt(128), window, c.scales.get("k_scale"), c.scales.get("v_scale"))
    bad = 0x7F if f8 else float("inf")
    for b, n in enumerate(lens):
        at = torch.arange(max(0, n - window), device="cuda")
        if at.numel():
            pg = c.table[b, at // 16].long()
            c.k[pg, at % 16], c.v[pg, at % 16] = bad, bad
    got, n = joins(hs2, lambda: c.run(hs2, window=window))
    assert n == 1
    near(got[0], want[0], want[2], "out")
    near(got[1], want[1], want[3], "lse")
