"""The e4m3 codes that qk_norm_rope_paged writes: value / scale rounded ONCE to nearest even, for scales that are no
power of two as well. The codes are integers: they have to be equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def codes(x, scale):
    """The e4m3 codes of x / scale (x, scale 32-bit values in float64, on the CPU). The 64-bit quotient stands for the real
    one: it differs from a border between two codes (5 significant bits) by 2^-30 of its size at least unless
    it is that border, for border * scale has 29 bits and x 24 of its own."""
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448 in order
    y = (x / scale).abs()
    border = (grid[1:] + grid[:-1]) / 2
    lo = torch.searchsorted(border, y, right=False)   # ties go down ..
    hi = torch.searchsorted(border, y, right=True)    # .. or up: to the even code
    c = torch.where((lo != hi) & (lo % 2 == 1), hi, lo)
    c = torch.where(torch.isnan(y), 127, c.clamp(max=126))
    return (c + 128 * torch.signbit(x)).to(torch.uint8)


def every_bf16(d):
    """All finite bf16 values, 0 and infinities, as rows of d elements."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    return x[~torch.isnan(x)]


def test_the_definition():
    """(of codes(): torch's own conversion where the quotient is exact)"""
    x = every_bf16(128)
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes(x.double(), 1.0), want)


@pytest.mark.parametrize("d,Hk", [(128, 2), (64, 3)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -5, 0.03, 1.7, 3.0, 0.07, 448.0 / 7.3, 1.0 / 3.0, 1.9999999, 1e-4, 5e5])
def test_every_value(hs2, scale, d, Hk):
    """The values as they are, and keys without a norm at position 0, whose rotation changes nothing."""
    x = every_bf16(d)
    T = -(-x.numel() // (Hk * d))
    x = torch.cat([x, torch.zeros(T * Hk * d - x.numel(), dtype=torch.bfloat16)]).view(T, Hk, d).cuda()
    s = float(torch.tensor(scale, dtype=torch.float32))
    q = torch.zeros(T, Hk, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = torch.ones(16, dtype=torch.float64, device="cuda")
    n = -(-T // 16)
    kp, vp = (torch.zeros(n, 16, Hk, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))  # (an infinite element's partner is no number)
    hs2.qk_norm_rope_paged(q, finite, x, pos, slots, kp, vp, freq, k_scale=scale, v_scale=scale)
    for pool, rows, name in ((vp, x, "v"), (kp, finite, "k")):
        got, rows = pool.view(n * 16, Hk, d)[:T].cpu(), rows.cpu()
        want = codes(rows.double(), s)
        zero = (rows == 0) if name == "k" else torch.zeros_like(rows, dtype=torch.bool)  # (-0 + 0 = 0 in the rotation)
        off = (got != want) & ~(zero & (got % 128 == 0))
        assert not bool(off.any()), (name, int(off.sum()), rows[off][:5].tolist(), got[off][:5].tolist(), want[off][:5].tolist())


def test_rotated_and_normalised_keys(hs2):
    """The keys' codes are those of what the plain form rotates, or the code beside where the 32-bit rotation lies within its
    own error of a border."""
    import plain64 as P
    g = P.gen(11)
    T, H, d, s = 3000, 4, 128, float(torch.tensor(0.03))
    k = P.randn(g, T, H, d, std=1.7)
    w = 1 + P.randn(g, d, dtype=torch.float32, std=0.2)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 41
    freq, m = hs2.rope_frequencies(d)
    kp, vp = (torch.zeros(188, 16, H, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    hs2.qk_norm_rope_paged(k, k, k, pos, torch.arange(T, dtype=torch.int32, device="cuda"), kp, vp, freq, q_weight=w,
                           k_weight=w, k_scale=0.03, v_scale=0.03)
    want, bound = P.norm_rope(k, w, pos, freq)
    got = kp.view(188 * 16, H, d)[:T].view(torch.float8_e4m3fn).double().cpu()
    lo, hi = (codes((want + e).float().double().cpu(), s).view(torch.float8_e4m3fn).double() for e in (-bound, bound))
    assert bool(((got >= lo) & (got <= hi)).all())
