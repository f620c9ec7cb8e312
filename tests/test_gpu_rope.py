"""qk_norm_rope, its backward and its paged form against the formulas in 64 bits (plain64)."""
import pytest
import torch

import plain64 as P
from plain64 import BF16, E4M3, gen, near, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def inputs(T, Hq, Hk, d, rot, norm, seed=1, first=0):
    """A fused projection's rows (queries, keys, values side by side), positions, frequencies, weights."""
    g = gen(seed)
    qkv = randn(g, T, (Hq + 2 * Hk) * d, std=1.7)
    q, k, v = qkv.split([Hq * d, Hk * d, Hk * d], 1)
    pos = first + torch.arange(T, dtype=torch.int32, device="cuda")
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    w = [None, None] if norm is None else [(1 + randn(g, d, dtype=torch.float32, std=0.3)).to(norm) for _ in range(2)]
    return q.view(T, Hq, d), k.view(T, Hk, d) if Hk else None, v.view(T, Hk, d) if Hk else None, pos, freq, w


SHAPES = [(1, 1, 1, 64, 64, 0), (7, 5, 2, 128, 32, 1000), (33, 64, 1, 128, 128, 1048576), (300, 3, 3, 64, 16, 2 ** 24),
          (2500, 8, 1, 128, 64, 7), (5, 17, 0, 128, 128, 40),
          (40001, 3, 1, 64, 32, 0), (2, 1024, 9, 64, 48, 9)]


@pytest.mark.parametrize("norm", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,first", SHAPES)
def test_forward(hs2, T, Hq, Hk, d, rot, first, interleaved, norm):
    q, k, _, pos, freq, (qw, kw) = inputs(T, Hq, Hk, d, rot, norm, first=first)
    kw = kw if Hk else None
    yq, yk = hs2.qk_norm_rope(q, k, pos, freq, q_weight=qw, k_weight=kw, interleaved=interleaved, mscale=1.25)
    for x, w, y, name in ((q, qw, yq, "q"), (k, kw, yk, "k"))[:2 if Hk else 1]:
        want, bound = P.norm_rope(x, w, pos, freq, interleaved, 1.25)
        near(y, want, BF16 * want.abs() + bound, name)


@pytest.mark.parametrize("norm", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("gk", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,first", SHAPES)
def test_backward(hs2, T, Hq, Hk, d, rot, first, interleaved, norm, gk):
    q, k, _, pos, freq, (qw, kw) = inputs(T, Hq, Hk, d, rot, norm, first=first)
    kw = kw if Hk else None
    g = gen(9)
    gq, gkk = randn(g, T, Hq, d), randn(g, T, Hk, d, dtype=gk, std=4.0) if Hk else None
    how = dict(q_weight=qw, k_weight=kw, interleaved=interleaved, mscale=0.8)
    dq, dk, dqw, dkw = hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gkk, **how)
    for x, w, dy, dx, dw, name in ((q, qw, gq, dq, dqw, "q"), (k, kw, gkk, dk, dkw, "k"))[:2 if Hk else 1]:
        want, wantw, bound, boundw = P.norm_rope_bwd(x, w, pos, freq, dy, interleaved, 0.8)
        near(dx, want, BF16 * want.abs() + bound, "d" + name)
        if w is not None:
            near(dw, wantw, boundw + 2.0 ** -24 * wantw.abs(), f"d{name}_weight")
    again = hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gkk, **how)
    for a, b in zip((dq, dk, dqw, dkw), again):
        assert a is None or torch.equal(a, b)


def test_backward_against_differences(hs2):
    """<dy, f(x + h s) - f(x - h s)> / 2 h in 64 bits against <dx, s> + <dw, t> of the kernel. With h = 2^-12 and rows of
    unit size the third-order term is below 2^-24 of the terms' absolute sum; dx is rounded to bf16 once."""
    T, Hq, Hk, d, rot = 21, 6, 2, 64, 32
    q, k, _, pos, freq, (qw, kw) = inputs(T, Hq, Hk, d, rot, torch.float32, first=100)
    g = gen(3)
    gq, gk = randn(g, T, Hq, d), randn(g, T, Hk, d, dtype=torch.float32)
    dq, dk, dqw, dkw = hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gk, q_weight=qw, k_weight=kw)
    h = 2.0 ** -12
    for x, w, dy, dx, dw in ((q, qw, gq, dq, dqw), (k, kw, gk, dk, dkw)):
        s, t = randn(g, *x.shape, dtype=torch.float64), randn(g, d, dtype=torch.float64)
        f = lambda e: (P.norm_rope(x.double() + e * s, w.double() + e * t, pos, freq)[0] * dy.double()).sum()
        want = (f(h) - f(-h)) / (2 * h)
        got = (dx.double() * s).sum() + (dw.double() * t).sum()
        terms = (dx.double() * s).abs().sum() + (dw.double() * t).abs().sum()
        assert abs(float(got - want)) <= float(terms) * (BF16 + 2.0 ** -16)


def test_batched_shapes_and_strides(hs2):
    """[B, L, H, d] with a key without a head dimension, rows apart, and outputs given."""
    g = gen(4)
    x = randn(g, 3, 11, 9 * 128)
    q, k = x[..., :8 * 128].unflatten(-1, (8, 128)), x[..., 8 * 128:]
    pos = torch.randint(0, 5000, (3, 11), generator=g, device="cuda", dtype=torch.int32)
    freq, m = hs2.rope_frequencies(128, 10000.0, scaling="yarn", factor=4.0, original_len=2048)
    qo, ko = torch.empty(3, 11, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(k, memory_format=torch.contiguous_format)
    a, b = hs2.qk_norm_rope(q, k, pos, freq, mscale=m, q_out=qo, k_out=ko)
    assert a is qo and b is ko
    for x, y in ((q.reshape(33, 8, 128), a), (k.reshape(33, 1, 128), b)):
        want, bound = P.norm_rope(x, None, pos, freq, False, m)
        near(y.reshape(want.shape), want, BF16 * want.abs() + bound, "rows")


def test_no_rows(hs2):
    z = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    f, w = torch.ones(32, dtype=torch.float64, device="cuda"), torch.ones(64, device="cuda")
    a, b = hs2.qk_norm_rope(z, z, i, f, q_weight=w, k_weight=w)
    assert a.shape == z.shape and b.shape == z.shape
    _, _, dqw, dkw = hs2.qk_norm_rope_bwd(z, z, i, f, z, z, q_weight=w, k_weight=w)
    assert not bool(dqw.any()) and not bool(dkw.any())
    pool = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16, device="cuda")
    hs2.qk_norm_rope_paged(z, z, z, i, i, pool, pool, f)
    assert not bool(pool.any())


def make_pools(g, layout, n, page, Hk, d, f8):
    shape = {"plain": (n, page, Hk, d), "heads first": (n, Hk, page, d)}
    new = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8) if f8 else randn(g, *s)
    if layout == "joined":  # K and V of a page side by side
        x = new(n, 2, page, Hk, d)
        return x[:, 0], x[:, 1]
    x, y = new(*shape[layout]), new(*shape[layout])
    return (x.transpose(1, 2), y.transpose(1, 2)) if layout == "heads first" else (x, y)


@pytest.mark.parametrize("layout", ["plain", "joined", "heads first"])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,page,norm", [(1, 1, 1, 64, 16, 16, None), (8, 64, 1, 128, 128, 128, torch.float32),
                                                     (77, 6, 3, 64, 64, 48, torch.bfloat16), (900, 8, 8, 128, 64, 16, None)])
def test_paged(hs2, T, Hq, Hk, d, rot, page, norm, f8, layout):
    g = gen(6)
    q, k, v, pos, freq, (qw, kw) = inputs(T, Hq, Hk, d, rot, norm, first=333)
    n = -(-T // page) + 2
    kp, vp = make_pools(g, layout, n, page, Hk, d, f8)
    slots = torch.randperm(n * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[T // 2::3] = -1
    if T > 3:
        v[1] = 1e30  # saturates in e4m3
        v[2, 0, 3] = float("nan")
    ks, vs = (2.0 ** -5, 0.03) if f8 else (None, None)
    k0, v0 = kp.clone(), vp.clone()
    qo = randn(g, T, Hq, d)
    q0 = qo.clone()
    hs2.qk_norm_rope_paged(q, k, v, pos, slots, kp, vp, freq, q_weight=qw, k_weight=kw, k_scale=ks, v_scale=vs, q_out=qo)
    live = slots >= 0
    assert torch.equal(qo[~live], q0[~live])
    want, bound = P.norm_rope(q, qw, pos, freq)
    near(qo[live], want[live], (BF16 * want.abs() + bound)[live], "q")
    at = slots[live].long()
    untouched = torch.ones(n * page, dtype=torch.bool, device="cuda")
    untouched[at] = False
    un = untouched.view(n, page)
    for pool, old, rows, s, name in ((kp, k0, P.norm_rope(k, kw, pos, freq), ks, "k"), (vp, v0, (v.double(), 0 * v.double()), vs, "v")):
        assert torch.equal(pool[un], old[un]), f"{name}: another row was written"
        got = pool[at // page, at % page]
        want, bound = rows[0][live], rows[1][live]
        if f8:
            want, bound = (want / s).clamp(-448, 448), bound / s
            near(got.view(torch.float8_e4m3fn), want, E4M3 * want.abs() + 2.0 ** -10 + bound + 2.0 ** -22 * want.abs(), name)
        else:
            near(got, want, (BF16 if name == "k" else 0) * want.abs() + bound, name)
    assert hs2.read_device_status(hs2.cached_workspace("rope_paged")) == 0


def test_paged_slot_outside_the_pool(hs2):
    q, k, v, pos, freq, _ = inputs(4, 2, 1, 64, 64, None)
    kp, vp = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([3, 32, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = hs2.qk_norm_rope_paged(q, k, v, pos, slots, kp, vp, freq, workspace=ws)
    assert hs2.read_device_status(ws) == hs2.ERR_DEVICE_BOUNDS
    want, bound = P.norm_rope(q, None, pos, freq)
    near(y[:3], want[:3], (BF16 * want.abs() + bound)[:3], "q")
    flat = kp.view(32, 64)
    assert bool(flat[3].any()) and not bool(flat[:3].any()) and not bool(flat[4:].any())
    assert torch.equal(vp.view(32, 64)[3], v[0, 0])


def test_another_stream_and_graphs(hs2):
    """A call on a side stream, and two graphs with a workspace each whose inputs change between replays."""
    q, k, v, pos, freq, (qw, kw) = inputs(50, 4, 2, 64, 64, torch.float32)
    g = gen(2)
    gq, gk = randn(g, 50, 4, 64), randn(g, 50, 2, 64)
    q, k = q.contiguous(), k.contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = hs2.qk_norm_rope(q, k, pos, freq, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    b = hs2.qk_norm_rope(q, k, pos, freq)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    nbytes = hs2.qk_norm_rope_bwd_workspace_bytes(50, 4, 2, 64)
    outs, graphs = [], []
    for _ in range(2):
        ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gk, q_weight=qw, k_weight=kw, workspace=ws))
        graphs.append((gr, ws))
    with pytest.raises(ValueError):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gk, q_weight=qw, k_weight=kw)
    for scale in (1.0, 0.5):
        q.mul_(scale)
        want = hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gk, q_weight=qw, k_weight=kw)
        for (gr, _), o in zip(graphs, outs):
            gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, want))
