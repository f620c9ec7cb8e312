"""What the operators around the paged cache refuse, and their host-side numbers (CPU only)."""
import ctypes
import math

import pytest
import torch

import long_context_mqa_b200 as hs2

L = hs2.lib
A = 1 << 20  # a 16-byte aligned stand-in address that no accepted call is given here
INF, NAN = float("inf"), float("nan")


def strides(*s):
    return (ctypes.c_longlong * 3)(*s)


ROPE = dict(q=A, k=A, qt=8192, qh=128, kt=128, kh=128, pos=A, freq=A, T=4, Hq=64, Hk=1, d=128, rot=128, inter=0, m=1.0,
            eps=1e-6, qw=A, kw=A, f32=0)


def rope(**over):
    a = {**ROPE, "qo": A, "ko": A, **over}
    return L.hs2_qk_norm_rope(*a.values(), None)


def rope_bwd(**over):
    a = {**ROPE, "gq": A, "gk": A, "g32": 0, "dq": A, "dk": A, "dqw": A, "dkw": A, "ws": A, "wsb": 1 << 30, **over}
    return L.hs2_qk_norm_rope_bwd(*a.values(), None)


def rope_paged(**over):
    s = strides(16384, 128, 128)
    a = dict(q=A, k=A, v=A, qt=8192, qh=128, kt=128, kh=128, vt=128, vh=128, pos=A, slots=A, freq=A, T=4, Hq=64, Hk=1, d=128,
             rot=128, inter=0, m=1.0, eps=1e-6, qw=A, kw=A, f32=0, qo=A, kp=A, vp=A, ks=s, vs=s, n=8, page=128, e4m3=0,
             kscale=1.0, vscale=1.0, ws=A, wsb=256)
    a.update(over)
    return L.hs2_qk_norm_rope_paged(*a.values(), None)


def table(**over):
    a = dict(t=A, B=4, width=8, lens=A, delta=A, ring=A, cap=64, state=A, page=16, T=9, lo=A, so=A, cu=A, pos=A, slots=A,
             ws=A, wsb=256)
    a.update(over)
    return L.hs2_page_table_update(*a.values(), None)


def attn(**over):
    s = strides(16384, 128, 128)
    a = dict(q=A, k=A, v=A, ks=s, vs=s, n=8, page=128, tab=A, width=8, lens=A, B=2, Hq=64, Hk=1, d=128, e4m3=0, kscale=1.0,
             vscale=1.0, scale=0.1, window=0, out=A, lse=A, ws=A, wsb=1 << 30)
    a.update(over)
    return L.hs2_paged_attn(*a.values(), None)


ROPE_BAD = [dict(q=None), dict(q=A + 8), dict(k=None), dict(pos=None), dict(freq=None), dict(T=-1), dict(Hq=0), dict(Hk=-1),
            dict(Hq=2000), dict(qt=8193), dict(kh=-128), dict(kw=None), dict(qw=None), dict(eps=-1.0), dict(eps=NAN),
            dict(m=INF), dict(m=NAN)]


@pytest.mark.parametrize("call,bad", [(rope, b) for b in ROPE_BAD + [dict(qo=None), dict(ko=A + 2)]]
                         + [(rope_bwd, b) for b in ROPE_BAD + [dict(gq=None), dict(gk=None), dict(dq=None), dict(dk=A + 4),
                                                               dict(dqw=None), dict(dkw=None)]]
                         + [(rope_paged, b) for b in [dict(v=None), dict(slots=None), dict(kp=None), dict(vp=A + 8),
                                                      dict(ks=None), dict(Hk=0), dict(n=0), dict(page=0),
                                                      dict(n=1 << 20, page=1 << 12), dict(ks=strides(16384, 0, 128)),
                                                      dict(vs=strides(16384, 132, 128)), dict(e4m3=1, kscale=0.0),
                                                      dict(e4m3=1, vscale=NAN), dict(e4m3=1, kscale=1e-39),
                                                      dict(e4m3=1, ks=strides(16384, 128, 8))]]
                         + [(table, b) for b in [dict(t=None), dict(B=0), dict(width=0), dict(cap=0), dict(page=0),
                                                 dict(T=-1), dict(pos=None), dict(lens=None), dict(cu=None),
                                                 dict(width=1 << 20, page=1 << 12)]]
                         + [(attn, b) for b in [dict(q=None), dict(k=A + 8), dict(out=None), dict(lens=None), dict(Hk=0),
                                                dict(Hq=3, Hk=2), dict(B=-1), dict(n=0), dict(page=0), dict(width=0),
                                                dict(window=-1), dict(scale=0.0), dict(scale=NAN), dict(scale=INF),
                                                dict(ks=strides(-16384, 128, 128)), dict(e4m3=1, kscale=INF),
                                                dict(width=1 << 20, page=1 << 12)]])
def test_bad_arguments_are_refused(call, bad):
    assert call(**bad) == hs2.ERR_INVALID_ARG


@pytest.mark.parametrize("call,bad", [(rope, dict(d=96, rot=96)), (rope, dict(rot=8)), (rope, dict(rot=144)),
                                      (rope_bwd, dict(rot=40)), (rope_paged, dict(d=256)), (table, dict(B=4097)),
                                      (attn, dict(Hq=65)), (attn, dict(page=24)), (attn, dict(d=64, e4m3=1)),
                                      (attn, dict(d=256))])
def test_unsupported_shapes_are_refused(call, bad):
    assert call(**bad) == hs2.ERR_UNSUPPORTED_SHAPE


def test_workspace_queries():
    assert hs2.paged_attn_workspace_bytes(8, 64, 1, 128) > 256
    for bad in ((8, 65, 1, 128), (8, 64, 0, 128), (8, 5, 2, 128), (8, 64, 1, 96), (-1, 64, 1, 128)):
        assert hs2.paged_attn_workspace_bytes(*bad) == 0
    assert hs2.qk_norm_rope_bwd_workspace_bytes(1000, 64, 1, 128) > 256
    assert hs2.qk_norm_rope_bwd_workspace_bytes(0, 64, 1, 128) == 256
    assert hs2.qk_norm_rope_bwd_workspace_bytes(10, 64, 1, 100) == 0


def test_host_tensors_and_wrong_tensors_are_refused():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    pool = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hs2.qk_norm_rope(q, q, i, f)
    with pytest.raises(ValueError):
        hs2.qk_norm_rope_bwd(q, q, i, f, q, q)
    with pytest.raises(ValueError):
        hs2.qk_norm_rope_paged(q, q, q, i, i, pool, pool, f)
    with pytest.raises(ValueError):
        hs2.qk_norm_rope_paged(q, q, q, i, i, pool, pool, f, k_scale=1.0)  # one scale without the other
    with pytest.raises(ValueError):
        hs2.page_table_update(torch.zeros(3, 4, dtype=torch.int32), i, i, i, i[:2], 16, 5)
    with pytest.raises(ValueError):
        hs2.paged_attn(q[:, None], pool, pool, torch.zeros(3, 1, dtype=torch.int32), i)


def test_rope_frequencies():
    f, m = hs2.rope_frequencies(8, 10000.0, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(hs2.rope_frequencies(8, scaling="linear", factor=4.0, device="cpu")[0], f / 4, rtol=1e-14)
    n, m = hs2.rope_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert m == 1.0 and float(n[0]) == 1.0  # the fastest pair as it was, the slowest interpolated by the factor
    assert math.isclose(float(n[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    y, m = hs2.rope_frequencies(64, 10000.0, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    g = hs2.rope_frequencies(64, 10000.0, device="cpu")[0]
    assert math.isclose(m, 0.1 * math.log(8.0) + 1.0)
    assert float(y[0]) == float(g[0]) and math.isclose(float(y[-1]), float(g[-1]) / 8, rel_tol=1e-12)
    assert bool(((y <= g) & (y >= g / 8 * (1 - 1e-12))).all())
    for bad in (dict(rot=7), dict(rot=8, base=0.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="yarn", factor=2.0), dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            hs2.rope_frequencies(device="cpu", **bad)
