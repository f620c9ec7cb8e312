"""Shapes that the operators around the paged cache refuse, each beside the call that they take: with a device the
refusal is the shape's. Every tensor is real and large enough for the shape that is asked for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def rope(hs2, d=128, rot=128, **kw):
    q = torch.zeros(5, 4, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    return hs2.qk_norm_rope(q, q, pos, torch.ones(rot // 2, dtype=torch.float64, device="cuda"), **kw)


def rope_bwd(hs2, d=128, rot=128):
    q = torch.zeros(5, 4, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    return hs2.qk_norm_rope_bwd(q, q, pos, torch.ones(rot // 2, dtype=torch.float64, device="cuda"), q, q, workspace=ws)


def rope_paged(hs2, d=128, rot=64):
    q = torch.zeros(5, 4, d, dtype=torch.bfloat16, device="cuda")
    i = torch.arange(5, dtype=torch.int32, device="cuda")
    pool = torch.zeros(2, 16, 4, d, dtype=torch.bfloat16, device="cuda")
    return hs2.qk_norm_rope_paged(q, q, q, i, i, pool, pool.clone(), torch.ones(rot // 2, dtype=torch.float64, device="cuda"))


def table(hs2, B=4096):
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    return hs2.page_table_update(torch.zeros(B, 2, dtype=torch.int32, device="cuda"), z, z, torch.zeros(9, dtype=torch.int32, device="cuda"),
                                 torch.zeros(2, dtype=torch.int32, device="cuda"), 16, 3)


def attn(hs2, Hq=64, Hk=1, page=32, d=128, f8=False):
    q = torch.zeros(2, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(4, page, Hk, d, dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    return hs2.paged_attn(q, pool, pool, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), i, workspace=ws,
                          **(dict(k_scale=1.0, v_scale=1.0) if f8 else {}))


@pytest.mark.parametrize("call,good,bad", [
    (rope, dict(d=64, rot=64), dict(d=96, rot=96)), (rope, dict(rot=16), dict(rot=8)), (rope, dict(rot=128), dict(rot=144)),
    (rope_bwd, dict(rot=48), dict(rot=40)), (rope_bwd, dict(d=64, rot=64), dict(d=32, rot=32)), (rope_paged, dict(d=64), dict(d=256)),
    (table, dict(B=4096), dict(B=4097)), (attn, dict(Hq=64), dict(Hq=65)), (attn, dict(page=48), dict(page=24)),
    (attn, dict(d=64), dict(d=64, f8=True)), (attn, dict(d=128, f8=True), dict(d=256)), (attn, dict(Hq=192, Hk=3), dict(Hq=195, Hk=3))])
def test_refused_by_its_shape(hs2, call, good, bad):
    call(hs2, **good)
    with pytest.raises(hs2.HS2Error) as e:
        call(hs2, **bad)
    assert e.value.code == hs2.ERR_UNSUPPORTED_SHAPE
    torch.cuda.synchronize()
