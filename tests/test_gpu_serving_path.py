"""The operators around the paged cache together, and with the framework's own attention: requests that
grow, shrink and end over one pool, and a training step's projection gradients."""
import math
import random

import pytest
import torch

import plain64 as P
from plain64 import BF16, gen, near, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


@pytest.mark.parametrize("Hq,Hk,d,page,f8", [(64, 1, 128, 128, False), (8, 2, 64, 16, False), (12, 3, 128, 32, True)])
def test_requests_over_one_pool(hs2, Hq, Hk, d, page, f8):
    """Prompts, chunks, single tokens, cut-backs and ends; every step page_table_update (in place),
    qk_norm_rope_paged, and attention of each request's newest token, against each request's own keys and
    values kept apart in 64 bits."""
    g, r = gen(1), random.Random(2)
    B, width, most = 6, 40, 40 * page
    n_pages = 70
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, state = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor([5, n_pages], dtype=torch.int32, device="cuda")
    ring = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    kind = torch.uint8 if f8 else torch.bfloat16
    bad = 0x7F if f8 else float("nan")
    k_pages, v_pages = (torch.full((n_pages, page, Hk, d), bad, dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (2.0 ** -4, 2.0 ** -5) if f8 else (None, None)
    freq, mscale = hs2.rope_frequencies(d // 2, 10000.0, scaling="linear", factor=2.0)
    qw, kw = (1 + randn(g, d, dtype=torch.float32, std=0.2) for _ in range(2))
    mine = [([], []) for _ in range(B)]  # each request's rows in 64 bits
    held = [0] * B
    for step in range(7):
        delta = [r.choice([1, 1, r.randrange(1, 4 * page), -(held[b] // 2), -held[b]]) if held[b] else r.randrange(1, 5 * page)
                 for b in range(B)]
        T = sum(max(x, 0) for x in delta) + 3  # padding rows at the end
        lens, state, cu, pos, slots = hs2.page_table_update(table, lens, torch.tensor(delta, dtype=torch.int32, device="cuda"),
                                                            ring, state, page, T, lens_out=lens, free_state_out=state)
        qkv = randn(g, T, (Hq + 2 * Hk) * d)
        q, k, v = qkv.split([Hq * d, Hk * d, Hk * d], 1)
        q, k, v = q.view(T, Hq, d), k.view(T, Hk, d), v.view(T, Hk, d)
        yq = hs2.qk_norm_rope_paged(q, k, v, pos, slots, k_pages, v_pages, freq, q_weight=qw, k_weight=kw, mscale=mscale,
                                    k_scale=ks, v_scale=vs)
        cu = cu.tolist()
        held = [n + x for n, x in zip(held, delta)]
        assert lens.tolist() == held and int(state[1]) == n_pages - sum(-(-n // page) for n in held)
        live = slice(0, cu[-1])
        wq, bq = P.norm_rope(q[live], qw, pos[live], freq, False, mscale)
        near(yq[live], wq, BF16 * wq.abs() + bq, "queries")
        wk, bk = P.norm_rope(k[live], kw, pos[live], freq, False, mscale)
        for b in range(B):
            K, V = mine[b]
            if delta[b] < 0:
                mine[b] = (K[:held[b]], V[:held[b]])
                continue
            K.extend(wk[cu[b]:cu[b + 1]])
            V.extend(v[cu[b]:cu[b + 1]].double())
        # one query per request against its whole cache
        q1 = randn(g, B, 1, Hq, d)
        out, lse = hs2.paged_attn(q1, k_pages, v_pages, table, lens, k_scale=ks, v_scale=vs)
        want = P.paged_attn(q1, k_pages, v_pages, table, held, 1 / math.sqrt(d), 0, ks, vs)
        near(out, want[0], want[2], "out")
        near(lse, want[1], want[3], "lse")
        # and the cache holds the requests' rows
        for b in range(B):
            if held[b]:
                at = torch.arange(held[b], device="cuda")
                for pool, rows, s in ((k_pages, mine[b][0], ks), (v_pages, mine[b][1], vs)):
                    rows = torch.stack(list(rows))
                    half = 2.0 ** -4 * rows.abs() + 2.0 ** -10 * s if f8 else BF16 * rows.abs()
                    near(P.cached(pool, table[b], at, f8, s or 1.0), rows, half + 2.0 ** -16 * rows.abs().amax(-1, keepdim=True), "cache")
    for key in ("page_table", "rope_paged", "paged_attn"):
        assert hs2.read_device_status(hs2.cached_workspace(key)) == 0


def test_the_selecting_layer_reads_the_same_pool(hs2):
    """A full layer (hs2_full_attn_select_paged) over pages that qk_norm_rope_paged filled, and paged_attn over them:
    the same attention."""
    g = gen(3)
    B, n, H, d, page = 3, 700, 64, 128, 128
    width = -(-n // page)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.tensor([700, 129, 384], dtype=torch.int32, device="cuda")
    T = int(lens.sum())
    ring = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32)
    _, _, _, pos, slots = hs2.page_table_update(table, zero, lens, ring, torch.tensor([0, B * width], dtype=torch.int32, device="cuda"),
                                                page, T)
    k_pages, v_pages = (torch.zeros(B * width, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freq, _ = hs2.rope_frequencies(d)
    q, k, v = randn(g, T, H, d), randn(g, T, d), randn(g, T, d)
    hs2.qk_norm_rope_paged(q, k, v, pos, slots, k_pages, v_pages, freq)
    q1 = randn(g, B, 1, H, d)
    out, lse = hs2.paged_attn(q1, k_pages, v_pages, table, lens)
    full = hs2.full_attn_select_paged(q1, k_pages, v_pages, table.clamp(min=0), lens.tolist())
    want = P.paged_attn(q1, k_pages[:, :, None], v_pages[:, :, None], table, lens.tolist(), 1 / math.sqrt(d))
    near(out, want[0], want[2], "out")
    assert float((full[0].double() - want[0]).abs().max()) < 2e-2  # (the framework's own bar)
    assert float((full[1].double() - lse.double()).abs().max()) < 2e-3


def test_training_step(hs2):
    """Norm and rotation, the causal full layer, its backward, and back through the rotation: the gradients of the
    projection's rows and of the norm weights against 64-bit differentiation of the whole. Between the
    operators the queries, keys, outputs and gradients are bf16, and the attention's own bars are 2e-2 of the
    largest value, relative L2 5e-3 forward and 1e-2 for its gradients; three of them add up."""
    g = gen(5)
    B, L, H, d = 2, 257, 64, 128
    x = randn(g, B, L, (H + 2) * d)
    q, k, v = x[..., :H * d].unflatten(-1, (H, d)), x[..., H * d:(H + 1) * d], x[..., (H + 1) * d:].contiguous()
    pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    freq, _ = hs2.rope_frequencies(d)
    qw, kw = (1 + randn(g, d, dtype=torch.float32, std=0.2) for _ in range(2))
    rq, rk = hs2.qk_norm_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    out, lse, _ = hs2.full_attn_select(rq, rk, v)
    dout = randn(g, B, L, H, d)
    got = hs2.full_attn_bwd(rq, rk, v, out, lse, dout)
    dq, dk, dqw, dkw = hs2.qk_norm_rope_bwd(q, k, pos, freq, got[0], got[1], q_weight=qw, k_weight=kw)

    leaves = [q.double().reshape(B * L, H, d), k.double().reshape(B * L, 1, d), qw.double(), kw.double()]
    leaves = [t.requires_grad_() for t in leaves]
    yq = P.norm_rope(leaves[0], leaves[2], pos, freq)[0].view(B, L, H, d)
    yk = P.norm_rope(leaves[1], leaves[3], pos, freq)[0].view(B, L, d)
    s = torch.einsum("bihd,bjd->bhij", yq, yk) / math.sqrt(d)
    s = s.masked_fill(torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    y = torch.einsum("bhij,bjd->bihd", torch.softmax(s, -1), v.double())
    want = torch.autograd.grad(y, leaves, dout.double())
    for a, b, name in zip((dq.view(B * L, H, d), dk.view(B * L, 1, d), dqw, dkw), want, ("dq", "dk", "dq_weight", "dk_weight")):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 3e-2, (name, rel)
