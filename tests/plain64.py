"""Plain 64-bit forms of the operators around the paged cache, and how far a kernel's result may lie
from them. A rounding to a type is off by at most half a step, torch.finfo(type).eps / 2 of the value."""
import math

import torch

BF16 = 2.0 ** -8   # half a bf16 step, relative
E4M3 = 2.0 ** -4   # half an e4m3 step, relative; below 2^-6 half a step is 2^-10
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def partner(x, rot, interleaved):
    """Each rotated element's partner with the sign it has in the rotation; zero from rot on."""
    y = torch.zeros_like(x)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = -x[..., 1:rot:2], x[..., 0:rot:2]
    else:
        h = rot // 2
        y[..., :h], y[..., h:rot] = -x[..., h:rot], x[..., :h]
    return y


def turns(pos, freq, d, rot, interleaved, mscale):
    """Cosine and sine of every element [T, 1, d] (1 and 0 from rot on)."""
    a = pos.double().reshape(-1)[:, None] * freq.double()
    a = a.repeat_interleave(2, -1) if interleaved else torch.cat([a, a], -1)
    cos = torch.ones(a.shape[0], 1, d, dtype=torch.float64, device=a.device)
    sin = torch.zeros_like(cos)
    cos[:, 0, :rot], sin[:, 0, :rot] = a.cos() * mscale, a.sin() * mscale
    return cos, sin


def norm_rope(x, w, pos, freq, interleaved=False, mscale=1.0, eps=EPS):
    """(y, bound): rows [T, H, d] normalised and rotated, and what the 32-bit arithmetic before the last
    rounding may add: a cosine or sine is off by 2^-22 (the reduced angle by 2^-24 turns pi, the function by two
    steps), the reciprocal root by 2^-21 (d squares summed in 32 bits, two steps of the function), four
    products and a sum by 2^-24 each: below 2^-19 of |n| m + |partner| m."""
    rot, d = 2 * freq.numel(), x.shape[-1]
    n = x.double()
    if w is not None:
        n = n / (n.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    cos, sin = turns(pos, freq, d, rot, interleaved, mscale)
    p = partner(n, rot, interleaved)
    return n * cos + p * sin, 2.0 ** -19 * max(1.0, abs(mscale)) * (n.abs() + p.abs())


def norm_rope_bwd(x, w, pos, freq, dy, interleaved=False, mscale=1.0, eps=EPS):
    """(dx, dw, bound_dx, bound_dw). The bounds count 2^-18 for the arithmetic (twice the forward's, the
    mean of u x among it) on the terms' absolute values, and for dw one rounding of 2^-24 a row."""
    rot, d = 2 * freq.numel(), x.shape[-1]
    cos, sin = turns(pos, freq, d, rot, interleaved, mscale)
    dy, x = dy.double(), x.double()
    g = dy * cos - partner(dy * sin, rot, interleaved)
    big = max(1.0, abs(mscale)) * (dy.abs() + partner(dy, rot, interleaved).abs())
    if w is None:
        return g, None, 2.0 ** -18 * big, None
    w = w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    u, ub = g * w, big * w.abs()
    dx = r * (u - x * r.square() * (u * x).mean(-1, keepdim=True))
    bound = 2.0 ** -18 * (r * ub + r ** 3 * x.abs() * (ub * x.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    return dx, (g * x * r).sum((0, 1)), bound, (2.0 ** -18 + rows * 2.0 ** -24) * (big * x.abs() * r).sum((0, 1))


def near(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    same = (got == want) | torch.isnan(want)  # (infinities)
    err = torch.where(same, torch.zeros_like(got), (got - want).abs())
    over = err > bound
    assert not bool(over.any()), f"{what}: {int(over.sum())} of {over.numel()} outside, worst error " \
        f"{float(err[over].max()):.3e}, largest excess {float((err / bound.clamp_min(1e-300))[over].max()):.3g} times the bound"


def cached(pages, table_row, at, e4m3=False, scale=1.0):
    """Rows [n, Hk, d] of one sequence's tokens `at`, in 64 bits."""
    page = pages.shape[1]
    rows = pages[table_row[at // page].long(), at % page]
    return rows.view(torch.float8_e4m3fn).double() * scale if e4m3 else rows.double()


def paged_attn(q, k_pages, v_pages, table, lens, scale, window=0, ks=None, vs=None, p_round=BF16):
    """(out, lse, bound_out, bound_lse) with pools [n_pages, page, Hk, d].

    Bounds. Every probability is rounded once: to bf16 (p_round), or to two e4m3 terms (2^-4 times 2^-4 of the value, and
    half a step of the second term, 2^-10, where the tile's largest probability counts 256: 2^-18 of it; a
    tile is 128 keys), then the output once more. A score is a sum of d products in 32 bits: 2^-16 of their
    absolute sum; an e4m3 cache's query elements are off by 2^-20 of the head's largest at most. 2^-13 for
    exp2, the sums and the rescaling. A probability below 2^-126 of its row's largest, and an output below
    2^-126, is no normal 32-bit (or bf16) number and may become zero: 2^-126 of each key's |v|, and 2^-126."""
    B, _, Hq, d = q.shape
    Hk, f8 = k_pages.shape[2], ks is not None
    out = torch.zeros(B, 1, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, 1, Hq), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        if n == 0:
            continue
        at = torch.arange(first, n, device=q.device)
        K, V = cached(k_pages, table[b], at, f8, ks or 1.0), cached(v_pages, table[b], at, f8, vs or 1.0)
        qb = q[b, 0].double().view(Hk, Hq // Hk, d)
        x = torch.einsum("hgd,nhd->hgn", qb, K) * scale
        p = torch.softmax(x, -1)
        o = torch.einsum("hgn,nhd->hgd", p, V)
        A = torch.einsum("hgn,nhd->hgd", p, V.abs())
        ds = 2.0 ** -16 * torch.einsum("hgd,nhd->hgn", qb.abs(), K.abs()).amax(-1) * scale
        if f8:
            ds = ds + 2.0 ** -20 * qb.abs().amax(-1) * K.abs().sum(-1).amax(0)[:, None] * scale
        e = BF16 * o.abs() + (p_round + 2.0 ** -13 + 2 * ds[..., None]) * A
        e = e + 2.0 ** -126 * (1 + V.abs().sum(0)[:, None])
        if f8:
            tile = torch.div(at, 128, rounding_mode="floor") - first // 128
            most = torch.zeros(Hk, Hq // Hk, int(tile[-1]) + 1, dtype=torch.float64, device=q.device)
            most.scatter_reduce_(2, tile.expand_as(p), p, "amax")
            e = e + 2.0 ** -18 * torch.einsum("hgn,nhd->hgd", most.gather(2, tile.expand_as(p)), V.abs())
        out[b, 0], bo[b, 0] = o.reshape(Hq, d), e.reshape(Hq, d)
        lse[b, 0] = torch.logsumexp(x, -1).reshape(Hq)
        bl[b, 0] = (ds + 2.0 ** -20).reshape(Hq) + 2.0 ** -21 * lse[b, 0].abs()
    return out, lse, bo, bl


def page_table_step(table, lens, delta, ring, head, count, page, max_tokens):
    """One request after the other (lists; table and ring are updated): none that needs pages is served after
    one that the free list could not serve. Returns (lens, head, count, cu, positions, slots)."""
    cap, taken, short, back, cu, pos, slots = len(ring), 0, False, [], [0], [], []
    new = []
    for b, (n, x) in enumerate(zip(lens, delta)):
        held, want = -(-n // page), -(-(n + x) // page)
        short = short or want - held > count - taken
        ok = want <= held or not short
        if want > held and ok:
            for j in range(held, want):
                table[b][j] = ring[(head + taken) % cap]
                taken += 1
        elif want < held:
            back += [table[b][j] for j in range(want, held)]
        for i in range(max(x, 0)):
            pos.append(n + i)
            slots.append(table[b][(n + i) // page] * page + (n + i) % page if ok else -1)
        cu.append(cu[-1] + max(x, 0))
        new.append(n + x if ok else n)
    for i, g in enumerate(back):
        ring[(head + count + i) % cap] = g
    pad = [-1] * (max_tokens - len(pos))
    return new, (head + taken) % cap, count - taken + len(back), cu, pos + pad, slots + pad
