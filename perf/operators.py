"""The operators around a paged K/V cache, in their plain form and as this package's calls.

    rope        qk_norm_rope: norm of every query and key head and the position rotation, one pass
    rope_bwd    qk_norm_rope_bwd: its gradient
    rope_paged  qk_norm_rope_paged: the same for serving, the rotated keys and the values written
                into the pages of a bf16 or e4m3 cache
    tables      page_table_update: page tables, slots and positions from the requests' lengths
    attn        paged_attn: attention of one new token per sequence over the paged cache

Every case is a dict of plain values; prepare() makes its inputs from a seed, run() makes one pass,
exact() gives the result in 64 bits from the definition.
"""
import math
import random

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _rope(op, T, Hq, Hk, d, rot, interleaved, norm, far, **more):
    return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "interleaved": interleaved, "norm": norm,
            "far": far, **more}


def _attn(B, L, mix, Hq, Hk, d, page, window, fp8):
    return {"op": "attn", "B": B, "L": L, "mix": mix, "Hq": Hq, "Hk": Hk, "d": d, "page": page, "window": window,
            "fp8": fp8}


def listed():
    return [
        # one decode step of eight sequences at 256k tokens: latency
        {"name": "rope_paged decode 8", **_rope("rope_paged", 8, 64, 1, 128, 128, False, True, 262144, page=128,
                                                 fp8=False, pad=0)},
        # a mixed batch of prompt chunks into an e4m3 cache, part of the head rotated, padded rows at the end
        {"name": "rope_paged chunk e4m3", **_rope("rope_paged", 4099, 32, 8, 128, 64, True, True, 20000, page=64,
                                                   fp8=True, pad=37)},
        # the full layer's queries and key of a 32k prompt
        {"name": "rope prompt 32k", **_rope("rope", 32768, 64, 1, 128, 128, False, True, 32768)},
        # the small model: 16 heads of 64, interleaved pairs, half of the head rotated, no norm
        {"name": "rope tiny 2k", **_rope("rope", 2048, 16, 1, 64, 32, True, False, 2048)},
        # training on a 32k prompt: the gradient that reaches the projection
        {"name": "rope_bwd 32k", **_rope("rope_bwd", 32768, 64, 1, 128, 128, False, True, 32768)},
        # an odd number of tokens, several key heads, interleaved
        {"name": "rope_bwd odd", **_rope("rope_bwd", 1009, 32, 4, 64, 64, True, True, 5000)},
        # one new token for each of 32 requests
        {"name": "tables decode 32", "op": "tables", "B": 32, "L": 32768, "page": 128, "chunk": 1, "mix": 1},
        # 511 requests: prompts, chunks, single tokens, some cut back, some ended
        {"name": "tables mixed 511", "op": "tables", "B": 511, "L": 8192, "page": 16, "chunk": 700, "mix": 2},
        # one sequence of a thousand tokens: latency
        {"name": "attn one 1000", **_attn(1, 1000, 0, 64, 1, 128, 128, 0, False)},
        # a ragged batch with groups of four heads and small pages
        {"name": "attn ragged gqa", **_attn(48, 8192, 3, 32, 8, 128, 16, 0, False)},
        # eight sequences of 256k tokens, 64 heads on one key head
        {"name": "attn 256k", **_attn(8, 262144, 0, 64, 1, 128, 128, 0, False)},
        # the same lengths, ragged, over an e4m3 cache
        {"name": "attn 256k e4m3", **_attn(8, 262144, 5, 64, 1, 128, 128, 0, True)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "rope_paged", "tables", "attn", "attn", "attn"])
    Hk = rng.choice([1, 1, 1, 2, 4, 8])
    if op == "tables":
        B = _log(rng, 1, 1024)
        return {"op": op, "B": B, "L": _log(rng, 16, 65536), "page": rng.choice([16, 32, 48, 64, 128]),
                "chunk": rng.choice([1, _log(rng, 2, max(3, 65536 // B))]), "mix": rng.randrange(1 << 20)}
    if op == "attn":
        G = rng.choice([1, 2, 3, 4, 7, 8, 16, 33, 64])
        B = _log(rng, 1, 256)
        fp8 = rng.random() < 0.4
        d = 128 if fp8 else rng.choice([64, 128, 128])
        most = min(262144, 2 * 1024 * 1024 // (B * Hk))
        window = rng.choice([0, 0, 0, 128, 1000])
        return _attn(B, _log(rng, 1, most), rng.choice([0, 1 + rng.randrange(1 << 20)]), G * Hk, Hk, d,
                     rng.choice([16, 32, 48, 64, 128]), window, fp8)
    d = rng.choice([64, 128])
    Hq = Hk * rng.choice([1, 2, 3, 5, 8, 16] + ([64] if Hk == 1 else []))
    most = min(32768, 32768 * 64 // Hq)
    more = {}
    if op == "rope_paged":
        more = {"page": rng.choice([16, 32, 48, 64, 128]), "fp8": rng.random() < 0.5, "pad": rng.choice([0, 0, 5, 64])}
        most = min(8192, most)
    T = _log(rng, 1, most)
    return _rope(op, T, Hq, Hk, d, rng.choice([16, 32, 64, d]), rng.random() < 0.5, rng.random() < 0.7,
                 _log(rng, 1000, 1000000), **more)


def _lens(case):
    """The cached lengths of the case's sequences: all L, or spread below it with some empty."""
    B, L = case["B"], case["L"]
    if not case["mix"]:
        return [L] * B
    r = random.Random(case["mix"])
    return [L if b == 0 else int(L * r.random() ** 2) for b in range(B)]


def _deltas(case):
    """What each request gains this step; a tenth of a mixed batch is cut back or ends."""
    r = random.Random(case["mix"] + 1)
    lens = _lens(case)
    if case["chunk"] == 1:
        return [1] * len(lens)
    got = []
    for n in lens:
        x = r.random()
        got.append(-n if x < 0.05 else -(n // 3) if x < 0.1 else 1 if x < 0.5 else r.randrange(case["chunk"]))
    return got


def _ceil(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "tables":
        lens, ds, page = _lens(case), _deltas(case), case["page"]
        toks = sum(max(x, 0) for x in ds)
        new = sum(max(_ceil(n + x, page) - _ceil(n, page), 0) for n, x in zip(lens, ds))
        gone = sum(max(_ceil(n, page) - _ceil(n + x, page), 0) for n, x in zip(lens, ds))
        # lengths and deltas read, lengths and offsets written; slot and position of every token;
        # every page gained or given back read once and written once
        return {"bytes": 16 * len(lens) + 8 * toks + 8 * (new + gone), "flops": 0}
    if op == "attn":
        B, d, Hk, Hq = case["B"], case["d"], case["Hk"], case["Hq"]
        seen = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
        kv = sum(seen) * Hk * d * 2 * (1 if case["fp8"] else 2)
        return {"bytes": kv + B * Hq * (4 * d + 4) + sum(_ceil(n, case["page"]) for n in seen) * 4 + 4 * B,
                "flops": 4 * sum(seen) * Hq * d}
    T, Hq, Hk, d, rot = case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
    if op == "rope":
        return {"bytes": T * ((Hq + Hk) * d * 4 + 4) + rot * 4, "flops": T * (Hq + Hk) * (4 * d + 3 * rot)}
    if op == "rope_bwd":
        return {"bytes": T * (Hq * d * 6 + Hk * d * 8 + 4) + rot * 4, "flops": T * (Hq + Hk) * (9 * d + 3 * rot)}
    live = T - min(case["pad"], T - 1)
    cache = 1 if case["fp8"] else 2
    return {"bytes": live * (Hq * d * 4 + Hk * d * 2 * (2 + cache) + 8) + rot * 4,
            "flops": live * (Hq + Hk) * (4 * d + 3 * rot)}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _codes(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").mul_(16).to(torch.float8_e4m3fn).view(torch.uint8)


def _inv_freq(rot, base=500000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if op in ("tables", "attn"):
        lens, page, B = _lens(case), case["page"], case["B"]
        ds = _deltas(case) if op == "tables" else [0] * B
        held = [_ceil(n, page) for n in lens]
        width = max(1, max(_ceil(max(n, n + x), page) for n, x in zip(lens, ds)))
        grow = sum(max(_ceil(n + x, page) - h, 0) for n, x, h in zip(lens, ds, held))
        n_pages = sum(held) + grow + 5
        perm = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
        h = torch.tensor(held, device="cuda")
        at = torch.cumsum(h, 0) - h
        col = torch.arange(width, device="cuda")
        table = torch.where(col < h[:, None], perm[(at[:, None] + col).clamp_(max=n_pages - 1)], -1).to(torch.int32)
        s.update(page_table=table.contiguous(), lens=torch.tensor(lens, **i32))
        if op == "tables":
            # the free pages in a ring that starts in the middle of its buffer
            ring = torch.full((n_pages,), -1, **i32)
            free = perm[sum(held):]
            head = seed % n_pages
            ring[(head + torch.arange(free.numel(), device="cuda")) % n_pages] = free
            T = sum(max(x, 0) for x in ds) + 3  # a few rows behind the last request
            s.update(delta=torch.tensor(ds, **i32), free_ring=ring,
                     free_state=torch.tensor([head, free.numel()], **i32), T=T,
                     lens_out=torch.zeros(B, **i32), state_out=torch.zeros(2, **i32), cu=torch.zeros(B + 1, **i32),
                     positions=torch.zeros(T, **i32), slots=torch.zeros(T, **i32))
            return s
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        make = _codes if case["fp8"] else _randn
        s.update(q=_randn(g, B, 1, Hq, d, std=1.5), k=make(g, n_pages, page, Hk, d), v=make(g, n_pages, page, Hk, d),
                 out=torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(B, 1, Hq, device="cuda"), scale=1 / math.sqrt(d), ks=2.0 ** -4, vs=2.0 ** -5)
        return s
    T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
    # the rows of a fused projection: queries, keys and values of a token side by side
    qkv = _randn(g, T, (Hq + 2 * Hk) * d, std=1.7)
    q, k, v = qkv.split([Hq * d, Hk * d, Hk * d], dim=1)
    s.update(q=q.view(T, Hq, d), k=k.view(T, Hk, d), v=v.view(T, Hk, d), inv_freq=_inv_freq(case["rot"]),
             mscale=1.0 if case["rot"] < 64 else 1.1, qw=None, kw=None)
    if case["norm"]:
        s.update(qw=1 + _randn(g, d, dtype=torch.float32, std=0.2), kw=1 + _randn(g, d, dtype=torch.float32, std=0.2))
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    first = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, **i32)
    s.update(positions=first + torch.arange(T, **i32))
    if op == "rope":
        s.update(q_out=torch.zeros(T, Hq, d, **bf), k_out=torch.zeros(T, Hk, d, **bf))
    elif op == "rope_bwd":
        # the attention's backward gives the queries' gradient in bf16 and the shared keys' in fp32
        s.update(dq_out=_randn(g, T, Hq, d), dk_out=_randn(g, T, Hk, d, dtype=torch.float32, std=4.0),
                 dq=torch.zeros(T, Hq, d, **bf), dk=torch.zeros(T, Hk, d, **bf))
        s.update(dqw=None, dkw=None)
        if case["norm"]:
            s.update(dqw=torch.zeros(d, device="cuda"), dkw=torch.zeros(d, device="cuda"))
    else:
        page = case["page"]
        n_pages = _ceil(T, page) + 3
        make = _codes if case["fp8"] else _randn
        live = T - min(case["pad"], T - 1)
        slots = torch.randperm(n_pages, generator=g, device="cuda")[torch.arange(T, device="cuda") // page] * page
        slots = (slots + torch.arange(T, device="cuda") % page).to(torch.int32)
        slots[live:] = -1
        s["positions"] = s["positions"].clone()
        s["positions"][live:] = -1
        s.update(slots=slots, k_pages=make(g, n_pages, page, Hk, d), v_pages=make(g, n_pages, page, Hk, d),
                 q_out=torch.zeros(T, Hq, d, **bf), ks=2.0 ** -5, vs=2.0 ** -5)
    return s


# --------------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------------
def _angles(s, dtype):
    """cos and sin [T, 1, rot / 2], angles in 64 bits."""
    a = s["positions"].double()[:, None] * s["inv_freq"]
    return (a.cos() * s["mscale"]).to(dtype)[:, None], (a.sin() * s["mscale"]).to(dtype)[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    """(a, b) -> (a cos - b sin, b cos + a sin) over the pairs of the first `rot` elements."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    ya.copy_(a * cos - b * sin)
    yb.copy_(b * cos + a * sin)
    return y


def _norm_rope(s, x, w, cos, sin):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _rotate(x, cos, sin, c["rot"], c["interleaved"])


def _norm_rope_bwd(s, x, w, dy, cos, sin):
    c = s["case"]
    x, g = x.float(), _rotate(dy.float(), cos, -sin, c["rot"], c["interleaved"])
    if w is None:
        return g, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    u = g * w
    return r * (u - x * r.square() * (u * x).mean(-1, keepdim=True)), (g * x * r).sum((0, 1))


def _to_cache(x, scale, fp8):
    if not fp8:
        return x.to(torch.bfloat16)
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _write_rows(pages, slots, rows):
    """rows [T, Hk, d] to the slots that are not negative (the others to a row behind the pool)."""
    flat = pages.view(-1, *pages.shape[2:])
    room = torch.cat([flat, flat[:1]])
    room[torch.where(slots < 0, flat.shape[0], slots).long()] = rows
    flat.copy_(room[:-1])


def _tables(s):
    c = s["case"]
    page, table, ring = c["page"], s["page_table"], s["free_ring"]
    lens, delta, T = s["lens"].long(), s["delta"].long(), s["T"]
    new = lens + delta
    held, want = (lens + page - 1) // page, (new + page - 1) // page
    grow, gone = (want - held).clamp(min=0), (held - want).clamp(min=0)
    cap, (head, count) = ring.numel(), s["free_state"].long().unbind()
    at = torch.cumsum(grow, 0) - grow
    col = torch.arange(table.shape[1], device="cuda")
    added = (col >= held[:, None]) & (col < want[:, None])
    table.copy_(torch.where(added, ring[(head + at[:, None] + col - held[:, None]) % cap], table))
    # pages given back go behind the last free one, in the order of the requests
    back = torch.cumsum(gone, 0) - gone
    room = torch.cat([ring, ring[:1]])
    left = (col >= want[:, None]) & (col < held[:, None])
    to = torch.where(left, (head + count + back[:, None] + col - want[:, None]) % cap, cap)
    room[to] = table
    ring.copy_(room[:-1])
    toks = delta.clamp(min=0)
    s["cu"][1:] = torch.cumsum(toks, 0)
    cu = s["cu"].long()
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], row, right=True)
    live = b < lens.numel()
    b = b.clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[b] + row - cu[b], -1)
    slot = table[b, pos.clamp(min=0) // page].long() * page + pos.clamp(min=0) % page
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, slot, -1))
    s["lens_out"].copy_(new)
    s["state_out"].copy_(torch.stack([(head + grow.sum()) % cap, count - grow.sum() + gone.sum()]))


def _attend(s):
    c = s["case"]
    B, Hq, Hk, d, page = c["B"], c["Hq"], c["Hk"], c["d"], c["page"]
    lens = s["lens"].long()
    L = s["page_table"].shape[1] * page
    at = torch.arange(L, device="cuda")
    seen = at < lens[:, None]
    if c["window"]:
        seen &= at >= lens[:, None] - c["window"]
    pages = s["page_table"].long().clamp(min=0)
    k, v = s["k"][pages].view(B, L, Hk, d), s["v"][pages].view(B, L, Hk, d)
    if c["fp8"]:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    k, v = k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)
    q = s["q"].float().view(B, Hk, Hq // Hk, d)
    x = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] * (s["ks"] if c["fp8"] else 1.0))
    del k
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen[:, None, :, None], 0)
    o = torch.matmul(p, v) * (s["vs"] if c["fp8"] else 1.0)
    s["out"].copy_(torch.where(l > 0, o / l, torch.zeros_like(o)).view(B, 1, Hq, d))
    s["lse"].copy_((m + l.log()).view(B, 1, Hq))


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def _outputs(s):
    c, op = s["case"], s["case"]["op"]
    if op == "tables":
        return [s[n] for n in ("page_table", "free_ring", "lens_out", "state_out", "cu", "positions", "slots")]
    if op == "attn":
        return [s["out"], s["lse"]]
    if op == "rope":
        return [s["q_out"], s["k_out"]]
    if op == "rope_bwd":
        return [s["dq"], s["dk"]] + ([s["dqw"], s["dkw"]] if c["norm"] else [])
    kind = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16  # (the values that the codes stand for)
    return [s["q_out"], s["k_pages"].view(kind), s["v_pages"].view(kind)]


def _run_own(s):
    import long_context_mqa_b200 as hs2
    c, op = s["case"], s["case"]["op"]
    if op == "tables":
        hs2.page_table_update(s["page_table"], s["lens"], s["delta"], s["free_ring"], s["free_state"], c["page"],
                              s["T"], lens_out=s["lens_out"], free_state_out=s["state_out"], cu_tokens=s["cu"],
                              positions=s["positions"], slots=s["slots"])
    elif op == "attn":
        more = {"k_scale": s["ks"], "v_scale": s["vs"]} if c["fp8"] else {}
        hs2.paged_attn(s["q"], s["k"], s["v"], s["page_table"], s["lens"], scale=s["scale"], window=c["window"],
                       out=s["out"], lse=s["lse"], **more)
    else:
        how = {"q_weight": s["qw"], "k_weight": s["kw"], "eps": EPS, "interleaved": c["interleaved"],
               "mscale": s["mscale"]}
        if op == "rope":
            hs2.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_out=s["q_out"], k_out=s["k_out"], **how)
        elif op == "rope_bwd":
            hs2.qk_norm_rope_bwd(s["q"], s["k"], s["positions"], s["inv_freq"], s["dq_out"], s["dk_out"], dq=s["dq"],
                                 dk=s["dk"], dq_weight=s["dqw"], dk_weight=s["dkw"], **how)
        else:
            if c["fp8"]:
                how.update(k_scale=s["ks"], v_scale=s["vs"])
            hs2.qk_norm_rope_paged(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pages"], s["v_pages"],
                                   s["inv_freq"], q_out=s["q_out"], **how)
    return _outputs(s)


def run(s):
    if own:
        return _run_own(s)
    c, op = s["case"], s["case"]["op"]
    if op == "tables":
        _tables(s)
    elif op == "attn":
        _attend(s)
    else:
        cos, sin = _angles(s, torch.float32)
        if op == "rope":
            s["q_out"].copy_(_norm_rope(s, s["q"], s["qw"], cos, sin))
            s["k_out"].copy_(_norm_rope(s, s["k"], s["kw"], cos, sin))
        elif op == "rope_bwd":
            dq, dqw = _norm_rope_bwd(s, s["q"], s["qw"], s["dq_out"], cos, sin)
            s["dq"].copy_(dq)
            del dq
            dk, dkw = _norm_rope_bwd(s, s["k"], s["kw"], s["dk_out"], cos, sin)
            s["dk"].copy_(dk)
            if c["norm"]:
                s["dqw"].copy_(dqw)
                s["dkw"].copy_(dkw)
        else:
            live = (s["slots"] >= 0)[:, None, None]
            s["q_out"].copy_(torch.where(live, _norm_rope(s, s["q"], s["qw"], cos, sin), s["q_out"].float()))
            k = _norm_rope(s, s["k"], s["kw"], cos, sin)
            _write_rows(s["k_pages"], s["slots"], _to_cache(k, s["ks"], c["fp8"]))
            _write_rows(s["v_pages"], s["slots"], _to_cache(s["v"], s["vs"], c["fp8"]))
    return _outputs(s)


# --------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# --------------------------------------------------------------------------------------------
def _exact_rows(s, x, w):
    """Rows [T, H, d] normalised and rotated, each pair as one complex number times m e^(i angle)."""
    c = s["case"]
    x, rot = x.double(), c["rot"]
    if w is not None:
        x = x / (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()
    t = torch.outer(s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.full_like(t, s["mscale"]), t)[:, None]
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        r = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        r = torch.cat([z.real, z.imag], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _exact_grads(s, x, w, dy):
    """The gradient of _exact_rows in blocks of tokens, by differentiating its 64-bit graph."""
    got, dw = [], None
    for i in range(0, x.shape[0], 4096):
        part = {**s, "positions": s["positions"][i:i + 4096]}
        xi = x[i:i + 4096].double().requires_grad_()
        leaves = [xi] if w is None else [xi, w.double().requires_grad_()]
        y = _exact_rows(part, xi, leaves[1] if w is not None else None)
        g = torch.autograd.grad(y, leaves, dy[i:i + 4096].double())
        got.append(g[0])
        if w is not None:
            dw = g[1] if dw is None else dw + g[1]
    return torch.cat(got), dw


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    if op == "attn":
        page, Hk, G, d = case["page"], case["Hk"], case["Hq"] // case["Hk"], case["d"]
        out = torch.zeros(case["B"], 1, case["Hq"], d, dtype=torch.float64, device="cuda")
        lse = torch.full((case["B"], 1, case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            at = torch.arange(first, n, device="cuda")
            page_of, in_page = s["page_table"][b, at // page].long(), at % page
            for h in range(Hk):
                k, v = s["k"][page_of, in_page, h], s["v"][page_of, in_page, h]
                if case["fp8"]:
                    k = k.view(torch.float8_e4m3fn).double() * s["ks"]
                    v = v.view(torch.float8_e4m3fn).double() * s["vs"]
                x = s["q"][b, 0, h * G:(h + 1) * G].double() @ k.double().T * s["scale"]
                lse[b, 0, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, 0, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v.double()
        return [out, lse]
    if op == "rope":
        return [_exact_rows(s, s["q"], s["qw"]), _exact_rows(s, s["k"], s["kw"])]
    if op == "rope_bwd":
        dq, dqw = _exact_grads(s, s["q"], s["qw"], s["dq_out"])
        dk, dkw = _exact_grads(s, s["k"], s["kw"], s["dk_out"])
        return [dq, dk] + ([dqw, dkw] if case["norm"] else [])
    live = s["slots"] >= 0
    q = torch.where(live[:, None, None], _exact_rows(s, s["q"], s["qw"]), s["q_out"].double())
    pools = []
    for pages, rows, scale in ((s["k_pages"], _exact_rows(s, s["k"], s["kw"]), s["ks"]),
                               (s["v_pages"], s["v"].double(), s["vs"])):
        pool = (pages.view(torch.float8_e4m3fn) if case["fp8"] else pages).double()
        at = s["slots"][live].long()
        rows = rows / scale if case["fp8"] else rows
        pool[at // case["page"], at % case["page"]] = rows[live].clamp(-448, 448) if case["fp8"] else rows[live]
        pools.append(pool)
    return [q, *pools]
