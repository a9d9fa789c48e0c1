"""The serving side of the softmax-attention layers, and their rotary positions: measured cases.

Four operators of gated_deltanet_dual_b200.binding, each with its plain form in elementary torch
operations: kv_extend (block tables and slot maps from request lengths), rotary_forward and
rotary_backward, rotary_append (rotary fused with the write into the paged key/value cache), and
prefix_attention (attention over a paged cache whose sequences share a long prefix).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 running requests: one new token each (the smallest call)
        dict(name="tables_64_decode", op="tables", n=64, page=16, longest=4096, new_most=1, prefix=512, lens=1),
        # a scheduler step that mixes decode steps with prompt chunks of up to 256 tokens
        dict(name="tables_1024_mixed", op="tables", n=1024, page=64, longest=8192, new_most=256, prefix=0, lens=2),
        # the training layout of the softmax layers: 8 x 4096 tokens, 16 heads, whole heads rotated
        dict(name="rotary_train_8x4096_h16", op="rotary", back=False, views=1, rows=32768, heads=16, kv_heads=16, d=128,
             rot=128, interleaved=False, dtype="bf16", scaling="none", factor=1.0, start=0),
        # gradients of both noisy views, grouped heads, half of each head rotated in pairs, long-context
        # frequencies, an odd number of rows
        dict(name="rotary_back_views_h32kv8", op="rotary", back=True, views=2, rows=6147, heads=32, kv_heads=8, d=128,
             rot=64, interleaved=True, dtype="fp32", scaling="ramp", factor=8.0, start=100000),
        # one decode step of 64 requests: rotate q and k, append k and v to the cache
        dict(name="append_64_decode", op="append", rows=64, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             page=16, padded=0, scaling="none", factor=1.0, start=3000),
        # a packed prefill of about 8192 tokens with padding rows behind the last request
        dict(name="append_8192_prefill", op="append", rows=8192, heads=32, kv_heads=8, d=128, rot=128,
             interleaved=False, page=64, padded=77, scaling="linear", factor=4.0, start=20000),
        # one request alone: the smallest attention call
        dict(name="attn_1_alone", op="attn", n=1, l=1, heads=16, kv_heads=16, d=128, page=16, prefix=512, longest=64,
             causal=True, lens=3),
        # 64 requests that share instructions of 8192 tokens, one token each
        dict(name="attn_64_decode", op="attn", n=64, l=1, heads=32, kv_heads=8, d=128, page=16, prefix=8192, longest=1024,
             causal=True, lens=4),
        # many requests on one shared document: the prefix is bound by the tensor cores
        dict(name="attn_256_decode", op="attn", n=256, l=1, heads=32, kv_heads=8, d=128, page=64, prefix=16384,
             longest=512, causal=True, lens=5),
        # block denoising: every token of a block of 4 sees the whole block, long shared prefix
        dict(name="attn_32_block4", op="attn", n=32, l=4, heads=32, kv_heads=8, d=128, page=64, prefix=32768, longest=2048,
             causal=False, lens=6),
        # verifying 8 drafted tokens, ungrouped heads of 64, odd prefix, ragged requests
        dict(name="attn_24_verify8_d64", op="attn", n=24, l=8, heads=16, kv_heads=16, d=64, page=32, prefix=1001,
             longest=4096, causal=True, lens=7),
        # long answers on a short prefix: the requests' own keys dominate
        dict(name="attn_32_long_answers", op="attn", n=32, l=1, heads=32, kv_heads=8, d=128, page=128, prefix=257,
             longest=16384, causal=True, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "append", "attn", "attn"])
    if op == "tables":
        return dict(op=op, n=_log(rng, 1, 1500), page=rng.choice([16, 32, 64, 128]), longest=_log(rng, 64, 16384),
                    new_most=_log(rng, 1, 170), prefix=rng.choice([0, _log(rng, 1, 32768)]), lens=rng.randrange(1 << 20))
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads <= 4 else [1, 2, 4] if kv_heads == 8 else [1, 2])
    rot = rng.choice([d, d, d // 2, d // 4])
    scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 4.0), ("ramp", 8.0), ("ramp", 32.0)])
    if op == "rotary":
        back, dtype, views = rng.random() < 0.5, rng.choice(["bf16", "fp32"]), rng.choice([1, 1, 2])
        most = 32768 * 32 * 128 * 2 // ((heads + kv_heads) * d * views * (2 if dtype == "bf16" else 4))
        return dict(op=op, back=back, views=views, rows=_log(rng, 1, min(most, 40000)), heads=heads, kv_heads=kv_heads,
                    d=d, rot=rot, interleaved=rng.random() < 0.5, dtype=dtype, scaling=scaling, factor=factor,
                    start=rng.choice([0, _log(rng, 1, 1000000)]))
    if op == "append":
        rows = _log(rng, 1, 16384)
        return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, d=d, rot=rot, interleaved=rng.random() < 0.5,
                    page=rng.choice([16, 32, 64, 128]), padded=rng.choice([0, rng.randrange(0, rows)]),
                    scaling=scaling, factor=factor, start=rng.choice([0, _log(rng, 1, 1000000)]))
    l = rng.choice([1, 1, 1, 2, 4, 8])
    n = _log(rng, 1, 256 // l)
    longest = _log(rng, 16, max(16, min(16384, 2000000 // n // kv_heads)))
    prefix = rng.choice([0, _log(rng, 16, max(16, min(65536, 16384 * 8192 // (n * l * heads))))])
    return dict(op=op, n=n, l=l, heads=heads, kv_heads=kv_heads, d=d, page=rng.choice([16, 32, 64, 128]), prefix=prefix,
                longest=max(l, longest), causal=rng.random() < 0.6, lens=rng.randrange(1 << 20))


# ---------------------------------------------------------------------------------- the inputs
def _lengths(case, least):
    """The requests' cached lengths, the same multiset for every seed (so the work is the case's)."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(least, case["longest"]) for _ in range(case["n"])]
    lens[0] = case["longest"]
    return lens


def _new_lengths(case):
    """New tokens per request: half of the requests decode one token, the others bring prompt chunks."""
    rng = random.Random(case["lens"] + 7)
    return [1 if i % 2 == 0 else rng.randint(0, case["new_most"]) for i in range(case["n"])]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def _frequencies(case):
    """Frequencies in 64 bits and the scale of the rotated part, by the scaling's definition."""
    rot, factor = case["rot"], case["factor"]
    base, scale = 10000.0, 1.0
    if case["scaling"] == "ntk":
        base *= factor ** (rot / (rot - 2.0))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "ramp":   # by the turns that a pair makes over the original context of 8192 tokens
        w = ((8192.0 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (w + (1.0 - w) / factor)
        scale = 0.1 * math.log(factor) + 1.0
    return f, scale


def _table(case):
    from gated_deltanet_dual_b200 import binding as gdn
    return gdn.rotary_table(case["rot"], interleaved=case["interleaved"], base=10000.0, scaling=case["scaling"],
                            factor=case["factor"], original_len=8192)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    normal = lambda *s, dtype=torch.bfloat16, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(dtype)  # noqa: E731
    i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)                                        # noqa: E731
    s = {"case": case}
    if case["op"] == "tables":
        n, page = case["n"], case["page"]
        order = host.permutation(n)
        lens, new = np.array(_lengths(case, 0))[order], np.array(_new_lengths(case))[host.permutation(n)]
        width = _pages(case["longest"] + case["new_most"] + 1, page)
        ids = host.permutation(n * width + 64)
        used = _pages(lens, page)
        table = ids[:n * width].reshape(n, width).copy()
        table[np.arange(width)[None, :] >= used[:, None]] = -1
        s.update(table=i32(table), lens=i32(lens), new=i32(new), free=i32(host.permutation(n * width + 64)[:n * width]),
                 count=i32([n * width - 5 if n * width > 5 + n * _pages(case["new_most"] + 1, page) else n * width]),
                 room=int(np.sum(_new_lengths(case))) + 3)
        if own:
            from gated_deltanet_dual_b200 import binding as gdn
            s["out"] = gdn.KvTables(n, s["room"], DEV)
    elif case["op"] == "rotary":
        dtype, v, t = TYPES[case["dtype"]], case["views"], case["rows"]
        s.update(q=normal(v, t, case["heads"], case["d"], dtype=dtype), k=normal(v, t, case["kv_heads"], case["d"], dtype=dtype),
                 pos=i32(case["start"] + host.integers(0, 8) + np.arange(t) % 4096))
        if not own:
            s["freq"], s["scale"] = _frequencies(case)
            s["freq"] = s["freq"].to(DEV)
        else:
            s["rope"] = _table(case)
    elif case["op"] == "append":
        t, h, hk, d, page = case["rows"], case["heads"], case["kv_heads"], case["d"], case["page"]
        live = t - case["padded"]
        pages = _pages(t, page) + 8
        qkv = normal(t, h + 2 * hk, d)      # one projection's output: q, k and v are slices of its rows
        s.update(q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:],
                 k_cache=torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device=DEV),
                 v_cache=torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device=DEV),
                 q_out=torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEV))
        slots, pos = np.full(t, -1), np.full(t, -1)
        ids = host.permutation(pages)       # requests fill their pages in order, the pages lie anywhere
        slots[:live] = ids[np.arange(live) // page] * page + np.arange(live) % page
        pos[:live] = case["start"] + np.arange(live)
        s.update(slots=i32(slots), pos=i32(pos), freq=_frequencies(case)[0].to(DEV), scale=_frequencies(case)[1])
        if own:
            s["rope"] = _table(case)
    else:
        n, hk, d, page = case["n"], case["kv_heads"], case["d"], case["page"]
        lens = np.array(_lengths(case, case["l"]))[host.permutation(n)]
        width = _pages(case["longest"], page)
        used = _pages(lens, page)
        own_pages, first = int(used.sum()), _pages(case["prefix"], page)
        ids = host.permutation(own_pages + first + 3)
        table = np.full((n, width), -1)
        table[np.arange(width)[None, :] < used[:, None]] = ids[first:first + own_pages]
        # keys around the queries' scale: scores of a few units, so that some keys carry most of a row
        s.update(q=normal(n, case["l"], case["heads"], d, std=2.0), k_cache=normal(len(ids), page, hk, d),
                 v_cache=normal(len(ids), page, hk, d), prefix_pages=i32(ids[:first]), table=i32(table), lens=i32(lens))
        if own:
            from gated_deltanet_dual_b200 import binding as gdn
            desc = gdn.make_prefix_attn_desc(n, case["l"], case["heads"], hk, d, page, len(ids), width, case["prefix"],
                                             case["causal"])
            s["ws"] = gdn.Workspace(gdn.prefix_attn_workspace_size(desc), device=DEV)
    return s


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return RUN[s["case"]["op"]](s)


def _run_tables(s):
    case, page = s["case"], s["case"]["page"]
    if own:
        from gated_deltanet_dual_b200 import binding as gdn
        o = gdn.kv_extend(s["table"], s["lens"], s["new"], s["free"], s["count"], page, s["out"], prefix_len=case["prefix"])
        return [s["table"], o.slot_map, o.positions, o.cu_new, o.seq_lens, o.free_left]
    table, lens, new = s["table"], s["lens"].long(), s["new"].long()
    n, width = table.shape
    have = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - have
    before = torch.cumsum(need, 0) - need
    column = torch.arange(width, device=DEV)[None, :]
    k = before[:, None] + column - have[:, None]            # which free page a new entry takes
    fresh = (column >= have[:, None]) & (column < (have + need)[:, None])
    taken = s["free"][(s["count"].long() - 1 - k).clamp(0, s["free"].numel() - 1)]
    table.copy_(torch.where(fresh, taken, table))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    token = torch.arange(s["room"], device=DEV)
    seq = (torch.searchsorted(cu, token, right=True) - 1).clamp(0, n - 1)
    at = lens[seq] + token - cu[seq]
    live = token < cu[n]
    slot = table[seq, (at // page).clamp(0, width - 1)].long() * page + at % page
    none = torch.full_like(slot, -1)
    return [table, torch.where(live, slot, none).int(), torch.where(live, at + case["prefix"], none).int(), cu.int(),
            (lens + new).int(), (s["count"].long() - need.sum()).int()]


def _rotate(x, pos, freq, scale, case, sign):
    """x [..., T, H, d] rotated by sign * pos * freq over its first `rot` elements, in 32 bits (angles in 64)."""
    rot, y = case["rot"], x.float()
    angle = pos.double()[:, None] * freq[None, :] * sign
    cos, sin = (torch.cos(angle) * scale).float()[:, None, :], (torch.sin(angle) * scale).float()[:, None, :]
    head, rest = y[..., :rot], y[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, rest], dim=-1).to(x.dtype)


def _run_rotary(s):
    case = s["case"]
    if own:
        from gated_deltanet_dual_b200 import binding as gdn
        call = gdn.rotary_backward if case["back"] else gdn.rotary_forward
        return list(call(s["q"], s["k"], s["pos"], s["rope"]))
    sign = -1.0 if case["back"] else 1.0
    return [_rotate(s[x], s["pos"], s["freq"], s["scale"], case, sign) for x in ("q", "k")]


def _run_append(s):
    if own:
        from gated_deltanet_dual_b200 import binding as gdn
        gdn.rotary_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["rope"], s["k_cache"], s["v_cache"], q_out=s["q_out"])
    else:
        case = s["case"]
        live = s["slots"] >= 0
        at = s["slots"].long()[live]
        q, k = (_rotate(s[x], s["pos"], s["freq"], s["scale"], case, 1.0) for x in ("q", "k"))
        s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
        s["k_cache"].flatten(0, 1)[at] = k[live]
        s["v_cache"].flatten(0, 1)[at] = s["v"][live]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _run_attn(s):
    case = s["case"]
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    if own:
        from gated_deltanet_dual_b200 import binding as gdn
        return gdn.prefix_attention(q, kc, vc, s["prefix_pages"], case["prefix"], s["table"], s["lens"],
                                    causal=case["causal"], workspace=s["ws"])
    n, l, h, d = q.shape
    hk, lp, width = kc.shape[2], case["prefix"], s["table"].shape[1] * case["page"]
    g = h // hk
    qf = q.float().reshape(n, l, hk, g, d) / math.sqrt(d)
    # the shared prefix, once for all requests: [hk, n l g, d] x [hk, d, lp]
    kp = kc[s["prefix_pages"].long()].flatten(0, 1)[:lp].float()
    vp = vc[s["prefix_pages"].long()].flatten(0, 1)[:lp].float()
    sp = qf.permute(2, 0, 1, 3, 4).reshape(hk, n * l * g, d) @ kp.permute(1, 2, 0)
    sp = sp.reshape(hk, n, l * g, lp).transpose(0, 1)
    # each request's own keys: [n, hk, l g, d] x [n, hk, d, width]
    at = s["table"].long().clamp(min=0)
    ko, vo = kc[at].flatten(1, 2).float(), vc[at].flatten(1, 2).float()
    so = qf.permute(0, 2, 1, 3, 4).reshape(n, hk, l * g, d) @ ko.permute(0, 2, 3, 1)
    last = torch.arange(l, device=DEV) - (l - 1) if case["causal"] else torch.zeros(l, dtype=torch.long, device=DEV)
    sees = torch.arange(width, device=DEV)[None, None, :] < (s["lens"].long()[:, None] + last[None, :])[:, :, None]
    so = so.masked_fill(~sees[:, None, :, None, :].expand(n, hk, l, g, width).reshape(n, hk, l * g, width), -math.inf)
    top = torch.maximum(so.amax(-1, keepdim=True), sp.amax(-1, keepdim=True)) if lp else so.amax(-1, keepdim=True)
    po, pp = torch.exp(so - top), torch.exp(sp - top)
    total = po.sum(-1, keepdim=True) + pp.sum(-1, keepdim=True)
    o = po @ vo.transpose(1, 2)
    o = o + (pp.transpose(0, 1).reshape(hk, n * l * g, lp) @ vp.transpose(0, 1)).reshape(hk, n, l * g, d).transpose(0, 1)
    return (o / total).reshape(n, hk, l, g, d).transpose(1, 2).reshape(n, l, h, d).to(q.dtype)


RUN = {"tables": _run_tables, "rotary": _run_rotary, "append": _run_append, "attn": _run_attn}


# ---------------------------------------------------------------------------------- the work
def work(case):
    if case["op"] == "tables":
        n, tokens, page = case["n"], sum(_new_lengths(case)), case["page"]
        # lengths in, slots, positions, sums and lengths out, one free page read and one entry written per new page
        return {"bytes": 8 * n + 8 * tokens + 8 * n + 8 * _pages(tokens, page), "flops": 0}
    if case["op"] == "rotary":
        values = case["views"] * case["rows"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * values * case["d"] * (2 if case["dtype"] == "bf16" else 4) + 4 * case["rows"],
                "flops": 3 * values * case["rot"]}
    if case["op"] == "append":
        rows = case["rows"] - case["padded"]
        return {"bytes": rows * (4 * (case["heads"] + 2 * case["kv_heads"]) * case["d"] + 8),
                "flops": 3 * rows * (case["heads"] + case["kv_heads"]) * case["rot"]}
    n, l, h, hk, d, lens = case["n"], case["l"], case["heads"], case["kv_heads"], case["d"], _lengths(case, case["l"])
    keys = case["prefix"] + sum(lens)
    pairs = h * l * (n * case["prefix"] + sum(lens) - (n * (l - 1) // 2 if case["causal"] else 0))
    return {"bytes": 4 * keys * hk * d + 4 * n * l * h * d + 4 * n, "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "rotary":
        sign = -1.0 if case["back"] else 1.0
        return [_exact_rotate(s[x], s["pos"], case, sign) for x in ("q", "k")]
    if case["op"] == "append":
        live = torch.nonzero(s["slots"] >= 0).flatten()
        q, kc, vc = s["q_out"].double(), s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
        q[live] = _exact_rotate(s["q"][live], s["pos"][live], case, 1.0)
        kc[s["slots"][live].long()] = _exact_rotate(s["k"][live], s["pos"][live], case, 1.0)
        vc[s["slots"][live].long()] = s["v"][live].double()
        return [q, kc.reshape(s["k_cache"].shape), vc.reshape(s["v_cache"].shape)]
    return _exact_attn(s)


def _exact_tables(s):
    """Request by request and page by page, as an allocator on the host would."""
    case, page = s["case"], s["case"]["page"]
    table, free = s["table"].cpu().numpy().astype(np.int64), s["free"].cpu().tolist()
    lens, new, left = s["lens"].cpu().tolist(), s["new"].cpu().tolist(), int(s["count"].item())
    slots, where, cu = [], [], [0]
    for r in range(case["n"]):
        for i in range(lens[r], lens[r] + new[r]):
            if i % page == 0:
                left -= 1
                table[r, i // page] = free[left]
            slots.append(int(table[r, i // page]) * page + i % page)
            where.append(case["prefix"] + i)
        cu.append(cu[-1] + new[r])
    pad = [-1] * (s["room"] - len(slots))
    answer = [table, slots + pad, where + pad, cu, [a + b for a, b in zip(lens, new)], [left]]
    return [torch.tensor(np.asarray(a), dtype=torch.int32) for a in answer]


def _exact_rotate(x, pos, case, sign):
    """The rotation as a product of complex numbers; the angle is reduced by whole turns in 64 bits."""
    rot = case["rot"]
    f, scale = _frequencies(case)
    turns = pos.to(torch.float64).unsqueeze(1) * (f.to(DEV) / (2 * math.pi)).unsqueeze(0)
    turns = turns - torch.round(turns)
    unit = torch.polar(torch.full_like(turns, scale), 2 * math.pi * sign * turns).unsqueeze(1)
    y = x.to(torch.float64)
    if case["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * unit
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_attn(s):
    """Request by request over its whole list of keys, prefix and own together."""
    case, q = s["case"], s["q"]
    n, l, h, d = q.shape
    hk, lp, page = s["k_cache"].shape[2], case["prefix"], case["page"]
    if 2 * n * l * h * (lp + case["longest"]) * d > 4e11 or n * (lp + case["longest"]) * hk * d > 2e10:
        return None
    rows_of = lambda pages, count: (pages.long()[:, None] * page + torch.arange(page, device=DEV)).flatten()[:count]  # noqa: E731
    first = rows_of(s["prefix_pages"], lp)
    k_all, v_all = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    out = torch.empty(n, l, h, d, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for r in range(n):
        keys = torch.cat([first, rows_of(s["table"][r], lens[r])])
        k, v = k_all[keys].double().transpose(0, 1), v_all[keys].double().transpose(0, 1)      # [hk, keys, d]
        x = q[r].double().reshape(l, hk, h // hk, d).permute(1, 0, 2, 3).reshape(hk, -1, d)
        score = torch.bmm(x, k.transpose(1, 2)).reshape(hk, l, h // hk, -1) * d ** -0.5
        for i in range(l if case["causal"] else 0):
            score[:, i, :, lp + max(0, lens[r] - (l - 1 - i)):] = -math.inf
        weight = torch.softmax(score, dim=-1).reshape(hk, l * (h // hk), -1)
        out[r] = torch.bmm(weight, v).reshape(hk, l, h // hk, d).permute(1, 0, 2, 3).reshape(l, h, d)
    return out
