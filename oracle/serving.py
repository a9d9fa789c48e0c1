"""fp64 oracle of the serving side of the softmax layers (include/gdn_rotary.h, include/gdn_kvcache.h).

numpy, written from the definitions, sharing no code with the CUDA library: rotary frequencies and the
rotation, block tables and slots as a page-by-page allocator, the append to the paged cache, and
attention row by row over each row's own list of visible keys."""
from __future__ import annotations

import math

import numpy as np


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def ints(t) -> np.ndarray:
    return t.detach().cpu().numpy().astype(np.int64) if hasattr(t, "detach") else np.asarray(t, dtype=np.int64)


# ----------------------------------------------------------------------------- rotary
def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of every pair."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "ramp":
        out = []
        for x in f:
            turns = original_len * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
            out.append(keep * x + (1.0 - keep) * x / factor)
        return np.array(out)
    return f


def rotate(x, positions, freq, *, interleaved=False, scale=1.0, sign=1.0):
    """x [..., T, H, d] with the first 2 len(freq) elements of every head rotated to its position."""
    x = f64(x).copy()
    n = len(freq)
    turns = ints(positions)[:, None].astype(np.longdouble) * (np.asarray(freq, np.longdouble) / (2 * np.longdouble(math.pi)))
    t = (2 * math.pi * (turns - np.rint(turns))).astype(np.float64) * sign
    c, s = scale * np.cos(t)[:, None, :], scale * np.sin(t)[:, None, :]
    i1 = np.arange(n) * 2 if interleaved else np.arange(n)
    i2 = i1 + 1 if interleaved else i1 + n
    a, b = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1], x[..., i2] = a * c - b * s, a * s + b * c
    return x


# ----------------------------------------------------------------------------- block tables
def kv_extend(table, lens, new, free, count, page, rows, prefix_len=0):
    """Returns dict(table, slot_map, positions, cu, lens, left, bad)."""
    table, lens, new, free = ints(table).copy(), ints(lens), ints(new), ints(free)
    n_seq, width = table.shape
    top = min(max(int(count), 0), len(free))
    bad = top != int(count)
    slots, pos = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    cu, out_lens, wanted, taken, at = [0], [], 0, 0, 0
    for n in range(n_seq):
        s, w = int(lens[n]), int(new[n])
        refused = s < 0 or w < 0 or s + w > min(width * page, 2 ** 31 - 1)
        w = max(w, 0)
        refused = refused or at + w > rows
        if not refused:
            need = -(-(s + w) // page) - -(-s // page)
            wanted += need
            refused = need > 0 and wanted > top
        if refused:
            bad = True
            out_lens.append(s)
        else:
            first = wanted - need
            taken = wanted if need else taken
            for j in range(need):
                table[n, -(-s // page) + j] = free[top - 1 - first - j]
            for i in range(w):
                slots[at + i] = table[n, (s + i) // page] * page + (s + i) % page
                pos[at + i] = prefix_len + s + i
            out_lens.append(s + w)
        at += w
        cu.append(at)
    return dict(table=table, slot_map=slots, positions=pos, cu=np.array(cu), lens=np.array(out_lens), left=top - taken,
                bad=bad)


# ----------------------------------------------------------------------------- append
def append(q, k, v, positions, slots, freq, k_cache, v_cache, q_out, *, interleaved=False, scale=1.0):
    """(q_out, k_cache, v_cache) after the append; rows with a negative slot change nothing."""
    slots = ints(slots)
    qr = rotate(q, positions, freq, interleaved=interleaved, scale=scale)
    kr = rotate(k, positions, freq, interleaved=interleaved, scale=scale)
    q_out, kc, vc, v = f64(q_out).copy(), f64(k_cache).copy(), f64(v_cache).copy(), f64(v)
    shape = kc.shape
    kc, vc = kc.reshape((-1,) + shape[2:]), vc.reshape((-1,) + shape[2:])
    for r, s in enumerate(slots):
        if s >= 0:
            q_out[r], kc[s], vc[s] = qr[r], kr[r], v[r]
    return q_out, kc.reshape(shape), vc.reshape(shape)


# ----------------------------------------------------------------------------- attention
def visible_own(length, l, tokens, causal):
    """How many of its own keys token l of a sequence sees."""
    return max(0, length - (tokens - 1 - l)) if causal else length


def prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, table, lens, *, causal=True, scale=None):
    """(out, spread, reach): the rows' outputs, sum_j w_j |v_j| of every output element (what a relative error of
    the weights can move), and the largest scale * sum_i |q_i k_i| of every row (what bounds the
    rounding of its scores)."""
    q, kc, vc = f64(q), f64(k_cache), f64(v_cache)
    table, lens = ints(table), ints(lens)
    n_seq, tokens, heads, d = q.shape
    page, kv_heads = kc.shape[1], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, spread = np.zeros_like(q), np.zeros_like(q)
    reach = np.zeros(q.shape[:3])
    first = [int(p) * page + o for p in ints(prefix_pages) for o in range(page)][:prefix_len] if prefix_len else []
    kc, vc = kc.reshape(-1, kv_heads, d), vc.reshape(-1, kv_heads, d)
    for n in range(n_seq):
        own = [int(table[n, i // page]) * page + i % page for i in range(int(lens[n]))]
        for l in range(tokens):
            keys = first + own[:visible_own(int(lens[n]), l, tokens, causal)]
            if not keys:
                continue
            for h in range(heads):
                k, v = kc[keys, h // (heads // kv_heads)], vc[keys, h // (heads // kv_heads)]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (k @ q[n, l, h])
                    w = np.exp(x - x.max())
                    w = w / w.sum()
                    out[n, l, h] = w @ v
                    spread[n, l, h] = w @ np.abs(v)
                    reach[n, l, h] = scale * (np.abs(k) @ np.abs(q[n, l, h])).max()
    return out, spread, reach
