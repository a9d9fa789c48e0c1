"""Attention with a shared prefix (gdn_prefix_attn) on the GPU against the fp64 oracle, element by element.

Tolerance of one output element o = sum_j w_j v_j, derived from the arithmetic: the weights enter the second
product as bf16 (half a step, 2^-8 relative); a score of d products is summed in fp32, off by at
most d 2^-24 times reach = scale sum |q k|, which moves a weight and the sum of weights by as much
each; exponentials, the sums over keys and the joining of parts are fp32 (1e-4 covers them at these lengths:
below 2^10 roundings of 2^-24); the output is rounded once, 2^-8 |o|."""
import numpy as np
import pytest
import torch

from gated_deltanet_dual_b200 import binding as b
from oracle import serving as o

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _problem(N, L, H, Hkv, d, page, prefix, lens, W=None, seed=0, std=1.0, spare=3):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    used = [-(-n // page) for n in lens]
    W = max(used + [0]) if W is None else W
    first = -(-prefix // page)
    P = sum(used) + first + spare
    ids = rng.permutation(P)
    table = np.full((N, W), -1)
    at = first
    for n, u in enumerate(used):
        table[n, :u] = ids[at:at + u]
        at += u
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(q=(normal(N, L, H, d) * std).to(torch.bfloat16), k_cache=normal(P, page, Hkv, d).to(torch.bfloat16),
                v_cache=normal(P, page, Hkv, d).to(torch.bfloat16), prefix_pages=_i32(ids[:first]), prefix_len=prefix,
                block_table=_i32(table).reshape(N, W), seq_lens=_i32(lens))


def _oracle(p, causal, scale=None):
    return o.prefix_attention(p["q"], p["k_cache"], p["v_cache"], p["prefix_pages"], p["prefix_len"], p["block_table"],
                              p["seq_lens"], causal=causal, scale=scale)


def _close(got, want, d, what=""):
    ref, spread, reach = want
    got = o.f64(got)
    eps = 2.0 ** -8 + 2 * d * 2.0 ** -24 * reach[..., None] + 1e-4
    bound = eps * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
    ok = np.where(np.isfinite(ref), np.abs(got - ref) <= bound, (got == ref) | (np.isnan(got) & np.isnan(ref)))
    assert np.all(ok), f"{what}: {np.nanmax((np.abs(got - ref) / bound)[np.isfinite(ref)]):.3f} of the bound, {np.argwhere(~ok)[:4].tolist()}"


def _run(p, causal, **kw):
    ws = kw.pop("workspace", None) or b.Workspace(1 << 26)
    out = b.prefix_attention(**p, causal=causal, workspace=ws, **kw)
    assert b.read_device_status(ws) == b.GDN_OK
    return out


CASES = [
    # N, L, H, Hkv, d, page, prefix, lens
    (1, 1, 1, 1, 128, 16, 0, [1]),
    (1, 1, 1, 1, 64, 16, 1, [0]),
    (1, 1, 4, 1, 128, 16, 17, [3]),
    (2, 1, 4, 2, 64, 32, 130, [127, 129]),
    (3, 1, 8, 2, 128, 64, 128, [128, 1, 0]),
    (3, 1, 8, 8, 128, 128, 255, [400, 256, 257]),
    (4, 1, 16, 2, 64, 256, 300, [513, 12, 0, 255]),
    (5, 2, 6, 3, 128, 16, 33, [2, 7, 100, 16, 1]),
    (2, 4, 4, 1, 128, 16, 0, [4, 333]),
    (2, 8, 16, 4, 64, 16, 100, [8, 65]),
    (2, 17, 8, 1, 128, 32, 64, [17, 150]),          # 136 rows of a sequence: two row tiles
    (1, 64, 8, 1, 64, 16, 40, [200]),               # 512 rows: two CTAs
    (40, 1, 16, 2, 64, 16, 500, None),              # 320 rows of a key/value head share the prefix
    (33, 1, 32, 2, 128, 16, 1000, None),            # 528 rows: three row-tile CTAs, the last with 16 rows
    (300, 1, 2, 1, 64, 16, 20, None),
    (9, 3, 4, 4, 128, 64, 2000, None),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(case, causal):
    N, L, H, Hkv, d, page, prefix, lens = case
    if lens is None:
        lens = np.random.default_rng(N).integers(0, 70, N).tolist()
    p = _problem(N, L, H, Hkv, d, page, prefix, lens, seed=N + d)
    _close(_run(p, causal), _oracle(p, causal), d)


@pytest.mark.parametrize("d", [64, 128])
def test_long_keys_and_splits(d):
    p = _problem(2, 1, 2, 1, d, 64, 9001, [5000, 4097], seed=1)
    _close(_run(p, True), _oracle(p, True), d)
    wide = _problem(3, 2, 2, 2, d, 16, 0, [700, 3, 0], W=4096, seed=2)     # a table far wider than the lengths
    _close(_run(wide, True), _oracle(wide, True), d)


@pytest.mark.parametrize("std", [0.0, 30.0])
def test_flat_and_peaked_scores(std):
    """All scores equal; and scores of hundreds (the running reference max moves from tile to tile)."""
    p = _problem(3, 2, 4, 2, 128, 32, 700, [300, 900, 2], seed=3, std=std)
    _close(_run(p, True), _oracle(p, True), 128)
    grow = _problem(1, 1, 2, 1, 128, 16, 512, [640], seed=4)
    ramp = torch.linspace(0, 8, grow["k_cache"].shape[0], device="cuda").bfloat16()      # scores that grow page by page
    order = torch.cat([grow["prefix_pages"], grow["block_table"][0]]).long()
    scale = torch.empty_like(ramp)
    scale[order] = ramp[:order.numel()]
    grow["k_cache"] = (grow["q"].mean(2).reshape(1, 1, 1, 128) * scale[:, None, None, None]).expand(-1, 16, 1, 128).contiguous()
    _close(_run(grow, True), _oracle(grow, True), 128)


def test_scale_argument():
    p = _problem(2, 1, 4, 2, 64, 16, 50, [20, 0], seed=5)
    _close(_run(p, True, scale=0.5), _oracle(p, True, scale=0.5), 64)
    with pytest.raises(ValueError):
        b.prefix_attention(**p, scale=0.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("L,G,d", [(1, 4, 128), (4, 2, 128), (5, 1, 64), (8, 8, 64)])
def test_what_is_not_seen_changes_nothing(causal, L, G, d):
    """NaN and infinities behind the last tokens, behind the prefix and on pages of nobody."""
    p = _problem(3, L, 2 * G, 2, d, 32, 70, [L, 130, 33], seed=6)
    want = _run(p, causal)
    for bad in (float("nan"), float("inf"), -float("inf")):
        used = torch.zeros(p["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
        for i in range(70):
            used[p["prefix_pages"][i // 32], i % 32] = True
        for n, s in enumerate(p["seq_lens"].tolist()):
            for i in range(s):
                used[p["block_table"][n, i // 32], i % 32] = True
        dirty = dict(p, k_cache=torch.where(used[..., None, None], p["k_cache"], bad).bfloat16(),
                     v_cache=torch.where(used[..., None, None], p["v_cache"], bad).bfloat16())
        assert torch.equal(_run(dirty, causal), want)


@pytest.mark.parametrize("L,H,Hkv,d", [(3, 4, 2, 128), (6, 8, 1, 64), (20, 8, 1, 128)])
def test_values_that_some_rows_see(L, H, Hkv, d):
    """Non-finite values among the newest tokens of a causal call reach the rows that see them, no others."""
    p = _problem(2, L, H, Hkv, d, 16, 20, [40 + L, L], seed=7)
    at = lambda n, i: (int(p["block_table"][n, i // 16]), i % 16)
    for n, i, c, x in ((0, 40 + L - 1, 3, float("inf")), (0, 40 + L - 2, 5, -float("inf")), (0, 40 + L - 1, 5, float("inf")),
                       (1, L - 1, 0, float("nan")), (1, 1, 7, float("nan"))):
        pg, off = at(n, i)
        p["v_cache"][pg, off, 0, c] = x
    want = _oracle(p, True)
    # weights of 0 in the oracle's matrix product of one row never meet a masked value: the row's own list
    _close(_run(p, True), want, d)
    pg, off = at(0, 40 + L - 1)
    p["k_cache"][pg, off, 0, 0] = float("nan")
    got = o.f64(_run(p, True))
    seen = np.isnan(got[0, :, :H // Hkv]).all(axis=(1, 2))
    assert seen.tolist() == [False] * (L - 1) + [True]


def test_nan_queries_stay_in_their_rows():
    p = _problem(3, 2, 4, 2, 128, 16, 150, [9, 40, 5], seed=8)
    want = _run(p, True)
    p["q"][1, 0, 2] = float("nan")
    got = _run(p, True)
    assert torch.isnan(got[1, 0, 2]).all()
    got[1, 0, 2] = want[1, 0, 2]
    assert torch.equal(got, want)


def test_rows_that_see_nothing_are_zero():
    p = _problem(3, 4, 2, 1, 128, 16, 0, [0, 2, 5], seed=9)
    out = _run(p, True)
    assert int(torch.count_nonzero(out[0])) == 0 and int(torch.count_nonzero(out[1, :2])) == 0
    assert torch.count_nonzero(out[1, 2:]) > 0
    _close(out, _oracle(p, True), 128)
    empty = _problem(2, 1, 2, 1, 64, 16, 0, [0, 0], W=0, seed=9)
    assert int(torch.count_nonzero(_run(empty, True))) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L,G,prefix", [(2, 1, 2, 0), (2, 1, 2, 40), (3, 17, 1, 0), (20, 1, 2, 300), (2, 20, 2, 200)])
def test_scores_without_bound(N, L, G, prefix, d):
    """Scores of -inf and +inf, by infinite queries and keys: as softmax has them, for few rows and for many."""
    own = 180
    p = _problem(N, L, 2 * G, 2, d, 16, prefix, [own] * N, seed=22)
    one = dict(p, q=p["q"].clone(), k_cache=p["k_cache"].clone())
    one["k_cache"][..., 0] = 1.0
    one["q"][0, 0, 0, 0], one["q"][N - 1, L - 1, G, 0] = -float("inf"), float("inf")
    got = _run(one, True)
    _close(got, _oracle(one, True), d)
    assert torch.isnan(got[0, 0, 0]).all() and torch.isnan(got[N - 1, L - 1, G]).all()
    some = dict(p, k_cache=p["k_cache"].clone(), q=p["q"].clone())             # one list of keys without bound
    some["q"][..., 0] = 1.0
    some["k_cache"][(p["prefix_pages"] if prefix else p["block_table"][0]).long(), :, 0, 0] = -float("inf")
    want = _oracle(some, True)
    _close(_run(some, True), want, d)
    assert np.isnan(want[0]).any() == (prefix == 0)
    if prefix:                                                                 # the own keys alone
        none = dict(some, prefix_len=0)
        assert torch.equal(_run(some, False)[:, :, :G], _run(none, False)[:, :, :G])


def test_bad_lengths_and_pages_are_reported():
    p = _problem(4, 1, 2, 1, 128, 16, 40, [20, 30, 10, 5], seed=10)
    good = _run(p, True)
    ws = b.Workspace(1 << 22)
    out = torch.full_like(good, 7.0)
    bad = dict(p, seq_lens=_i32([20, -1, 33, 5]))
    b.prefix_attention(**bad, workspace=ws, out=out)
    assert b.read_device_status(ws) == b.GDN_ERR_INVALID_ARG
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    assert bool((out[1] == 7).all()) and bool((out[2] == 7).all())
    for page in (-1, p["k_cache"].shape[0], 2**31 - 1):
        table = p["block_table"].clone()
        table[1, 0] = page
        out = b.prefix_attention(**dict(p, block_table=table), workspace=ws)
        assert b.read_device_status(ws) == b.GDN_ERR_INVALID_ARG
        assert bool(torch.isfinite(out).all()) and torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])
        # zero keys and values in the page's place
        zero = dict(p, k_cache=p["k_cache"].clone(), v_cache=p["v_cache"].clone())
        zero["k_cache"][p["block_table"][1, 0]] = 0
        zero["v_cache"][p["block_table"][1, 0]] = 0
        assert torch.equal(out[1], _run(zero, True)[1])


def test_device_status():
    """What is found wrong on the device reaches a caller who keeps no workspace; on other streams and in graphs too."""
    p = _problem(4, 1, 2, 1, 128, 16, 40, [20, 30, 10, 5], seed=10)
    want, status = _run(p, True), _i32([55])
    assert torch.equal(b.prefix_attention(**p, device_status=status), want) and int(status) == b.GDN_OK
    bad = dict(p, seq_lens=_i32([20, -1, 33, 5]))
    b.prefix_attention(**bad, device_status=status)
    assert int(status) == b.GDN_ERR_INVALID_ARG
    b.prefix_attention(**p, workspace=b.Workspace(1 << 22), device_status=status)
    assert int(status) == b.GDN_OK
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.prefix_attention(**bad, device_status=status, stream=side.cuda_stream)
    side.synchronize()
    assert int(status) == b.GDN_ERR_INVALID_ARG
    g, lens = torch.cuda.CUDAGraph(), p["seq_lens"].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = b.prefix_attention(**dict(p, seq_lens=lens), device_status=status)
    for now, code in ((p["seq_lens"], b.GDN_OK), (bad["seq_lens"], b.GDN_ERR_INVALID_ARG), (p["seq_lens"], b.GDN_OK)):
        lens.copy_(now)
        status.fill_(55)
        g.replay()
        assert int(status) == code
    assert torch.equal(out, want)
    for wrong in (_i32([0, 0]), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises((ValueError, TypeError)):
            b.prefix_attention(**p, device_status=wrong)
    with pytest.raises(ValueError):
        b.prefix_attention(**p, device_status=p["seq_lens"][1:2])
    with pytest.raises(ValueError):
        b.prefix_attention(**p, out=torch.empty_like(want), device_status=p["q"].view(-1).view(torch.int32)[:1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L,G,prefix", [(2, 1, 2, 70), (20, 1, 2, 300), (4, 17, 2, 300), (1, 40, 1, 0)])
def test_every_bad_page_id_is_reported(N, L, G, prefix, d):
    """Ids just outside the cache and far from it, in both tables, for few rows and for many, in the first key tile
    and in a later one: reported, and read as zero keys and values."""
    own = 200
    p = _problem(N, L, 2 * G, 2, d, 16, prefix, [own] * N, seed=21)
    ws, P = b.Workspace(1 << 24), p["k_cache"].shape[0]
    places = [("block_table", (N - 1, 0)), ("block_table", (0, own // 16))]
    places += [("prefix_pages", (0,)), ("prefix_pages", (prefix // 16,))] if prefix else []
    for name, at in places:
        page = int(p[name][at])
        zero = dict(p, k_cache=p["k_cache"].clone(), v_cache=p["v_cache"].clone())
        zero["k_cache"][page] = zero["v_cache"][page] = 0
        want = _run(zero, False)
        for bad in (-1, -2, -3, P, P + 1, 2**31 - 1, -2**31):
            table = p[name].clone()
            table[at] = bad
            out = b.prefix_attention(**{**p, name: table}, causal=False, workspace=ws)
            assert b.read_device_status(ws) == b.GDN_ERR_INVALID_ARG, (name, at, bad)
            assert torch.equal(out, want), (name, at, bad)


def test_same_bits_streams_and_graphs():
    p = _problem(20, 2, 8, 2, 128, 16, 900, [37] * 20, seed=11)
    want = _run(p, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = b.prefix_attention(**p)
    c = b.prefix_attention(**p, stream=side.cuda_stream)             # its own buffers, another stream than the current
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want) and torch.equal(c, want)
    # two graphs with a workspace each; lengths and queries change between replays
    ws, out = [b.Workspace(1 << 24) for _ in range(2)], [torch.zeros_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g, w, x in zip(graphs, ws, out):
        with torch.cuda.graph(g):
            b.prefix_attention(**p, workspace=w, out=x)
    for lens in ([37] * 20, list(range(20)), [48] * 20):
        p["seq_lens"].copy_(_i32(lens))
        p["q"].mul_(-1.0)
        want = _run(p, True)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)


def test_far_pages_of_a_large_cache():
    """Pages whose byte offset passes 2^32."""
    P, page, Hkv, d = 9000, 256, 8, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    kc = torch.empty(P, page, Hkv, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    vc = torch.empty_like(kc).normal_(generator=g)
    q = torch.randn(2, 1, 8, d, generator=g, device="cuda").bfloat16()
    far = dict(q=q, k_cache=kc, v_cache=vc, prefix_pages=_i32([P - 1, P - 3]), prefix_len=300,
               block_table=_i32([[P - 2, 5], [7, P - 5]]), seq_lens=_i32([257, 400]))
    pages = [P - 1, P - 3, P - 2, 5, 7, P - 5]
    near = dict(far, k_cache=kc[pages].contiguous(), v_cache=vc[pages].contiguous(), prefix_pages=_i32([0, 1]),
                block_table=_i32([[2, 3], [4, 5]]))
    got = _run(far, True)
    assert torch.equal(got, _run(near, True))
    _close(got, _oracle(near, True), d)


def test_refusals():
    p = _problem(2, 1, 4, 2, 128, 16, 40, [5, 6], seed=12)
    with pytest.raises(ValueError):
        b.prefix_attention(**dict(p, prefix_len=49))                          # more tokens than the pages hold
    with pytest.raises(ValueError):
        b.prefix_attention(**dict(p, q=p["q"].transpose(0, 1)))
    with pytest.raises(TypeError):
        b.prefix_attention(**dict(p, k_cache=p["k_cache"].float()))
    with pytest.raises(TypeError):
        b.prefix_attention(**dict(p, seq_lens=p["seq_lens"].long()))
    with pytest.raises(b.GdnError) as e:
        b.prefix_attention(**{k: v.float() if k in ("q", "k_cache", "v_cache") else v for k, v in p.items()})
    assert e.value.status == b.GDN_ERR_UNSUPPORTED
    with pytest.raises(b.GdnError) as e:
        b.prefix_attention(**p, workspace=b.Workspace(256))
    assert e.value.status == b.GDN_ERR_INVALID_ARG


def test_a_step_as_it_is_served():
    """kv_extend -> rotary_append -> prefix_attention over three steps, against attention over the whole
    rotated history kept on the host; decode side of the softmax layers as a server runs it."""
    rng, page, N, H, Hkv, d, Lp = np.random.default_rng(13), 16, 3, 4, 2, 64, 37
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    table, f = b.rotary_table(d), o.frequencies(d)
    P, W = 40, 6
    kc, vc = normal(P, page, Hkv, d), normal(P, page, Hkv, d)
    prefix_pages = _i32([9, 4, 30])
    q, k, v = normal(Lp, H, d), normal(Lp, Hkv, d), normal(Lp, Hkv, d)
    slots = prefix_pages.long().repeat_interleave(page)[:Lp] * page + torch.arange(Lp, device="cuda") % page
    b.rotary_append(q, k, v, torch.arange(Lp, device="cuda", dtype=torch.int32), slots.int(), table, kc, vc)
    past_k = [[o.rotate(k, np.arange(Lp), f)] for _ in range(N)]
    past_v = [[o.f64(v)] for _ in range(N)]
    free = _i32([p for p in rng.permutation(P) if p not in (9, 4, 30)])
    bt, lens, left = _i32(np.full((N, W), -1)), _i32([0] * N), _i32([P - 3])
    for L in (7, 1, 13):
        new = _i32([L] * N)
        t = b.KvTables(N, N * L + 2)
        b.kv_extend(bt, lens, new, free, left, page, t, prefix_len=Lp)
        rows = N * L + 2                                                       # two padding rows
        q, k, v = normal(rows, H, d), normal(rows, Hkv, d), normal(rows, Hkv, d)
        q_rot = b.rotary_append(q, k, v, t.positions, t.slot_map, table, kc, vc)
        out = b.prefix_attention(q_rot[:N * L].view(N, L, H, d), kc, vc, prefix_pages, Lp, bt, t.seq_lens)
        start = Lp + o.ints(lens)
        for n in range(N):
            pos = start[n] + np.arange(L)
            past_k[n].append(o.rotate(k[n * L:(n + 1) * L], pos, f))
            past_v[n].append(o.f64(v[n * L:(n + 1) * L]))
            keys, vals = np.concatenate(past_k[n]), np.concatenate(past_v[n])
            qr = o.rotate(q[n * L:(n + 1) * L], pos, f)
            for l in range(L):
                for h in range(H):
                    seen = pos[l] + 1
                    x = keys[:seen, h // 2] @ qr[l, h] / d ** 0.5
                    w = np.exp(x - x.max())
                    ref = w @ vals[:seen, h // 2] / w.sum()
                    a = w @ np.abs(vals[:seen, h // 2]) / w.sum()
                    # q and k are rounded to bf16 after the rotation: scores move by 2 x 2^-8 of sum |q k| at most
                    reach = (np.abs(keys[:seen, h // 2]) @ np.abs(qr[l, h])).max() / d ** 0.5
                    tol = (np.exp(2 * 2 * 2.0 ** -8 * reach) - 1 + 2.0 ** -8 + 1e-4) * a + 2.0 ** -8 * np.abs(ref)
                    assert np.all(np.abs(o.f64(out[n, l, h]) - ref) <= tol)
        lens, left = t.seq_lens, t.free_left
    assert o.ints(lens).tolist() == [21] * N and int(left) == P - 3 - 6


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_another_device_than_the_current_one():
    p = _problem(2, 1, 4, 2, 128, 16, 40, [5, 6], seed=14)
    want = _run(p, True)
    other = {k: v.to("cuda:1") if torch.is_tensor(v) else v for k, v in p.items()}
    assert torch.equal(b.prefix_attention(**other).to("cuda:0"), want)


@pytest.mark.parametrize("N,L,H,Hkv,d,page,prefix,own", [(32, 4, 32, 8, 128, 64, 2500, False), (24, 8, 16, 16, 64, 32, 1001, True),
                                                           (64, 1, 32, 8, 128, 16, 3000, True), (300, 1, 4, 2, 64, 16, 129, True)])
def test_every_call_gives_the_same_bits(N, L, H, Hkv, d, page, prefix, own):
    """Many calls back to back: lists that end inside a key tile, several rounds of every ring, both kernels at
    once.  (A value tile cleaned before it had landed showed here once in some thousand calls.)"""
    lens = np.random.default_rng(N).integers(8, 900, N).tolist() if own else [0] * N
    p = _problem(N, L, H, Hkv, d, page, prefix, lens, W=None if own else 0, seed=15)
    ws = b.Workspace(1 << 27)
    outs = [b.prefix_attention(**p, workspace=ws) for _ in range(5)]
    base = max(outs, key=lambda x: sum(torch.equal(x, y) for y in outs))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(4000):
        wrong += (b.prefix_attention(**p, workspace=ws) != base).any()
    assert int(wrong) == 0 and b.read_device_status(ws) == b.GDN_OK


def test_buffers_of_a_call_on_another_stream():
    """A call on another stream takes no memory that queued work of the current stream still writes."""
    p = _problem(4, 1, 8, 2, 128, 16, 300, [40] * 4, seed=14)
    want = _run(p, True)
    q, k = torch.randn(700, 8, 128, device="cuda"), torch.randn(700, 2, 128, device="cuda")
    pos, table = torch.arange(700, device="cuda", dtype=torch.int32), b.rotary_table(128)
    want_q, want_k = b.rotary_forward(q, k, pos, table)
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    freed = [[torch.empty_like(t) for _ in range(8)] for t in (want, want_q, want_k)]
    for _ in range(20):
        a @ a                                                                  # holds the writes below back
    for like in freed:
        for t in like:
            t.fill_(float("nan"))
    del t, like
    freed.clear()
    got = b.prefix_attention(**p, stream=side.cuda_stream)
    got_q, got_k = b.rotary_forward(q, k, pos, table, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_q, want_q) and torch.equal(got_k, want_k)


def test_scales_and_pages_that_are_none():
    p = _problem(2, 1, 4, 2, 64, 16, 40, [5, 6], seed=15)
    for over in (dict(scale=1e-50), dict(scale=float("nan")), dict(scale=-1.0), dict(prefix_pages=None)):
        with pytest.raises(ValueError):
            b.prefix_attention(**dict(p, **over))
    with pytest.raises(b.GdnError):
        b.prefix_attention(**p, scale=3e38)


def test_capture_behind_two_streams_and_of_an_empty_call():
    """A capture whose call follows work joined from another stream, and one of a call without any key."""
    p = _problem(20, 1, 8, 2, 128, 16, 700, [37] * 20, seed=16)
    want = _run(p, True)
    none = dict(p, prefix_len=0, block_table=p["block_table"][:, :0].contiguous(), seq_lens=_i32([0] * 20))
    ws, side, g = b.Workspace(1 << 24), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    src, out, zero = p["q"].clone(), torch.empty_like(want), torch.empty_like(want)
    kc, vc = p["k_cache"].clone(), p["v_cache"].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            p["k_cache"].copy_(kc)
            p["v_cache"].copy_(vc)
        p["q"].copy_(src)
        cur.wait_stream(side)
        b.prefix_attention(**p, workspace=ws, out=out)
        b.prefix_attention(**none, workspace=ws, out=zero)
        b.prefix_attention(**p, workspace=ws, out=out)
    for t in (p["q"], p["k_cache"], p["v_cache"], out, zero):
        t.fill_(1.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not zero.any()


@pytest.mark.parametrize("N,L,H,Hkv,d,prefix,own", [(20, 2, 8, 2, 128, 900, 37), (2, 1, 4, 2, 64, 700, 300), (3, 40, 4, 4, 64, 700, 300),
                                                    (2, 40, 4, 2, 128, 0, 900), (9, 8, 8, 4, 128, 0, 900)])
def test_wait_gives_up_then_next_call_is_correct(N, L, H, Hkv, d, prefix, own):
    p = _problem(N, L, H, Hkv, d, 16, prefix, [own] * N, seed=17)
    ws, out = b.Workspace(1 << 25), torch.empty_like(p["q"])
    want = _run(p, True)
    desc = b.make_prefix_attn_desc(N, L, H, Hkv, d, 16, p["k_cache"].shape[0], p["block_table"].shape[1], prefix, True)
    for attempt in range(2):
        st = b.prefix_attention_test_wait_limit_raw(desc, p["q"], p["k_cache"], p["v_cache"], p["prefix_pages"],
                                                    p["block_table"], p["seq_lens"], out, ws.tensor, 1)
        assert st == b.GDN_OK, b.status_string(st)
        status, where = b.read_device_status_where(ws.tensor)
        assert status == b.GDN_ERR_TIMEOUT and where > 0, (attempt, status, where)
    assert torch.equal(b.prefix_attention(**p, workspace=ws), want)
    assert b.read_device_status_where(ws.tensor) == (b.GDN_OK, 0)


def test_two_calls_at_once():
    """Calls on two streams with a workspace each run beside one another and give the bits that they give alone."""
    ps = [_problem(20, 2, 8, 2, 128, 16, 900, [37] * 20, seed=18), _problem(16, 1, 8, 2, 64, 32, 1500, [200] * 16, seed=19)]
    want = [_run(p, True) for p in ps]
    streams, ws = [torch.cuda.Stream() for _ in ps], [b.Workspace(1 << 25) for _ in ps]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(100):
        for p, s, w, o in zip(ps, streams, ws, outs):
            with torch.cuda.stream(s):
                o.append(b.prefix_attention(**p, workspace=w))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


@pytest.mark.parametrize("N,L,H,Hkv,d,page", [(40, 1, 16, 2, 128, 16), (3, 4, 4, 1, 64, 64)])
def test_tables_far_wider_than_the_lengths(N, L, H, Hkv, d, page):
    lens = np.random.default_rng(N).integers(0, 90, N).tolist()
    p = _problem(N, L, H, Hkv, d, page, 3000, lens, W=4000, seed=20)
    _close(_run(p, True), _oracle(p, True), d)


def _newest(p, n, back):
    """(page, offset) of the token `back` places before the last of sequence n."""
    i, page = int(p["seq_lens"][n]) - 1 - back, p["k_cache"].shape[1]
    return int(p["block_table"][n, i // page]), i % page


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("N,L,H,Hkv,d,page,prefix,most", [
    (38, 17, 4, 4, 64, 16, 0, 1400),        # 152 CTAs of own keys, up to 11 key tiles each: two turns of the ring
    (13, 20, 12, 12, 128, 64, 0, 1300),     # 156 CTAs
    (3, 33, 8, 1, 128, 256, 300, 2000),     # 264 rows of a sequence: two CTAs a list, split
    (2, 160, 2, 1, 64, 32, 100, 900),       # 320 rows; the newest tokens cover more than one key tile
])
def test_long_own_keys_of_many_rows(N, L, H, Hkv, d, page, prefix, most, causal):
    """Own keys by the kernel of many rows, over many key tiles: lengths of their own, keys that grow along the list (the
    reference max moves in later tiles), values that only some rows see."""
    rng = np.random.default_rng(N)
    lens = rng.integers(L, most, N)
    lens[0], lens[-1] = most, L + 3
    p = _problem(N, L, H, Hkv, d, page, prefix, lens.tolist(), seed=23)
    grow = torch.ones(p["k_cache"].shape[:2], device="cuda")
    for n, s in enumerate(lens.tolist()):
        i = torch.arange(s, device="cuda")
        grow[p["block_table"][n].long()[i // page], i % page] = 0.1 + 6.0 * i / s
    p["k_cache"] = (p["k_cache"] * grow[..., None, None]).bfloat16()
    _close(_run(p, causal), _oracle(p, causal), d)
    if causal:
        for n, back, c, x in ((0, 0, 3, float("inf")), (0, L - 2, 5, -float("inf")), (N - 1, 1, 0, float("nan"))):
            pg, off = _newest(p, n, back)
            p["v_cache"][pg, off, 0, c] = x
        _close(_run(p, causal), _oracle(p, causal), d)


@pytest.mark.parametrize("N,L,H,Hkv,d,page", [(3, 20, 4, 4, 128, 64), (2, 40, 4, 1, 64, 16), (150, 17, 1, 1, 64, 16)])
def test_wide_tables_of_many_rows(N, L, H, Hkv, d, page):
    lens = np.random.default_rng(N).integers(0, 400, N).tolist()
    lens[0] = 0
    p = _problem(N, L, H, Hkv, d, page, 200, lens, W=4000, seed=24)
    _close(_run(p, True), _oracle(p, True), d)


def test_a_mixed_step_as_it_is_served():
    """Steps of decode rows and prompt chunks of unequal lengths: kv_extend packs them, rotary_append writes the cache, and
    the queries go to prefix_attention behind padding on the left (token l is the l-th of the L newest)."""
    rng, page, H, Hkv, d, Lp = np.random.default_rng(31), 16, 4, 2, 64, 37
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    table, f = b.rotary_table(d), o.frequencies(d)
    N, P, W = 4, 120, 24
    kc, vc = normal(P, page, Hkv, d), normal(P, page, Hkv, d)
    prefix_pages = _i32([9, 4, 30])
    slots = prefix_pages.long().repeat_interleave(page)[:Lp] * page + torch.arange(Lp, device="cuda") % page
    q, k, v = normal(Lp, H, d), normal(Lp, Hkv, d), normal(Lp, Hkv, d)
    b.rotary_append(q, k, v, torch.arange(Lp, device="cuda", dtype=torch.int32), slots.int(), table, kc, vc)
    free = _i32([p for p in rng.permutation(P) if p not in (9, 4, 30)])
    bt, lens, left = _i32(np.full((N, W), -1)), _i32([0] * N), _i32([P - 3])
    status = _i32([0])
    for new in ([150, 1, 40, 0], [1, 1, 1, 1], [33, 0, 200, 7], [1, 17, 1, 1]):
        t, M, L = b.KvTables(N, sum(new) + 5), sum(new), max(new)
        b.kv_extend(bt, lens, _i32(new), free, left, page, t, prefix_len=Lp, device_status=status)
        assert int(status) == b.GDN_OK
        q, k, v = normal(M + 5, H, d), normal(M + 5, Hkv, d), normal(M + 5, Hkv, d)
        q_rot = b.rotary_append(q, k, v, t.positions, t.slot_map, table, kc, vc, device_status=status)
        assert int(status) == b.GDN_OK
        padded, cu = normal(N, L, H, d), t.cu_new.tolist()
        for n in range(N):
            padded[n, L - new[n]:] = q_rot[cu[n]:cu[n + 1]]
        out = b.prefix_attention(padded, kc, vc, prefix_pages, Lp, bt, t.seq_lens, device_status=status)
        assert int(status) == b.GDN_OK
        # against the oracle's own tables, positions and rotation; the cache's keys are bf16 there and here
        want = o.prefix_attention(padded, kc, vc, prefix_pages, Lp, bt, t.seq_lens, causal=True)
        _close(out, want, d)
        for n in range(N):
            pos = Lp + o.ints(lens)[n] + np.arange(new[n])
            assert np.array_equal(o.ints(t.positions)[cu[n]:cu[n + 1]], pos)
            i = o.ints(lens)[n] + np.arange(new[n])
            at = o.ints(bt)[n][i // page], i % page
            assert np.array_equal(o.f64(vc)[at], o.f64(v[cu[n]:cu[n + 1]]))
            ref = o.rotate(k[cu[n]:cu[n + 1]], pos, f)
            # the rounding to bf16, 2^-8 of the value, and the rotation's own 4e-7 (|x1| + |x2|), at most 8e-7 of the largest
            near = np.abs(o.f64(k[cu[n]:cu[n + 1]])).max() if new[n] else 0.0
            assert np.all(np.abs(o.f64(kc)[at] - ref) <= 2.0 ** -8 * np.abs(ref) + 8e-7 * near)
        lens, left = t.seq_lens, t.free_left
    assert o.ints(lens).tolist() == [185, 19, 242, 9]
