"""Rotary positions and rotary + append on the GPU against the fp64 oracle, element by element.

Tolerance of one element y = a (x1 c - x2 s), derived from the arithmetic: the angle is off by at most
2 pi 2^-32 (dropped bits of the fixed-point turn) + pi 2^-25 (rounding of the half-turns to fp32) <
9.6e-8, sincospi by one ulp <= 2^-24, the scaling of c and s, the two products and the sum by 2^-24
each: |err| <= a (|x1| + |x2|) (9.6e-8 + 5 x 6e-8) < 4e-7 a (|x1| + |x2|); a bf16 output adds half a
step, 2^-8 |y|."""
import numpy as np
import pytest
import torch

from gated_deltanet_dual_b200 import binding as b
from oracle import serving as o

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _close(got, x, ref, freq, il, scale, what):
    x, ref = np.abs(o.f64(x)), np.asarray(ref)
    n = len(freq)
    bound = np.zeros_like(ref)
    i1 = np.arange(n) * 2 if il else np.arange(n)
    i2 = i1 + 1 if il else i1 + n
    bound[..., i1] = bound[..., i2] = 4e-7 * scale * (x[..., i1] + x[..., i2])
    if got.dtype == torch.bfloat16:
        bound[..., :2 * n] += 2.0 ** -8 * np.abs(ref[..., :2 * n]) + 1e-38
    err = np.abs(o.f64(got) - ref)
    assert np.all(err <= bound), f"{what}: {np.max(err - bound):.3e} over the bound"


CASES = [
    # T, H, Hkv, d, rot, interleaved, scaling, factor
    (1, 1, 1, 2, 2, False, "none", 1.0),
    (5, 4, 2, 64, 64, False, "none", 1.0),
    (5, 4, 2, 64, 64, True, "none", 1.0),
    (33, 16, 16, 128, 128, False, "linear", 4.0),
    (7, 8, 1, 128, 64, True, "ramp", 8.0),
    (7, 8, 1, 128, 32, False, "ramp", 8.0),
    (3, 3, 1, 80, 20, False, "ntk", 2.0),           # element path: 20 is no multiple of a vector pair
    (3, 3, 1, 80, 20, True, "none", 1.0),
    (4, 2, 2, 256, 256, False, "none", 1.0),
    (4, 2, 2, 255, 254, True, "none", 1.0),         # odd head
    (6, 5, 3, 16, 0, False, "none", 1.0),           # nothing rotated: a copy
    (2500, 2, 1, 64, 64, False, "none", 1.0),       # several rows per CTA
    (40007, 1, 1, 16, 16, True, "none", 1.0),
]


def _table(rot, il, scaling, factor):
    kw = dict(scaling=scaling, factor=factor, original_len=4096)
    t = b.rotary_table(rot, interleaved=il, **kw)
    return t, o.frequencies(rot, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, dtype):
    T, H, Hkv, d, rot, il, scaling, factor = case
    g = _gen(T + d)
    q, k = _normal(g, T, H, d, dtype=TYPES[dtype]), _normal(g, T, Hkv, d, dtype=TYPES[dtype])
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    table, f = _table(rot, il, scaling, factor)
    for call, sign in ((b.rotary_forward, 1.0), (b.rotary_backward, -1.0)):
        qo, ko = call(q, k, pos, table)
        for got, x, name in ((qo, q, "q"), (ko, k, "k")):
            ref = o.rotate(x, pos, f, interleaved=il, scale=table.scale, sign=sign)
            _close(got, x, ref, f, il, table.scale, name)
            assert torch.equal(got[..., rot:], x[..., rot:])


def test_far_and_negative_positions():
    table, f = _table(64, False, "none", 1.0)
    pos = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 1 << 24, 123456789], dtype=torch.int32, device="cuda")
    q = _normal(_gen(0), 7, 3, 64, dtype=torch.float32)
    qo, none = b.rotary_forward(q, None, pos, table)
    assert none is None
    exact = np.array([float(10000.0 ** (-2 * np.longdouble(i) / 64)) for i in range(32)])
    # in 80-bit arithmetic, so that the oracle's own frequencies keep 64 bits at 2^31 positions
    turns = np.array([10000.0 ** (-2 * np.longdouble(i) / 64) for i in range(32)], np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    t = o.ints(pos)[:, None].astype(np.longdouble) * turns
    t = (2 * np.pi * (t - np.rint(t))).astype(np.float64)[:, None, :]
    x = o.f64(q)
    ref = np.concatenate([x[..., :32] * np.cos(t) - x[..., 32:] * np.sin(t), x[..., :32] * np.sin(t) + x[..., 32:] * np.cos(t)], -1)
    _close(qo, q, ref, exact, False, 1.0, "far")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_views_slices_in_place_and_orders(dtype):
    """Views share positions; q and k are slices of one projection; heads before rows; in place."""
    dt, g = TYPES[dtype], _gen(3)
    table, f = _table(32, False, "none", 1.0)
    V, T, H, Hkv, d = 2, 9, 4, 2, 64
    pos = torch.arange(50, 50 + T, device="cuda", dtype=torch.int32)
    qkv = _normal(g, V, T, H + 2 * Hkv, d, dtype=dt)
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    before = qkv.clone()
    qo, ko = b.rotary_forward(q, k, pos, table)
    ref_q, ref_k = o.rotate(q, pos, f), o.rotate(k, pos, f)
    _close(qo, q, ref_q, f, False, 1.0, "q of views")
    _close(ko, k, ref_k, f, False, 1.0, "k of views")
    assert torch.equal(qkv, before)
    b.rotary_forward(q, k, pos, table, q_out=q, k_out=k)            # in place: v untouched
    assert torch.equal(qkv[:, :, :H], qo) and torch.equal(qkv[:, :, H:H + Hkv], ko)
    assert torch.equal(qkv[:, :, H + Hkv:], before[:, :, H + Hkv:])
    heads_first = _normal(g, H, T, d, dtype=dt).transpose(0, 1)     # [T, H, d] with heads outermost in memory
    out = torch.zeros(H, T, d, dtype=dt, device="cuda").transpose(0, 1)
    b.rotary_forward(heads_first, None, pos, table, q_out=out)
    _close(out, heads_first, o.rotate(heads_first, pos, f), f, False, 1.0, "heads first")
    odd = _normal(g, T * H * d + 1, dtype=dt)[1:].view(T, H, d)     # not 16-byte aligned: element path
    got, _ = b.rotary_forward(odd, None, pos, table)
    _close(got, odd, o.rotate(odd, pos, f), f, False, 1.0, "unaligned")
    none, only_k = b.rotary_backward(None, k, pos, table)
    assert none is None and only_k.shape == k.shape


def test_backward_is_the_gradient():
    """Against differences of the oracle's forward (the rotation is linear: any step is exact), and
    <dy, R x> = <R^T dy, x> of the kernels themselves."""
    g = _gen(4)
    for il in (False, True):
        table, f = _table(8, il, "ramp", 8.0)
        x, dy = _normal(g, 3, 2, 12, dtype=torch.float32), _normal(g, 3, 2, 12, dtype=torch.float32)
        pos = torch.tensor([3, 700, 31], dtype=torch.int32, device="cuda")
        dx, _ = b.rotary_backward(dy, None, pos, table)
        base = o.f64(x)
        up = o.f64(dy)
        num = np.zeros_like(base)
        for idx in np.ndindex(base.shape):
            e = np.zeros_like(base)
            e[idx] = 1.0
            diff = o.rotate(base + e, pos, f, interleaved=il, scale=table.scale) - o.rotate(base - e, pos, f, interleaved=il, scale=table.scale)
            num[idx] = (diff / 2 * up).sum()
        _close(dx, dy, num, f, il, table.scale, "difference gradient")
        y, _ = b.rotary_forward(x, None, pos, table)
        left, right = (y.double() * dy.double()).sum(), (dx.double() * x.double()).sum()
        assert abs(float(left - right)) <= 4e-7 * 2 * float((x.abs().double().sum(-1) * dy.abs().double().sum(-1)).sum())


def test_empty_and_refusals():
    table, _ = _table(8, False, "none", 1.0)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 16, device="cuda")
    assert b.rotary_forward(q, None, pos, table)[0].shape == (0, 2, 16)
    q = torch.zeros(4, 2, 16, device="cuda")
    with pytest.raises(ValueError):
        b.rotary_forward(q, None, pos, table)                                            # positions too short
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        b.rotary_forward(q, q.bfloat16(), pos, table)
    with pytest.raises(TypeError):
        b.rotary_forward(q, None, pos.long(), table)
    with pytest.raises(ValueError):
        b.rotary_forward(q.transpose(1, 2), None, pos, table)                            # heads not contiguous
    with pytest.raises(b.GdnError):
        b.rotary_forward(q[..., :4].contiguous(), None, pos, table)                      # rot_dim over head_dim
    with pytest.raises(b.GdnError):
        b.rotary_forward(q, None, pos, table, q_out=q[:1].expand(4, 2, 16))              # rows on top of one another


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,H,Hkv,d,rot,il,page", [(1, 4, 4, 64, 64, False, 16), (37, 8, 2, 128, 128, False, 16),
                                                    (300, 2, 1, 128, 64, True, 64), (9, 3, 1, 72, 36, False, 5),
                                                    (2600, 2, 2, 64, 32, False, 128)])
def test_append(R, H, Hkv, d, rot, il, page, dtype):
    dt, g = TYPES[dtype], _gen(R)
    table, f = _table(rot, il, "linear", 2.0)
    P = R // page + 3
    qkv = _normal(g, R, H + 2 * Hkv, d, dtype=dt)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    v[0, 0, 0] = float("nan")                                        # copied bit for bit
    kc, vc = _normal(g, P, page, Hkv, d, dtype=dt), _normal(g, P, page, Hkv, d, dtype=dt)
    slots = torch.randperm(P * page, generator=g, device="cuda")[:R].to(torch.int32)
    slots[R // 2::7] = -1
    pos = torch.arange(1000, 1000 + R, device="cuda", dtype=torch.int32)
    q_out = _normal(g, R, H, d, dtype=dt)
    want = o.append(q, k, v, pos, slots, f, kc, vc, q_out, interleaved=il)
    kc0, vc0, qo0 = kc.clone(), vc.clone(), q_out.clone()
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    got = b.rotary_append(q, k, v, pos, slots, table, kc, vc, q_out=q_out, device_status=status)
    assert got is q_out and int(status) == 0
    live = slots >= 0
    at = slots[live].long()
    _close(q_out[live], q[live], want[0][live.cpu().numpy()], f, il, 1.0, "q_out")
    _close(kc.flatten(0, 1)[at], k[live], want[1].reshape(-1, Hkv, d)[at.cpu().numpy()], f, il, 1.0, "k_cache")
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(vc.flatten(0, 1)[at].view(bits), v[live].contiguous().view(bits))
    rest = torch.ones(P * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(kc.flatten(0, 1)[rest], kc0.flatten(0, 1)[rest])
    assert torch.equal(vc.flatten(0, 1)[rest], vc0.flatten(0, 1)[rest])
    assert torch.equal(q_out[~live], qo0[~live])


def test_append_skips_bad_slots():
    table, _ = _table(64, False, "none", 1.0)
    q, k, v = (torch.ones(4, 1, 64, device="cuda") for _ in range(3))
    kc, vc = torch.zeros(2, 16, 1, 64, device="cuda"), torch.zeros(2, 16, 1, 64, device="cuda")
    slots = torch.tensor([5, 32, -2, 2**31 - 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.rotary_append(q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), slots, table, kc, vc,
                          q_out=torch.zeros_like(q), device_status=status)
    assert int(status) == b.GDN_ERR_INVALID_ARG
    assert float(vc.sum()) == 64 and float(kc.sum()) == 64 and float(out.sum()) == 64
    b.rotary_append(q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), slots.clamp(-1, 31)[:1].repeat(4) - 1,
                    table, kc, vc, q_out=out, device_status=status)
    assert int(status) == 0


def test_append_far_into_a_large_cache():
    """A cache whose byte offsets pass 2^32: the last page."""
    table, f = _table(128, False, "none", 1.0)
    P, page, Hkv, d = 9000, 256, 8, 128                              # 2.3e6 slots x 2 KB = 4.7 GB a cache
    kc = torch.zeros(P, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = _gen(5)
    q, k, v = (_normal(g, 2, h, d, dtype=torch.bfloat16) for h in (16, 8, 8))
    slots = torch.tensor([P * page - 1, P * page // 2 + 77], dtype=torch.int32, device="cuda")
    b.rotary_append(q, k, v, torch.zeros(2, dtype=torch.int32, device="cuda"), slots, table, kc, vc)
    assert torch.equal(kc.flatten(0, 1)[slots.long()], k) and torch.equal(vc.flatten(0, 1)[slots.long()], v)
    assert int(torch.count_nonzero(vc[:P // 2 - 1])) == 0 and int(torch.count_nonzero(vc[P // 2 + 2:-1])) == 0


def test_slices_of_one_buffer_in_place_and_beside():
    """q, k and both outputs as column slices of one buffer: their extents overlap, their rows alternate."""
    g = _gen(21)
    buf = _normal(g, 33, 4 + 2 + 4 + 2, 64, dtype=torch.bfloat16)
    pos, table = torch.arange(33, dtype=torch.int32, device="cuda"), b.rotary_table(64)
    q, k, qo, ko = buf.split((4, 2, 4, 2), dim=1)
    want = b.rotary_forward(q.contiguous(), k.contiguous(), pos, table)
    b.rotary_forward(q, k, pos, table, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    b.rotary_forward(q, k, pos, table, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    with pytest.raises(b.GdnError):
        b.rotary_forward(q, k, pos, table, q_out=buf[:, 1:5], k_out=ko)


def test_one_position_of_many_views():
    """A slice of one position: its views lie as far apart as the whole tensor's."""
    table, f = _table(32, False, "none", 1.0)
    x, out = _normal(_gen(8), 5, 7, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 7, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    q, k = x[:, 3:4, :2], x[:, 3:4, 2:]
    qo, ko = b.rotary_forward(q, k, pos, table, k_out=out[:, 6:])
    _close(qo, q, o.rotate(q, pos, f), f, False, 1.0, "q")
    _close(ko, k, o.rotate(k, pos, f), f, False, 1.0, "k")
    assert ko.data_ptr() == out[:, 6:].data_ptr() and int(out[:, :6].count_nonzero()) == 0
    with pytest.raises(ValueError):                          # two positions of every view: no single row stride
        b.rotary_forward(x[:, 3:5], None, torch.tensor([3, 4], dtype=torch.int32, device="cuda"), table)
