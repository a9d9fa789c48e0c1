"""Pins of the fp64 serving oracle (oracle/serving.py) that do not retype its formulas: closed forms,
invariants and planted mistakes.  CPU only."""
import math

import numpy as np
import pytest

from oracle import serving as o


def test_rotation_is_orthogonal_and_relative():
    """Scores of rotated vectors depend on the distance of the positions alone; norms stay."""
    rng = np.random.default_rng(0)
    f = o.frequencies(8)
    for il in (False, True):
        q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
        a = o.rotate(q, [100], f, interleaved=il)[0, 0] @ o.rotate(k, [93], f, interleaved=il)[0, 0]
        b = o.rotate(q, [7], f, interleaved=il)[0, 0] @ o.rotate(k, [0], f, interleaved=il)[0, 0]
        assert abs(a - b) < 1e-12
        assert abs(np.linalg.norm(o.rotate(q, [12345], f, interleaved=il)) - np.linalg.norm(q)) < 1e-12


def test_rotation_closed_form():
    """One pair, base 1 (one radian per position): position 1 turns (1, 0) to (cos 1, sin 1)."""
    f = o.frequencies(2, base=1.0)
    y = o.rotate(np.array([[[1.0, 0.0, 5.0]]]), [1], f)
    assert np.allclose(y[0, 0], [math.cos(1), math.sin(1), 5.0], atol=1e-15)
    back = o.rotate(y, [1], f, sign=-1.0)
    assert np.allclose(back[0, 0], [1.0, 0.0, 5.0], atol=1e-15)


def test_layouts_are_permutations_of_one_another():
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((3, 2, 8)), o.frequencies(8)
    half = o.rotate(x, [0, 5, 9], f)
    perm = np.array([0, 4, 1, 5, 2, 6, 3, 7])           # half layout -> neighbours
    assert np.allclose(o.rotate(x[..., perm], [0, 5, 9], f, interleaved=True), half[..., perm])


def test_frequency_scalings():
    f = o.frequencies(64)
    assert np.allclose(o.frequencies(64, scaling="linear", factor=4.0), f / 4)
    ntk = o.frequencies(64, scaling="ntk", factor=4.0)
    assert abs(ntk[0] - 1.0) < 1e-15 and abs(ntk[-1] - f[-1] / 4) < 1e-15      # fastest kept, slowest interpolated
    ramp = o.frequencies(64, scaling="ramp", factor=4.0, original_len=4096)
    assert ramp[0] == f[0] and abs(ramp[-1] - f[-1] / 4) < 1e-18
    assert np.all(ramp <= f + 1e-18) and np.all(ramp >= f / 4 - 1e-18)


def test_lengths_stay_int32():
    """A sequence's tokens do not pass 2^31 - 1, however much room its table has."""
    table = np.zeros((2, 2049), int)
    r = o.kv_extend(table, [2**31 - 10, 2**31 - 10], [10, 9], [], 0, 1 << 20, 19)
    assert r["bad"] and list(r["lens"]) == [2**31 - 10, 2**31 - 1] and r["slot_map"][:10].tolist() == [-1] * 10


def test_tables_keep_every_page_single():
    """Pages of all sequences stay distinct, slots of all tokens too, over several steps."""
    rng = np.random.default_rng(2)
    N, W, page, F = 5, 9, 4, 40
    table, lens, free, left = np.full((N, W), -1), np.zeros(N, int), rng.permutation(F), F
    seen = set()
    for _ in range(4):
        new = rng.integers(0, 8, N)
        r = o.kv_extend(table, lens, new, free, left, page, int(new.sum()) + 2)
        assert not r["bad"]
        live = r["slot_map"][:int(new.sum())]
        assert len(set(live)) == len(live) and not seen & set(live.tolist()) and np.all(r["slot_map"][int(new.sum()):] == -1)
        seen |= set(live.tolist())
        used = r["table"][r["table"] >= 0]
        assert len(set(used.tolist())) == len(used) == F - r["left"]
        assert np.array_equal(r["lens"], lens + new)
        table, lens, left = r["table"], r["lens"], r["left"]


def _cache(rng, P=6, page=4, hk=1, d=4):
    return rng.standard_normal((P, page, hk, d)), rng.standard_normal((P, page, hk, d))


def test_attention_pins():
    rng = np.random.default_rng(3)
    kc, vc = _cache(rng)
    # equal scores give the mean of the visible values
    q = np.zeros((1, 2, 1, 4))
    out, _, _ = o.prefix_attention(q, kc, vc, [2], 3, np.array([[5, 0]]), [6], causal=True)
    rows = [(2, 0), (2, 1), (2, 2), (5, 0), (5, 1), (5, 2), (5, 3), (0, 0), (0, 1)]
    assert np.allclose(out[0, 1, 0], np.mean([vc[p, i, 0] for p, i in rows], axis=0))
    assert np.allclose(out[0, 0, 0], np.mean([vc[p, i, 0] for p, i in rows[:-1]], axis=0))
    # one visible key gives its value; none gives zero
    q = rng.standard_normal((1, 1, 1, 4))
    assert np.allclose(o.prefix_attention(q, kc, vc, [], 0, np.array([[3]]), [1])[0][0, 0, 0], vc[3, 0, 0])
    assert np.all(o.prefix_attention(q, kc, vc, [], 0, np.array([[3]]), [0])[0] == 0)
    # the prefix is the same as own keys in its place
    q = rng.standard_normal((1, 1, 2, 4))
    a = o.prefix_attention(q, kc, vc, [1, 4], 8, np.array([[2]]), [3])[0]
    b = o.prefix_attention(q, kc, vc, [], 0, np.array([[1, 4, 2]]), [11])[0]
    assert np.allclose(a, b)
    # scale: two keys with scores 0 and ln 3 have weights 1/4 and 3/4
    kc = np.zeros((1, 4, 1, 4))
    kc[0, 1, 0, 0] = 2 * math.log(3)
    vc = np.zeros((1, 4, 1, 4))
    vc[0, 1, 0] = 1.0
    q = np.zeros((1, 1, 1, 4))
    q[..., 0] = 1.0
    assert np.allclose(o.prefix_attention(q, kc, vc, [], 0, np.array([[0]]), [2])[0], 0.75)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_ignores_what_a_row_does_not_see(causal):
    rng = np.random.default_rng(4)
    kc, vc = _cache(rng, P=8)
    q = rng.standard_normal((2, 3, 2, 4))
    table, lens = np.array([[1, 2], [3, 4]]), [5, 2]
    base = o.prefix_attention(q, kc, vc, [0], 2, table, lens, causal=causal)[0]
    kc2, vc2 = kc.copy(), vc.copy()
    kc2[0, 2:], vc2[0, 2:] = np.nan, np.nan              # behind the prefix
    kc2[2, 1:], vc2[2, 1:] = np.inf, np.nan              # behind sequence 0
    kc2[4:], vc2[4:] = np.nan, np.nan                    # behind sequence 1, and free pages
    assert np.array_equal(base, o.prefix_attention(q, kc2, vc2, [0], 2, table, lens, causal=causal)[0])
    vc2 = vc.copy()
    vc2[2, 0] += 1.0                                     # the newest token of sequence 0
    moved = o.prefix_attention(q, kc, vc2, [0], 2, table, lens, causal=causal)[0] != base
    assert not moved[1].any() and moved[0, 2].all() and moved[0, :2].any() == (not causal)
