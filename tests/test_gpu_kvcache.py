"""Block tables and slot maps (gdn_kv_extend) against the page-by-page allocator of the oracle: equal."""
import numpy as np
import pytest
import torch

from gated_deltanet_dual_b200 import binding as b
from oracle import serving as o

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _check(table, lens, new, free, count, page, rows, prefix=0):
    want = o.kv_extend(table, lens, new, free, count, page, rows, prefix)
    t = b.KvTables(len(lens), rows)
    for x in (t.slot_map, t.positions, t.cu_new, t.seq_lens, t.free_left):
        x.fill_(-99)
    dev = _i32(table)
    status = _i32([55])
    args = (dev, _i32(lens), _i32(new), _i32(free), _i32([count]), page, t)
    for _ in range(2):                                      # the same inputs: the same answer
        b.kv_extend(*args, prefix_len=prefix, device_status=status)
        assert np.array_equal(o.ints(dev), want["table"])
        assert np.array_equal(o.ints(t.slot_map), want["slot_map"])
        assert np.array_equal(o.ints(t.positions), want["positions"])
        assert np.array_equal(o.ints(t.cu_new), want["cu"])
        assert np.array_equal(o.ints(t.seq_lens), want["lens"])
        assert int(t.free_left) == want["left"]
        assert int(status) == (b.GDN_ERR_INVALID_ARG if want["bad"] else 0)
    return want


def _random(N, W, page, most, seed, prefix=0, count=None, rows=None, zeros=0.3):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, W * page - most + 1, N)
    new = np.where(rng.random(N) < zeros, 0, rng.integers(0, most + 1, N))
    ids = rng.permutation(2 * N * W)
    table = ids[:N * W].reshape(N, W)
    free = ids[N * W:]
    return _check(table, lens, new, free, len(free) if count is None else count, page,
                  int(new.sum()) + 3 if rows is None else rows, prefix)


@pytest.mark.parametrize("N,W,page,most", [(1, 1, 1, 1), (1, 4, 16, 64), (2, 300, 16, 4800), (7, 9, 5, 11), (64, 256, 16, 1),
                                           (1023, 8, 16, 8), (1025, 8, 32, 40), (4096, 6, 16, 3), (4097, 6, 16, 20),
                                           (9001, 5, 64, 9)])
def test_against_the_allocator(N, W, page, most):
    _random(N, W, page, most, seed=N, prefix=N % 3 * 1000)


def test_long_runs_and_many_ctas():
    _random(3, 1 << 14, 16, 200000, seed=1, zeros=0.0)
    _random(600, 64, 64, 3000, seed=2)


def test_nothing_new():
    w = _random(5, 4, 16, 0, seed=3, rows=0)
    assert not w["bad"]
    _random(5, 4, 16, 0, seed=3, rows=6)


def test_refusals_on_the_device():
    page, W = 4, 3
    table = np.arange(18).reshape(6, 3)
    free = np.arange(100, 110)
    # too long, negative length, negative count: the others are served
    w = _check(table, [12, -1, 4, 3, 0, 5], [1, 2, -3, 2, 4, 1], free, 10, page, 40)
    assert w["bad"] and list(w["lens"]) == [12, -1, 4, 5, 4, 6]
    # pages run out in the middle; those that need none are still served
    w = _check(table, [4, 4, 4, 2, 0, 5], [1, 1, 1, 1, 1, 1], free, 2, page, 6)
    assert w["bad"] and list(w["lens"]) == [5, 5, 4, 3, 0, 6] and w["left"] == 0
    # rows run out
    w = _check(table, [0, 0, 0, 0, 0, 0], [3, 3, 3, 0, 2, 1], free, 10, page, 7)
    assert w["bad"] and list(w["lens"]) == [3, 3, 0, 0, 0, 0]
    # an empty list, and counts outside the list
    assert _check(table, [1] * 6, [1] * 6, free[:0], 0, page, 6)["bad"] is False
    assert _check(table, [0] * 6, [1] * 6, free, 11, page, 6)["bad"]
    assert _check(table, [0] * 6, [1] * 6, free, -3, page, 6)["bad"]


def test_sums_past_32_bits():
    """Counts whose sum passes 2^32: refused rows, saturated offsets, no write out of place."""
    N, W, page = 6, 1 << 20, 2048
    t = b.KvTables(N, 10)
    table = torch.zeros(N, W, dtype=torch.int32, device="cuda")
    lens, new = _i32([0] * N), _i32([3, 2**31 - 1, 2**31 - 1, 2**31 - 1, 1, 0])
    status = _i32([0])
    b.kv_extend(table, lens, new, _i32([7, 8, 9]), _i32([3]), page, t, device_status=status)
    assert o.ints(t.slot_map).tolist() == [9 * 2048, 9 * 2048 + 1, 9 * 2048 + 2] + [-1] * 7
    assert o.ints(t.cu_new).tolist() == [0, 3, 2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1]
    assert o.ints(t.seq_lens).tolist() == [3, 0, 0, 0, 0, 0] and int(t.free_left) == 2
    assert int(status) == b.GDN_ERR_INVALID_ARG and int(table.count_nonzero()) == 1


def test_lengths_near_the_last_int32():
    """Tables with room for more tokens than an int32 length counts: refused past 2^31 - 1, served up to it."""
    page, W = 1 << 20, 2049
    table = np.arange(3 * W).reshape(3, W) % 2000
    w = _check(table, [2**31 - 10, 2**31 - 10, 5], [20, 9, 2], [2001, 2002], 2, page, 34)
    assert w["bad"] and list(w["lens"]) == [2**31 - 10, 2**31 - 1, 7] and w["left"] == 2
    # pages of 2^31 - 1 tokens, the count of pages next to 2^32; the free list is empty
    table = np.array([[0, 7, 7], [0, 7, 7], [0, 7, 7]])
    w = _check(table, [2**31 - 1, 2**31 - 3, 2**31 - 1], [5, 2, 0], [], 0, 2**31 - 1, 8)
    assert w["bad"] and list(w["lens"]) == [2**31 - 1] * 3 and np.array_equal(w["table"], table)
    # positions saturate where the prefix takes them past the last int32
    t = b.KvTables(1, 2)
    b.kv_extend(_i32([[0] * W]), _i32([2**31 - 4]), _i32([2]), _i32([]), _i32([0]), page, t, prefix_len=2)
    assert t.positions.tolist() == [2**31 - 2, 2**31 - 1] and t.seq_lens.tolist() == [2**31 - 2]
    b.kv_extend(_i32([[0] * W]), _i32([2**31 - 4]), _i32([2]), _i32([]), _i32([0]), page, t, prefix_len=2**31 - 1)
    assert t.positions.tolist() == [2**31 - 1] * 2


def test_bad_page_ids_give_no_slot():
    t = b.KvTables(2, 2)
    status = _i32([0])
    b.kv_extend(_i32([[-5], [2**27]]), _i32([1, 1]), _i32([1, 1]), _i32([0]), _i32([0]), 16, t, device_status=status)
    assert o.ints(t.slot_map).tolist() == [-1, -1] and int(status) == b.GDN_ERR_INVALID_ARG


def test_refusals():
    t = b.KvTables(2, 4)
    ok = dict(block_table=_i32([[0], [1]]), seq_lens=_i32([0, 0]), new_lens=_i32([1, 1]), free_pages=_i32([3, 4]),
              free_count=_i32([2]), page_size=16, tables=t)
    b.kv_extend(**ok)
    with pytest.raises(ValueError):
        b.kv_extend(**ok | dict(seq_lens=_i32([0])))
    with pytest.raises(TypeError):
        b.kv_extend(**ok | dict(new_lens=torch.ones(2, dtype=torch.int64, device="cuda")))
    with pytest.raises(b.GdnError):
        b.kv_extend(**ok | dict(page_size=0))
    with pytest.raises(b.GdnError):
        b.kv_extend(**ok | dict(seq_lens=t.seq_lens))       # in place
    with pytest.raises(ValueError):
        b.kv_extend(**ok | dict(block_table=_i32([[0, 1], [2, 3]])[:, :1]))


def test_sizes_past_32_bits_are_refused():
    def run(page, prefix):
        return b.kv_extend(_i32([[-1, -1]]), _i32([0]), _i32([3]), _i32([7, 5]), _i32([2]), page, b.KvTables(1, 3), prefix_len=prefix)
    assert run(16, 4).positions.tolist() == [4, 5, 6]
    for page, prefix in (((1 << 32) + 16, 4), (16, (1 << 32) + 4), (16, -(1 << 32))):
        with pytest.raises(ValueError):
            run(page, prefix)


def test_tables_past_32_bits_are_refused():
    """Tensors whose sizes do not fit an int32 (17 GB, never written or read)."""
    far = torch.empty((1 << 32) + 2, dtype=torch.int32, device="cuda")
    args = dict(block_table=_i32([[-1, -1]]), seq_lens=_i32([0]), new_lens=_i32([3]), free_pages=_i32([7, 5]),
                free_count=_i32([2]), page_size=16, tables=b.KvTables(1, 3))
    for over in (dict(block_table=far.view(1, -1)), dict(free_pages=far)):
        with pytest.raises(ValueError):
            b.kv_extend(**args | over)
    q, cache, few = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device="cuda"), _i32([0])
    rows = q.expand(1 << 32, 1, 64)
    with pytest.raises(ValueError):                         # 2^32 rows are not none
        b.rotary_append(rows, rows, rows, far[:1 << 32], far[:1 << 32], b.rotary_table(64), cache, cache.clone(), q_out=rows)
    with pytest.raises(ValueError):
        b.rotary_forward(rows, None, far[:1 << 32], b.rotary_table(64), q_out=rows)
    for over in (dict(block_table=far.view(1, -1)), dict(prefix_pages=far, prefix_len=(1 << 32) + 5)):
        with pytest.raises(ValueError):
            b.prefix_attention(**dict(q=q.view(1, 1, 1, 64), k_cache=cache, v_cache=cache, prefix_pages=None, prefix_len=0,
                                      block_table=_i32([[0]]), seq_lens=few) | over)


def test_tables_that_were_resized():
    t = b.KvTables(1, 3)
    args = (_i32([[-1, -1]]), _i32([0]), _i32([3]), _i32([7, 5]), _i32([2]), 16, t)
    b.kv_extend(*args)
    t.slot_map.resize_(1 << 20)
    with pytest.raises(ValueError):
        b.kv_extend(*args)
    none = b.KvTables(1, 0)                                  # no rows: nothing to move
    b.kv_extend(_i32([[-1]]), _i32([0]), _i32([0]), _i32([]), _i32([0]), 16, none)
    assert none.cu_new.tolist() == [0, 0]
