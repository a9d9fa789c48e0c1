"""Refusals of the serving calls (include/gdn_rotary.h, include/gdn_kvcache.h) and the host-side tables.
CPU only: placeholder addresses that the host validation must reject before anything is enqueued."""
import copy
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from gated_deltanet_dual_b200 import binding as b
from oracle import serving as o

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: host-only check")
A = [0x7f0000000000 + i * (1 << 30) for i in range(14)]      # addresses apart, 256-byte aligned


def _call(name, desc, ptrs, *tail):
    return getattr(b.load_library(), name)(ctypes.byref(desc) if desc is not None else None, *ptrs, *tail)


def _with(desc, **over):
    d = copy.copy(desc)
    for k, v in over.items():
        setattr(d, k, v)
    return d


# ----------------------------------------------------------------------------- frequencies
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "ramp"])
@pytest.mark.parametrize("rot", [2, 20, 64, 256])
def test_frequencies_against_the_formula(scaling, rot):
    if scaling == "ntk" and rot < 4:
        with pytest.raises(b.GdnError):
            b.rotary_frequencies(rot, scaling=scaling, factor=8.0)
        return
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, original_len=8192, beta_fast=4.0, beta_slow=1.0)
    got = b.rotary_frequencies(rot, **kw).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # the oracle's frequencies are doubles: a few roundings of 2^-53 each, relative; an entry is a whole
    # multiple of 2^-64 turns, so it is off by up to 2^-65 turns = 2 pi 2^-65 = 1.703e-19 radians, absolute
    assert np.allclose(got, o.frequencies(rot, **kw), rtol=2e-14, atol=1.71e-19)


def test_frequencies_wrap_whole_turns():
    """A frequency of more than a turn per position keeps its fraction (positions are whole)."""
    got = b.rotary_frequencies(4, base=1e-4)                # f = 1, 100 radians
    want = (100.0 / (2 * math.pi)) % 1.0
    assert abs(float(got[1]) / 2.0 ** 64 - want) < 1e-14


@pytest.mark.parametrize("bad", [dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=258), dict(base=0.0), dict(base=math.inf),
                                 dict(factor=0.5), dict(factor=math.nan), dict(scaling="ramp"),
                                 dict(scaling="ramp", original_len=4096, beta_fast=1.0, beta_slow=1.0)])
def test_frequencies_refusals(bad):
    kw = dict(rot_dim=64) | bad
    with pytest.raises(b.GdnError):
        b.rotary_frequencies(kw.pop("rot_dim"), **kw)


def test_unknown_scaling_is_refused():
    with pytest.raises(ValueError):
        b.rotary_frequencies(64, scaling="cubic")


# ----------------------------------------------------------------------------- rotary
ROT = b.RotaryDesc(6, 3, 4, 2, 64, 64, 0, b.GDN_BF16, 1.0, 0, 256, 64, 128, 64, 256, 64, 128, 64)


@no_gpu
@pytest.mark.parametrize("name", ["gdn_rotary_forward", "gdn_rotary_backward"])
@pytest.mark.parametrize("over,want", [
    (dict(num_rows=-1), 1), (dict(num_positions=0), 1), (dict(num_positions=4), 1), (dict(num_heads=-1), 1),
    (dict(num_heads=0, num_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(rot_dim=7), 1), (dict(rot_dim=66), 1),
    (dict(interleaved=2), 1), (dict(dtype=5), 1), (dict(scale=math.nan), 1), (dict(reserved=1), 1),
    (dict(q_row_stride=-1), 1), (dict(q_out_row_stride=0), 1), (dict(q_out_head_stride=32), 1),
    (dict(head_dim=300, rot_dim=64, q_row_stride=1200, q_head_stride=300, k_row_stride=600, k_head_stride=300,
          q_out_row_stride=1200, q_out_head_stride=300, k_out_row_stride=600, k_out_head_stride=300), 3),
])
def test_rotary_refuses_descriptors(name, over, want):
    assert _call(name, _with(ROT, **over), A[:6], None) == want


@no_gpu
def test_rotary_refuses_pointers():
    f = lambda *p: _call("gdn_rotary_forward", ROT, p, None)
    assert _call("gdn_rotary_forward", None, A[:6], None) == 1
    for i in range(6):
        p = list(A[:6])
        p[i] = None
        assert f(*p) == 1, i
        p = list(A[:6])
        p[i] += 1
        assert f(*p) == 2, i
    d = _with(ROT, q_out_row_stride=512)                    # in place with other strides
    assert _call("gdn_rotary_forward", d, [A[0], A[1], A[2], A[3], A[2], A[5]], None) == 1
    assert _call("gdn_rotary_forward", _with(ROT, num_rows=0), [None] * 6, None) == 0      # nothing to do


# order: turns, positions, q, k, q_out, k_out
@no_gpu
@pytest.mark.parametrize("out,other,shift", [(4, 3, 0), (5, 2, 0), (4, 5, 0), (4, 1, -8), (5, 0, -8), (4, 2, 128), (5, 3, -2),
                                             (4, 3, 1024)])
def test_rotary_refuses_overlaps(out, other, shift):
    p = list(A[:6])
    p[out] = p[other] + shift
    assert _call("gdn_rotary_forward", ROT, p, None) == 1


@no_gpu
def test_rotary_takes_an_output_behind_an_input():
    p = list(A[:6])
    p[4] = p[3] + 256 * 2 * 4                               # k's 6 rows of 256 bytes end 512 bytes before
    assert _call("gdn_rotary_forward", ROT, p, None) == 4   # no device: past the checks


@no_gpu
def test_rotary_refuses_strides_past_any_memory():
    for over in (dict(q_row_stride=1 << 45), dict(k_out_row_stride=1 << 62), dict(q_out_head_stride=(1 << 63) - 1)):
        assert _call("gdn_rotary_forward", _with(ROT, **over), A[:6], None) == 1, over


# ----------------------------------------------------------------------------- append
APP = b.AppendDesc(6, 4, 2, 64, 64, 0, 16, 10, b.GDN_BF16, 1.0, 512, 64, 512, 64, 512, 64, 256, 64)


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_rows=-1), 1), (dict(num_heads=0), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(rot_dim=65), 1), (dict(interleaved=-1), 1), (dict(page_size=0), 1), (dict(num_pages=0), 1),
    (dict(page_size=256, num_pages=1 << 23), 1), (dict(dtype=-1), 1), (dict(scale=math.inf), 1),
    (dict(v_row_stride=-4), 1), (dict(q_out_row_stride=64), 1),
])
def test_append_refuses_descriptors(over, want):
    assert _call("gdn_rotary_append", _with(APP, **over), A[:10], None) == want


@no_gpu
def test_append_refuses_pointers():
    for i in range(9):
        p = list(A[:10])
        p[i] = None
        assert _call("gdn_rotary_append", APP, p, None) == 1, i
    for i in range(10):
        p = list(A[:10])
        p[i] += 1
        assert _call("gdn_rotary_append", APP, p, None) == 2, i
    p = list(A[:10])
    p[6] = p[3]                                             # q_out = q with other strides
    assert _call("gdn_rotary_append", APP, p, None) == 1


# order: turns, positions, slots, q, k, v, q_out, k_cache, v_cache, status
@no_gpu
@pytest.mark.parametrize("out,other,shift", [(8, 7, 0), (8, 7, 16 * 10 * 2 * 64 * 2 - 2), (7, 4, 0), (8, 5, -2), (7, 3, 0),
                                             (6, 7, 0), (6, 4, 0), (9, 2, 20), (7, 1, -2048), (6, 3, 2)])
def test_append_refuses_overlaps(out, other, shift):
    p = list(A[:10])
    p[out] = p[other] + shift
    assert _call("gdn_rotary_append", APP, p, None) == 1


# ----------------------------------------------------------------------------- tables
EXT = b.KvExtendDesc(8, 16, 32, 100, 64, 0, 0, 0)


@no_gpu
@pytest.mark.parametrize("over", [dict(num_seqs=0), dict(table_width=0), dict(page_size=0), dict(num_free=-1),
                                  dict(max_new_tokens=-1), dict(prefix_len=-1), dict(reserved0=1), dict(reserved1=1),
                                  dict(num_seqs=2**31 - 1)])
def test_extend_refuses_descriptors(over):
    assert _call("gdn_kv_extend", _with(EXT, **over), A[:11], None) == 1


@no_gpu
def test_extend_refuses_pointers_and_aliases():
    for i in range(10):
        p = list(A[:11])
        p[i] = None
        assert _call("gdn_kv_extend", EXT, p, None) == 1, i
    for i in range(11):
        p = list(A[:11])
        p[i] += 2
        assert _call("gdn_kv_extend", EXT, p, None) == 2, i
    # order: table, lens, new, free, count | slots, positions, cu, lens_out, left, status
    for out, other in [(8, 1), (9, 4), (5, 6), (7, 2), (0, 3), (10, 9), (10, 4)]:
        p = list(A[:11])
        p[out] = p[other]
        assert _call("gdn_kv_extend", EXT, p, None) == 1, (out, other)
    p = list(A[:11])
    p[8] = p[1] + 4 * 7                                     # overlaps the last length only
    assert _call("gdn_kv_extend", EXT, p, None) == 1


# ----------------------------------------------------------------------------- attention
ATT = b.make_prefix_attn_desc(4, 2, 8, 2, 128, 16, 100, 8, 40, True)


def test_attention_workspace_size():
    n = b.prefix_attn_workspace_size(ATT)
    assert n >= 256 and n % 256 == 0
    assert b.prefix_attn_workspace_size(_with(ATT, head_dim=96)) == 0
    assert b.prefix_attn_workspace_size(_with(ATT, num_seqs=0)) == 0
    assert b.prefix_attn_workspace_size(_with(ATT, prefix_len=0, table_width=0)) >= 256


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_seqs=0), 1), (dict(num_tokens=0), 1), (dict(num_heads=0), 1), (dict(num_kv_heads=3), 1),
    (dict(head_dim=0), 1), (dict(head_dim=96), 3), (dict(page_size=0), 1), (dict(page_size=24), 3), (dict(page_size=8), 3),
    (dict(page_size=512), 3), (dict(num_pages=0), 1), (dict(num_pages=1 << 28), 1), (dict(table_width=-1), 1),
    (dict(table_width=1 << 28), 1), (dict(prefix_len=-1), 1), (dict(prefix_len=2**31 - 1), 1), (dict(causal=2), 1),
    (dict(dtype=b.GDN_FP32), 3), (dict(dtype=9), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(num_seqs=1 << 20, num_tokens=1 << 10), 3),
])
def test_attention_refuses_descriptors(over, want):
    assert _call("gdn_prefix_attn", _with(ATT, **over), A[:8], ctypes.c_size_t(1 << 60), None) == want


@no_gpu
def test_attention_refuses_pointers():
    big = ctypes.c_size_t(1 << 60)
    for i in range(8):
        p = list(A[:8])
        p[i] = None
        assert _call("gdn_prefix_attn", ATT, p, big, None) == 1, i
        p = list(A[:8])
        p[i] += 2
        assert _call("gdn_prefix_attn", ATT, p, big, None) == 2, i
    size = b.prefix_attn_workspace_size(ATT)
    assert _call("gdn_prefix_attn", ATT, A[:8], ctypes.c_size_t(size - 1), None) == 1


# order: q, k_cache, v_cache, prefix_pages, block_table, seq_lens, out, workspace
@no_gpu
@pytest.mark.parametrize("out,other,shift", [(6, 0, 0), (6, 1, 16), (6, 2, 100 * 16 * 2 * 128 * 2 - 16), (6, 5, 0), (7, 0, 0),
                                             (7, 4, -256), (7, 6, 256), (6, 3, -16)])
def test_attention_refuses_overlaps(out, other, shift):
    p = list(A[:8])
    p[out] = p[other] + shift
    assert _call("gdn_prefix_attn", ATT, p, ctypes.c_size_t(1 << 60), None) == 1


@no_gpu
def test_attention_refuses_a_scale_past_fp32():
    assert _call("gdn_prefix_attn", _with(ATT, scale=3e38), A[:8], ctypes.c_size_t(1 << 60), None) == 1


def test_register_split_is_one_instruction_a_side():
    """setmaxnreg must be the same instruction for all four warps of a warpgroup: one that takes and one that gives."""
    with open(os.path.join(os.path.dirname(b.LIB_PATH), "csrc", "gdn_prefix_attn.cu")) as f:
        source = f.read()
    assert source.count("setmaxnreg.dec") == 1 and source.count("setmaxnreg.inc") == 1


# ----------------------------------------------------------------------------- the Python layer
def test_python_layer_wants_cuda_tensors():
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)
    t = b.RotaryTable(z(4, dtype=torch.int64), 8, False, 1.0)
    with pytest.raises(ValueError):
        b.rotary_forward(z(2, 1, 8), z(2, 1, 8), i(2), t)
    with pytest.raises(ValueError):
        b.rotary_append(z(2, 1, 8), z(2, 1, 8), z(2, 1, 8), i(2), i(2), t, z(1, 16, 1, 8), z(1, 16, 1, 8))
    with pytest.raises(ValueError):
        b.kv_extend(i(2, 2), i(2), i(2), i(4), i(1), 16, b.KvTables(2, 4, "cpu"))
    with pytest.raises(ValueError):
        b.prefix_attention(z(1, 1, 1, 64), z(1, 16, 1, 64), z(1, 16, 1, 64), i(0), 0, i(1, 1), i(1))
    with pytest.raises(ValueError):
        b.rotary_forward(None, None, i(2), t)


def test_tables_that_moved_are_refused():
    """Memory that a caller has taken from a table's tensors is not written or read."""
    make = lambda: b.KvTables(2, 4, "cpu")
    assert len(make()._where()) == 5 and b.KvTables(2, 0, "cpu")._where()[:2] == (0, 0)
    for name in ("slot_map", "positions", "cu_new", "seq_lens", "free_left"):
        t = make()
        getattr(t, name).fill_(3)                           # its contents are the caller's
        t._where()
        getattr(t, name).resize_(1 << 20)
        with pytest.raises(ValueError):
            t._where()
        t = make()
        getattr(t, name).data = torch.zeros(5, dtype=torch.int32)
        with pytest.raises(ValueError):
            t._where()
        t = make()
        getattr(t, name).untyped_storage().resize_(0)
        with pytest.raises(ValueError):
            t._where()
    r = b.RotaryTable(torch.zeros(4, dtype=torch.int64), 8, False, 1.0)
    r._on(-1)
    r.turns.resize_(1 << 20)
    with pytest.raises(ValueError):
        r._on(-1)


def test_python_layer_refuses_what_32_bits_do_not_hold():
    for rot in (1 << 32, (1 << 32) + 64, -(1 << 32)):
        with pytest.raises(ValueError):
            b.rotary_frequencies(rot)


@no_gpu
def test_wait_limit_of_zero_is_refused():
    assert _call("gdn_prefix_attn_test_wait_limit", ATT, A[:8], ctypes.c_size_t(1 << 60), ctypes.c_uint32(0), None) == 1
