"""Host-side argument checks of the plain-decoding and 8-bit-cache calls: a
refused call returns its code before anything is launched."""

import ctypes

import pytest

import speculative_decoding_tree_build_gb300 as tv
from speculative_decoding_tree_build_gb300.build import build

P = 0x10000  # a non-null, 256-byte aligned value; never dereferenced
OK, NULL, GEOM, SIZE, WS, MIS = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    build()
    return tv.load()


def swap(args, **at):
    out = list(args)
    for i, v in at.items():
        out[int(i[1:])] = v
    return out


def test_rope_axes_refusals(lib):
    g = tv.rope_axes_geom(4, 2, 128, [16, 24, 24])
    # geom, rows, dtype, q, ld, k, ld, positions, ld, inv_freq, q_out, ld, k_out, ld, stream
    args = [ctypes.byref(g), 3, 0, P, 512, P, 256, P, 3, P, P, 512, P, 256, None]

    def call(a):
        return lib.tv_rope_axes(*a)

    assert call(swap(args, _1=0)) == OK
    assert call(swap(args, _0=None)) == NULL
    for bad in (tv.rope_axes_geom(0, 2, 128, [64]), tv.rope_axes_geom(4, -1, 128, [64]),
                tv.rope_axes_geom(4, 2, 128, [65]), tv.rope_axes_geom(4, 2, 128, [40, 25]),
                tv.rope_axes_geom(4, 2, 128, [0]), tv.rope_axes_geom(4, 2, 128, [-1, 2]),
                tv.rope_axes_geom(4, 2, 514, [64]), tv.rope_axes_geom(4, 2, 1, [1]),
                tv.rope_axes_geom(4, 2, 128, [64], rope_style=2),
                tv.rope_axes_geom(4, 2, 128, [64], section_order=2)):
        assert call(swap(args, _0=ctypes.byref(bad))) == GEOM
    five = tv.rope_axes_geom(4, 2, 128, [1, 1, 1, 1])
    five.num_axes = 5
    assert call(swap(args, _0=ctypes.byref(five))) == GEOM
    assert call(swap(args, _2=2)) == GEOM
    assert call(swap(args, _1=-1)) == SIZE
    assert call(swap(args, _4=511)) == SIZE and call(swap(args, _6=255)) == SIZE
    assert call(swap(args, _11=511)) == SIZE and call(swap(args, _13=255)) == SIZE
    assert call(swap(args, _8=2)) == SIZE
    for i in (3, 5, 7, 9, 10, 12):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    assert call(swap(args, _3=P + 1)) == MIS and call(swap(args, _7=P + 2)) == MIS
    assert call(swap(args, _2=1, _12=P + 2)) == MIS
    with pytest.raises(ValueError):
        tv.rope_axes_geom(4, 2, 128, [1, 1, 1, 1, 1])


def test_kv_quant_refusals(lib):
    g, d96 = tv.geom(32, 8, 128), tv.geom(32, 8, 96)
    # geom, fmt, batch, rows, k, v, ld, cu, start, table, n_blocks, max_blocks, kc, vc, ks, vs,
    # num_blocks, status, stream
    args = [ctypes.byref(g), 1, 2, 5, P, P, 1024, P, P, P, P, 4, P, P, P, P, 9, P, None]

    def call(a):
        return lib.tv_kv_quant_append(*a)

    assert call(swap(args, _2=0)) == OK and call(swap(args, _3=0)) == OK
    assert call(swap(args, _0=None)) == NULL
    assert call(swap(args, _0=ctypes.byref(d96))) == GEOM
    assert call(swap(args, _1=0)) == GEOM and call(swap(args, _1=3)) == GEOM
    for i, v in ((2, -1), (2, 4097), (3, -1), (6, 1023), (11, 0), (16, 0)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (4, 5, 7, 8, 9, 10, 12, 13, 14, 15, 17):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    for i, v in ((4, P + 8), (5, P + 2), (6, 1028), (12, P + 8), (13, P + 4), (14, P + 2), (15, P + 1)):
        assert call(swap(args, **{f"_{i}": v})) == MIS
    # geom, fmt, batch, first, last, table, n_blocks, max_blocks, kc, vc, ks, vs, num_blocks,
    # out table, out n_blocks, out max_blocks, k_out, v_out, out num_blocks, status, stream
    args = [ctypes.byref(g), 2, 2, P, P, P, P, 4, P, P, P, P, 9, P, P, 4, P, P, 9, P, None]

    def read(a):
        return lib.tv_kv_quant_read(*a)

    assert read(swap(args, _2=0)) == OK
    assert read(swap(args, _0=ctypes.byref(d96))) == GEOM and read(swap(args, _1=0)) == GEOM
    for i, v in ((2, -1), (2, 4097), (7, 0), (12, 0), (15, 0), (18, 0)):
        assert read(swap(args, **{f"_{i}": v})) == SIZE
    for i in (4, 5, 6, 8, 9, 10, 11, 13, 14, 16, 17, 19):
        assert read(swap(args, **{f"_{i}": None})) == NULL
    for i, v in ((8, P + 8), (9, P + 1), (10, P + 2), (11, P + 3), (16, P + 8), (17, P + 2)):
        assert read(swap(args, **{f"_{i}": v})) == MIS


def test_decode_attention_refusals(lib):
    g = tv.geom(32, 8, 128)
    # geom, fmt, batch, q, ld, seq_len, table, n_blocks, max_blocks, kc, vc, ks, vs, num_blocks,
    # out, lse, workspace, bytes, status, stream
    args = [ctypes.byref(g), 1, 2, P, 4096, P, P, P, 4, P, P, P, P, 9, P, P, P, 1 << 40, P, None]

    def call(a):
        return lib.tv_decode_attention(*a)

    assert call(swap(args, _2=0)) == OK
    assert call(swap(args, _0=None)) == NULL
    for bad in (tv.geom(32, 8, 96), tv.geom(30, 8, 128), tv.geom(34, 2, 128),
                tv.geom(32, 8, 128, block_size=32)):
        assert call(swap(args, _0=ctypes.byref(bad))) == GEOM
    assert call(swap(args, _1=3)) == GEOM and call(swap(args, _1=-1)) == GEOM
    for i, v in ((2, -1), (2, 4097), (4, 4095), (8, 0), (13, 0)):
        assert call(swap(args, **{f"_{i}": v})) == SIZE
    for i in (3, 5, 6, 7, 9, 10, 11, 12, 14, 16, 18):
        assert call(swap(args, **{f"_{i}": None})) == NULL
    for i, v in ((3, P + 8), (4, 4100), (9, P + 8), (10, P + 8), (11, P + 2), (12, P + 1), (14, P + 8),
                 (15, P + 2), (16, P + 128)):
        assert call(swap(args, **{f"_{i}": v})) == MIS
    n = ctypes.c_size_t()
    assert lib.tv_decode_workspace_bytes(ctypes.byref(g), -1, ctypes.byref(n)) == SIZE
    assert lib.tv_decode_workspace_bytes(ctypes.byref(g), 4097, ctypes.byref(n)) == SIZE
    assert lib.tv_decode_workspace_bytes(ctypes.byref(g), 2, None) == NULL
    assert lib.tv_decode_workspace_bytes(ctypes.byref(tv.geom(32, 8, 96)), 2, ctypes.byref(n)) == GEOM
