"""The paged-cache entry points reject bad arguments before touching the device (CPU
only: no call here reaches a kernel launch)."""
import ctypes
import os

import pytest

import state_space_model_mamba_amd as ssd

FAKE = 1 << 40           # well-aligned "device" addresses 8 GiB apart, never dereferenced
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIBRARY):
        pytest.fail("libssd.so is not built (run __graft_entry__.build())")
    return ssd.load()


def at(i, off=0):
    return ctypes.c_void_p(FAKE + (i << 33) + off)


def offsets(*x):
    return (ctypes.c_int64 * len(x))(*x)


def dims(**kw):
    base = dict(batch=2, rows=2, q_heads=8, kv_heads=2, head_dim=128, num_pages=100, page_size=64, max_pages=10,
                q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, k_out_stride=0, scale=0.1,
                io_dtype=ssd.SSD_BF16, page_format=ssd.SSD_PAGES_IO, reserved=0)
    base.update(kw)
    return ssd.SsdPagedDims(*(base[f] for f, _ in ssd.SsdPagedDims._fields_))


def rope(**kw):
    base = dict(inv_freq=FAKE + (20 << 33), q_weight=FAKE + (21 << 33), k_weight=FAKE + (22 << 33),
                positions=FAKE + (23 << 33), rot_dim=128, interleaved=0, eps=1e-6, reserved=0)
    base.update(kw)
    return ssd.SsdQkRope(*(base[f] for f, _ in ssd.SsdQkRope._fields_))


def replaced(n, over):
    args = [at(i) for i in range(n)]
    for i, p in over:
        args[i] = p
    return args


def norm(lib, d, r, over=()):
    return lib.ssd_attn_qk_norm_rope(ctypes.byref(d), ctypes.byref(r), *replaced(4, over), None)


# q, k, v, k_pages, v_pages, k_scales, v_scales, table, lengths, q_out, k_out
def append(lib, d, r=None, over=(), cu=None):
    return lib.ssd_attn_paged_append(ctypes.byref(d), ctypes.byref(rope(positions=None) if r is None else r),
                                     None if cu is None else offsets(*cu), *replaced(11, over), None)


# k_pages, v_pages, k_scales, v_scales, table, k, v
def gather(lib, d, cu, starts=None, over=()):
    return lib.ssd_attn_paged_gather(ctypes.byref(d), None if cu is None else offsets(*cu),
                                     None if starts is None else offsets(*starts), *replaced(7, over), None)


# q, k_pages, v_pages, k_scales, v_scales, table, lengths, o, workspace
def step(lib, d, over=(), ws=1 << 32):
    return lib.ssd_attn_paged_decode_step(ctypes.byref(d), *replaced(9, over), ws, None)


HEADS = [(dict(q_heads=0), 2), (dict(kv_heads=0), 2), (dict(kv_heads=3), 2), (dict(reserved=1), 2),
         (dict(head_dim=96), 3), (dict(io_dtype=2), 3), (dict(q_heads=1 << 17), 3),
         (dict(q_heads=1 << 16, kv_heads=1 << 16), 3), (dict(q_stride=-8), 2), (dict(q_stride=512), 2),
         (dict(q_stride=1 << 23), 3), (dict(q_stride=1025), 7)]
PAGES = [(dict(num_pages=0), 2), (dict(max_pages=0), 2), (dict(page_size=0), 2), (dict(page_size=8), 3),
         (dict(page_size=48), 3), (dict(page_size=2048), 3), (dict(num_pages=1 << 31), 3), (dict(page_format=2), 3),
         (dict(max_pages=1 << 26), 3), (dict(max_pages=1 << 58), 2), (dict(batch=1 << 40, rows=1 << 40), 3)]


@pytest.mark.parametrize("kw,code", HEADS + [(dict(rows=-1), 2), (dict(rows=1 << 31), 3), (dict(k_stride=128), 2),
                                             (dict(q_out_stride=8), 2), (dict(k_out_stride=261), 7)])
def test_norm_sizes(lib, kw, code):
    assert norm(lib, dims(**kw), rope()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=-8), 2), (dict(rot_dim=136), 2), (dict(rot_dim=12), 3), (dict(interleaved=2), 2),
    (dict(reserved=1), 2), (dict(eps=-1e-6), 3), (dict(eps=INF), 3), (dict(eps=float("nan")), 3),
    (dict(inv_freq=None), 1), (dict(positions=None), 1), (dict(inv_freq=FAKE + 2), 7), (dict(q_weight=FAKE + 2), 7),
    (dict(k_weight=FAKE + 1), 7), (dict(positions=FAKE + 2), 7)])
def test_rope_arguments(lib, kw, code):
    assert norm(lib, dims(), rope(**kw)) == code
    if "positions" not in kw or kw["positions"] is not None:
        assert append(lib, dims(), rope(**kw)) == code


def test_norm_pointers(lib):
    d, r = dims(rows=100), rope()
    for i in range(4):
        assert norm(lib, d, r, [(i, None)]) == 1 and norm(lib, d, r, [(i, at(i, 8))]) == 7
    for i, j in ((2, 1), (3, 0), (3, 2), (2, 20), (3, 21), (2, 22), (3, 23)):
        assert norm(lib, d, r, [(i, at(j))]) == 4, (i, j)
    assert norm(lib, d, r, [(2, at(0, 2048))]) == 4           # q_out one row further on
    # in place but with other distances between rows
    assert norm(lib, dims(rows=100, q_stride=2048), r, [(2, at(0))]) == 4
    # slices of one projection: q_out over k's columns, and k_out over q_out's
    wide = dict(rows=100, q_stride=1536, k_stride=1536, q_out_stride=1536, k_out_stride=1536)
    one = [(0, at(0)), (1, at(0, 2048)), (2, at(0, 512)), (3, at(5))]
    assert norm(lib, dims(**wide), r, one) == 4
    assert norm(lib, dims(**wide), r, [(0, at(0)), (1, at(0, 2048)), (2, at(5)), (3, at(5, 1024))]) == 4
    assert norm(lib, dims(**wide), r, [(0, at(0, 512)), (1, at(0)), (2, at(0, 512)), (3, at(0, 2560 - 256))]) == 4
    # a slice that wraps into the next row
    assert norm(lib, dims(**wide), r, [(0, at(0, 1024)), (1, at(6)), (2, at(7)), (3, at(0, 512 + 256))]) == 4
    assert norm(lib, dims(rows=0), rope(positions=None), [(i, None) for i in range(4)]) == 0
    assert lib.ssd_attn_qk_norm_rope(None, ctypes.byref(r), *replaced(4, ()), None) == 1
    assert lib.ssd_attn_qk_norm_rope(ctypes.byref(d), None, *replaced(4, ()), None) == 1


@pytest.mark.parametrize("kw,code", HEADS + PAGES + [(dict(batch=-1), 2), (dict(rows=-1), 2)])
def test_append_sizes(lib, kw, code):
    assert append(lib, dims(**kw)) == code


@pytest.mark.parametrize("fmt", [ssd.SSD_PAGES_IO, ssd.SSD_PAGES_4BIT])
def test_append_pointers(lib, fmt):
    d, q4 = dims(page_format=fmt), fmt == ssd.SSD_PAGES_4BIT
    scales = (5, 6) if q4 else ()
    for i in (0, 1, 2, 3, 4, 7, 8, 9) + scales:
        assert append(lib, d, over=[(i, None)]) == 1, i
    for i in (0, 1, 2, 3, 4, 9, 10) + scales:
        assert append(lib, d, over=[(i, at(i, 8))]) == 7, i
    assert append(lib, d, over=[(7, at(7, 2))]) == 7 and append(lib, d, over=[(8, at(8, 2))]) == 7
    for i, j in ((3, 4), (3, 0), (4, 2), (3, 7), (4, 8), (9, 1), (9, 2), (10, 0), (10, 2), (9, 3), (10, 9), (9, 7), (3, 20)):
        assert append(lib, d, over=[(i, at(j))]) == 4, (i, j)
    for i in scales:
        for j in (0, 3, 4, 7, 8, 11 - i):
            assert append(lib, d, over=[(i, at(j))]) == 4, (i, j)
    assert append(lib, dims(page_format=fmt, rows=3)) == 2                    # not one token each
    for cu in ((0, 1, 3), (1, 1, 2), (0, 3, 2), (0, -1, 2)):
        assert append(lib, d, cu=cu) == 2, cu
    none = [(i, None) for i in range(11)]
    assert append(lib, dims(page_format=fmt, batch=0, rows=0), over=none) == 0
    assert append(lib, dims(page_format=fmt, rows=0), over=none, cu=(0, 0, 0)) == 0
    assert lib.ssd_attn_paged_append(None, ctypes.byref(rope()), None, *replaced(11, ()), None) == 1
    assert lib.ssd_attn_paged_append(ctypes.byref(d), None, None, *replaced(11, ()), None) == 1


@pytest.mark.parametrize("kw,code", PAGES[:-1] + [(dict(kv_heads=3), 2), (dict(rows=-1), 2), (dict(head_dim=32), 3)])
def test_gather_sizes(lib, kw, code):
    assert gather(lib, dims(**kw), (0, 1, 2)) == code


def test_gather_arguments(lib):
    d = dims(rows=700)
    assert gather(lib, d, None) == 1
    for i in (0, 1, 4, 5, 6):
        assert gather(lib, d, (0, 100, 700), over=[(i, None)]) == 1
    for i in (0, 1, 5, 6):
        assert gather(lib, d, (0, 100, 700), over=[(i, at(i, 8))]) == 7
    for i, j in ((5, 6), (5, 0), (6, 1), (5, 4)):
        assert gather(lib, d, (0, 100, 700), over=[(i, at(j))]) == 4
    four = dims(rows=700, page_format=ssd.SSD_PAGES_4BIT)
    for i in (2, 3):
        assert gather(lib, four, (0, 100, 700), over=[(i, None)]) == 1
        assert gather(lib, four, (0, 100, 700), over=[(i, at(i, 4))]) == 7
        assert gather(lib, four, (0, 100, 700), over=[(5, at(i))]) == 4
    for cu in ((0, 100, 699), (1, 100, 700), (0, 701, 700), (0, 50, 700)):
        assert gather(lib, d, cu) == 2, cu                                    # the last: 650 rows of 640
    for starts in ((-1, 0), (0, 41), (541, 0), (2 ** 62, 0), (0, 2 ** 63 - 1)):
        assert gather(lib, d, (0, 100, 700), starts) == 2, starts
    assert gather(lib, dims(rows=0), (0, 0, 0), over=[(i, None) for i in range(7)]) == 0
    assert lib.ssd_attn_paged_gather(None, offsets(0), None, *replaced(7, ()), None) == 1


@pytest.mark.parametrize("kw,code", HEADS + PAGES + [(dict(scale=INF), 3), (dict(scale=float("nan")), 3),
                                                     (dict(batch=1 << 23), 3), (dict(batch=-1), 2)])
def test_step_sizes(lib, kw, code):
    assert step(lib, dims(**kw)) == code
    n = ctypes.c_size_t(7)
    assert lib.ssd_attn_paged_decode_workspace_size(ctypes.byref(dims(**kw)), ctypes.byref(n)) == code
    assert n.value == 7


@pytest.mark.parametrize("fmt", [ssd.SSD_PAGES_IO, ssd.SSD_PAGES_4BIT])
@pytest.mark.parametrize("io", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 2), (256, 64)])
def test_step_pointers(lib, fmt, io, D, Hq):
    d, q4 = dims(page_format=fmt, io_dtype=io, head_dim=D, q_heads=Hq), fmt == ssd.SSD_PAGES_4BIT
    n = ctypes.c_size_t()
    assert lib.ssd_attn_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert 0 < n.value < 1 << 28
    scales = (3, 4) if q4 else ()
    for i in (0, 1, 2, 5, 6, 7) + scales:
        assert step(lib, d, [(i, None)], n.value) == 1, i
    for i in (0, 1, 2, 7, 8) + scales:
        assert step(lib, d, [(i, at(i, 8))], n.value) == 7, i
    for i in (5, 6):
        assert step(lib, d, [(i, at(i, 2))], n.value) == 7, i
    assert step(lib, d, [(8, None)], n.value) == 5 and step(lib, d, ws=n.value - 1) == 5
    for j in (0, 1, 2, 5, 6) + scales:
        assert step(lib, d, [(7, at(j))], n.value) == 4 and step(lib, d, [(8, at(j))], n.value) == 4, j
    assert step(lib, d, [(7, at(8))], n.value) == 4
    assert step(lib, dims(batch=0), [(i, None) for i in range(9)], 0) == 0
    assert lib.ssd_attn_paged_decode_step(None, *replaced(9, ()), 0, None) == 1
    assert lib.ssd_attn_paged_decode_workspace_size(ctypes.byref(d), None) == 1
    # the workspace depends on neither lengths nor tables
    wide = dims(page_format=fmt, io_dtype=io, head_dim=D, q_heads=Hq, batch=500, max_pages=4000)
    m = ctypes.c_size_t()
    assert lib.ssd_attn_paged_decode_workspace_size(ctypes.byref(wide), ctypes.byref(m)) == 0 and m.value == n.value
