"""The linear-attention and softmax-attention entry points reject bad arguments
before touching the device (CPU only: no call here reaches a kernel launch)."""
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


def lin(**kw):
    base = dict(batch=2, seqlen=300, qk_heads=2, v_heads=4, dk=128, dv=128, q_stride=0, k_stride=0,
                v_stride=0, scale=1.0, io_dtype=ssd.SSD_BF16)
    base.update(kw)
    return ssd.SsdLinattnDims(*(base[f] for f, _ in ssd.SsdLinattnDims._fields_))


def lin_scan(lib, d, over=(), ws_bytes=1 << 33, cu=None):
    args = [at(i) for i in range(8)]      # q, k, v, g, init, o, fin, ws
    for i, p in over:
        args[i] = p
    if cu is not None:
        return lib.ssd_linattn_chunk_scan_varlen(ctypes.byref(d), cu, *args, ws_bytes, None)
    return lib.ssd_linattn_chunk_scan(ctypes.byref(d), *args, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seqlen=-1), 2), (dict(qk_heads=0), 2), (dict(qk_heads=3), 2),
    (dict(dk=96), 3), (dict(dv=32), 3), (dict(io_dtype=2), 3), (dict(scale=INF), 3),
    (dict(scale=float("nan")), 3), (dict(q_stride=-256), 2), (dict(k_stride=128), 2),
    (dict(v_stride=516), 7), (dict(q_stride=1 << 23), 3), (dict(v_heads=1 << 17), 3),
    (dict(v_heads=1 << 16, qk_heads=1), 3), (dict(seqlen=1 << 60), 2), (dict(batch=1, seqlen=1 << 31), 3),
    (dict(batch=1 << 40, seqlen=0), 3)])
def test_linattn_sizes(lib, kw, code):
    assert lin_scan(lib, lin(**kw)) == code
    n = ctypes.c_size_t(7)
    assert lib.ssd_linattn_chunk_scan_workspace_size(ctypes.byref(lin(**kw)), ctypes.byref(n)) == code
    assert n.value == 7


def test_linattn_pointers(lib):
    d = lin(seqlen=2000)
    for i in (0, 1, 2, 3, 5, 6):
        assert lin_scan(lib, d, [(i, None)]) == 1
    for i in (0, 1, 2, 4, 5, 6, 7):
        assert lin_scan(lib, d, [(i, at(i, 8))]) == 7
    assert lin_scan(lib, d, [(3, at(3, 2))]) == 7
    assert lin_scan(lib, d, [(7, None)]) == 5
    assert lin_scan(lib, d, ws_bytes=1024) == 5
    for i in (0, 1, 2, 4, 6, 7):
        assert lin_scan(lib, d, [(5, at(i, 64))]) == 4        # o over anything
    for i in (0, 1, 2, 3, 7):
        assert lin_scan(lib, d, [(6, at(i))]) == 4            # the final state over an input or the workspace
    assert lin_scan(lib, d, [(6, at(4, 1024))]) == 4          # part of the initial state
    assert lin_scan(lib, d, [(7, at(4, 1024))]) == 4          # workspace over the initial state
    assert lin_scan(lib, lin(batch=0), [(i, None) for i in range(8)]) == 0
    assert lib.ssd_linattn_chunk_scan(None, *([None] * 8), 0, None) == 1
    assert lib.ssd_linattn_chunk_scan_workspace_size(ctypes.byref(d), None) == 1


def test_linattn_offsets(lib):
    d = lin(batch=2, seqlen=300)
    for cu in ((0, 100, 299), (1, 100, 300), (0, 200, 100), (0, 301, 300), (0, -1, 300)):
        assert lin_scan(lib, d, cu=offsets(*cu)) == 2, cu
    assert lib.ssd_linattn_chunk_scan_varlen(ctypes.byref(d), None, *[at(i) for i in range(8)], 0, None) == 1


def test_linattn_workspace(lib):
    def size(**kw):
        n = ctypes.c_size_t()
        assert lib.ssd_linattn_chunk_scan_workspace_size(ctypes.byref(lin(**kw)), ctypes.byref(n)) == 0
        return n.value

    assert size(batch=0) == size(seqlen=0) == size(seqlen=1) == 0
    long = size(batch=1, seqlen=131072)
    assert long > 0 and long % (4 * 128 * 128 * 4) == 0 and long < 1 << 30


def test_linattn_step(lib):
    base = [at(i) for i in range(6)]      # q, k, v, g, state, o

    def call(over=(), **kw):
        args = list(base)
        for i, p in over:
            args[i] = p
        return lib.ssd_linattn_decode_step(ctypes.byref(lin(**kw)), *args, None)

    for i in range(6):
        assert call([(i, None)]) == 1
    for i, off in ((0, 1), (1, 1), (2, 1), (3, 2), (4, 8), (5, 1)):
        assert call([(i, at(i, off))]) == 7
    for i in range(5):
        assert call([(5, at(i))]) == 4
    for i in range(4):
        assert call([(4, at(i))]) == 4
    assert call(dk=32) == 3 and call(qk_heads=3) == 2 and call(scale=INF) == 3
    assert call([(i, None) for i in range(6)], batch=0) == 0
    assert lib.ssd_linattn_decode_step(None, *base, None) == 1


def attn(**kw):
    base = dict(batch=2, q_rows=300, kv_rows=300, q_heads=8, kv_heads=2, head_dim=128, q_stride=0,
                k_stride=0, v_stride=0, scale=0.1, io_dtype=ssd.SSD_BF16)
    base.update(kw)
    return ssd.SsdAttnDims(*(base[f] for f, _ in ssd.SsdAttnDims._fields_))


def prefill(lib, d, over=(), cu=(0, 100, 300), starts=None, lens=None):
    args = [at(i) for i in range(4)]
    for i, p in over:
        args[i] = p
    return lib.ssd_attn_prefill(ctypes.byref(d), None if cu is None else offsets(*cu),
                                None if starts is None else offsets(*starts),
                                None if lens is None else offsets(*lens), *args, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(q_rows=-1), 2), (dict(kv_rows=-1), 2), (dict(kv_heads=0), 2),
    (dict(kv_heads=3), 2), (dict(head_dim=80), 3), (dict(io_dtype=5), 3), (dict(scale=-INF), 3),
    (dict(q_stride=1000), 2), (dict(k_stride=260), 7), (dict(v_stride=1 << 23), 3),
    (dict(q_heads=1 << 17), 3), (dict(q_rows=1 << 58, kv_rows=1 << 58), 2)])
def test_attn_sizes(lib, kw, code):
    assert prefill(lib, attn(**kw)) == code


def test_attn_prefill(lib):
    d = attn()
    assert prefill(lib, d, cu=None) == 1
    for i in range(4):
        assert prefill(lib, d, [(i, None)]) == 1
        assert prefill(lib, d, [(i, at(i, 8))]) == 7
    for i in range(3):
        assert prefill(lib, d, [(3, at(i, 4096))]) == 4
    for cu in ((0, 100, 299), (1, 100, 300), (0, 301, 300)):
        assert prefill(lib, d, cu=cu) == 2
    for starts, lens in (((-1, 0), (1, 1)), ((0, 0), (301, 1)), ((0, 300), (1, 1)), ((0, 0), (-1, 1)),
                         ((0, 2 ** 62), (1, 2 ** 62))):
        assert prefill(lib, d, starts=starts, lens=lens) == 2
    assert prefill(lib, d, starts=(0, 0)) == 1 and prefill(lib, d, lens=(0, 0)) == 1
    assert prefill(lib, attn(kv_rows=200)) == 2
    big = 1 << 31
    assert prefill(lib, attn(batch=1, q_rows=big, kv_rows=big), cu=(0, big)) == 3
    assert prefill(lib, attn(batch=1, q_rows=1 << 29, kv_rows=1 << 29), cu=(0, 1 << 29)) == 3
    assert prefill(lib, attn(q_rows=0, kv_rows=0), [(i, None) for i in range(4)], cu=(0, 0, 0)) == 0
    assert prefill(lib, attn(batch=0, q_rows=0, kv_rows=0), cu=(0,)) == 0
    assert lib.ssd_attn_prefill(None, offsets(0), None, None, *([None] * 5)) == 1


def test_attn_step(lib):
    d = attn(batch=4, kv_rows=4096)
    n = ctypes.c_size_t()
    assert lib.ssd_attn_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    base = [at(i) for i in range(8)]      # q, k, v, kc, vc, lengths, o, ws

    def call(over=(), ws_bytes=n.value, **kw):
        args = list(base)
        for i, p in over:
            args[i] = p
        dd = attn(**{**dict(batch=4, kv_rows=4096), **kw})
        return lib.ssd_attn_decode_step(ctypes.byref(dd), *args, ws_bytes, None)

    for i in range(7):
        assert call([(i, None)]) == 1
    assert call([(7, None)]) == 5 and call(ws_bytes=n.value - 1) == 5
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 8), (4, 8), (5, 2), (6, 8), (7, 8)):
        assert call([(i, at(i, off))]) == 7
    for i, j in ((6, 0), (6, 3), (6, 5), (6, 7), (3, 4), (3, 1), (4, 2), (4, 5), (7, 0), (7, 3)):
        assert call([(i, at(j))]) == 4, (i, j)
    assert call(kv_rows=-1) == 2 and call(kv_rows=1 << 31) == 3 and call(head_dim=96) == 3
    assert call(batch=1 << 30) == 3
    assert call([(i, None) for i in range(8)], batch=0) == 0
    assert lib.ssd_attn_decode_step(None, *base, 0, None) == 1
    assert lib.ssd_attn_decode_workspace_size(ctypes.byref(d), None) == 1
