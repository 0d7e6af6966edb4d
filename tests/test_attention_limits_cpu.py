"""Sizes at the attention layers' limits (CPU only: no call here reaches a launch)."""
import ctypes

import pytest

import state_space_model_mamba_amd as ssd
from test_attention_abi_cpu import at, attn, lib, lin, lin_scan, offsets  # noqa: F401 (lib: a fixture)


def test_scan_tokens(lib):  # noqa: F811
    """Token counts and offsets within a sequence are 32-bit sums of a token and a
    segment's length: 2^30 tokens fit, more are refused."""
    most = 1 << 30
    small = dict(qk_heads=1, v_heads=1, dk=64, dv=64)
    n = ctypes.c_size_t(7)
    size = lib.ssd_linattn_chunk_scan_workspace_size
    assert size(ctypes.byref(lin(batch=1, seqlen=most, **small)), ctypes.byref(n)) == 0 and n.value > 7
    assert size(ctypes.byref(lin(batch=1, seqlen=most + 1, **small)), ctypes.byref(n)) == 3
    assert lin_scan(lib, lin(batch=1, seqlen=most + 1, **small)) == 3
    d = lin(batch=2, seqlen=2 * most, **small)
    size = lib.ssd_linattn_chunk_scan_varlen_workspace_size
    assert size(ctypes.byref(d), offsets(0, most, 2 * most), ctypes.byref(n)) == 0
    assert size(ctypes.byref(d), offsets(0, most - 1, 2 * most), ctypes.byref(n)) == 3


def test_decode_launches(lib):  # noqa: F811
    """A launch holds fewer than 2^32 threads: a step of more work-groups of 256 is
    refused with the size, not by the device."""
    n = ctypes.c_size_t(7)
    size = lib.ssd_attn_decode_workspace_size
    one = dict(kv_rows=1, head_dim=64)
    for kw in (dict(batch=1 << 24, q_heads=1, kv_heads=1), dict(batch=1 << 22, q_heads=8, kv_heads=4),
               dict(batch=1 << 22, q_heads=128, kv_heads=1)):
        assert size(ctypes.byref(attn(**one, **kw)), ctypes.byref(n)) == 3
        assert lib.ssd_attn_decode_step(ctypes.byref(attn(**one, **kw)), *[at(8 * i) for i in range(8)], 0, None) == 3
        kw["batch"] -= 1
        assert size(ctypes.byref(attn(**one, **kw)), ctypes.byref(n)) == 0
    for kw in (dict(batch=1 << 24, v_heads=1, dv=64), dict(batch=1 << 20, v_heads=4, dv=256)):
        d = lin(qk_heads=1, dk=64, **kw)
        assert lib.ssd_linattn_decode_step(ctypes.byref(d), *[at(64 * i) for i in range(6)], None) == 3


def test_planner_segment_counts(lib):  # noqa: F811
    """The scan planner's segment counts at shapes whose times are documented, read back
    from the workspace size (one fp32 dk x dv state per head and segment of a sequence
    of more than one)."""
    for batch, seqlen, hk, hv, dk, dv, io, segments in (
            (1, 77, 16, 32, 128, 128, ssd.SSD_BF16, 0),        # one: no workspace
            (8, 2048, 8, 24, 128, 64, ssd.SSD_BF16, 4),
            (4, 8192, 16, 32, 128, 128, ssd.SSD_BF16, 4),
            (2, 4096, 16, 16, 256, 256, ssd.SSD_BF16, 4),
            (1, 13384, 4, 4, 256, 64, ssd.SSD_BF16, 84),
            (2, 1000, 4, 8, 64, 64, ssd.SSD_F32, 16),
            (1, 11370, 1, 1, 256, 128, ssd.SSD_F32, 119)):
        size = ssd.ssd_linattn_chunk_scan_workspace_size(batch, seqlen, hk, hv, dk, dv, io)
        assert size == batch * segments * hv * dk * dv * 4, (seqlen, dk, dv, size / (batch * hv * dk * dv * 4))
    cu = [0, 8192, 12289, 15289, 17337, 18837, 19861, 20638, 21150]
    assert ssd.ssd_linattn_chunk_scan_varlen_workspace_size(cu, 16, 32, 128, 128) == 12 * 32 * 128 * 128 * 4


def test_offsets_of_a_size_query():
    size = ssd.ssd_linattn_chunk_scan_varlen_workspace_size
    for cu in ([], [[0, 4]]):
        with pytest.raises(ValueError):
            size(cu, 1, 1, 64, 64)
    with pytest.raises(ssd.SsdError) as e:               # one offset, not 0
        size(5, 1, 1, 64, 64)
    assert e.value.code == 2
