"""The attention layers on arrays of more than 2^31 elements: the sequence that is
checked lies past them, in rows far apart or after a long one."""
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import host, lin_bounds, within
from oracle import attention as att
from test_gpu_attn import check as check_attn
from test_gpu_linattn import check as check_lin

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows_apart(io, rows, stride, widths):
    """Tensors [rows, heads, dim] that are slices of rows `stride` elements apart."""
    buf = torch.empty(rows, stride, dtype=DT[io], device="cuda")
    gen = torch.Generator().manual_seed(rows)
    out, at = [], stride - sum(h * d for h, d in widths)   # (at the rows' ends: the last one ends the buffer)
    for h, d in widths:
        x = buf[:, at:at + h * d]
        x.copy_(torch.randn(rows, h * d, generator=gen).to(DT[io]))
        out.append(x.unflatten(-1, (h, d)))
        at += h * d
    return out


@pytest.mark.parametrize("io,rows,stride", [("bf16", 600, 1 << 22), ("bf16", 1100, (1 << 21) + 8), ("f32", 530, 1 << 22)])
def test_rows_far_apart(io, rows, stride):
    """The largest strides: a tile's rows span up to 1 GB."""
    dk = dv = d = 64
    q, k, v = rows_apart(io, rows, stride, [(1, dk), (1, dk), (2, dv)])
    assert rows * stride > 1 << 31
    g = torch.tensor([-0.02, -0.3], device="cuda")
    o, fin = ssd.ssd_linattn_chunk_scan_varlen(q, k, v, g, [0, rows - 200, rows], scale=0.125)
    s = slice(rows - 200, rows)
    check_lin(io, o[s], fin[1], host(q[s]), host(k[s]), host(v[s]), host(g), None, 0.125, "scan")
    o = ssd.ssd_attn_prefill(v, q, k, [0, rows - 200, rows])
    check_attn(io, o[s], host(v[s]), host(q[s]), host(k[s]), d ** -0.5, "prefill")


def test_scan_after_a_long_sequence():
    """v and o of more than 2^31 elements: the second sequence's rows lie past them."""
    n, L, hk, hv, dk, dv = 1 << 19, 130, 1, 32, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = lambda h, d: torch.randn(n + L, h, d, generator=gen, device="cuda", dtype=torch.bfloat16) * d ** -0.5
    q, k, v = new(hk, dk), new(hk, dk), new(hv, dv)
    assert (n * hv * dv) >> 31
    g = -torch.exp2(-8.0 * torch.arange(1, hv + 1, device="cuda") / hv)
    o, fin = ssd.ssd_linattn_chunk_scan_varlen(q, k, v, g, [0, n, n + L])
    s = slice(n, n + L)
    check_lin("bf16", o[s], fin[1], host(q[s]), host(k[s]), host(v[s]), host(g), None, 1.0, "after a long one")
    # the long one's last tokens, in a head that forgets all before them (e^-0.84 a token)
    t = slice(n - 200, n)
    ro, _, ao, A = att.linattn(host(q[t]), host(k[t]), host(v[t])[:, :1], host(g[:1]))
    bound, _ = lin_bounds("bf16", ro, ao, A, 200, dk)
    within(o[n - 50:n, :1], ro[150:], bound[150:], "the long one's end")


def test_prefill_past_2_31_elements():
    """Queries, outputs, keys and values past 2^31 elements, after a sequence that has no
    keys."""
    n, nk, L, hq, hkv, d = 1 << 19, 1 << 21, 90, 32, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    q = torch.zeros(n + L, hq, d, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(nk + L, hkv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for x, at in ((q, n), (k, nk), (v, nk)):
        x[at:] = torch.randn(L, *x.shape[1:], generator=gen, device="cuda").to(x.dtype)
    assert (n * hq * d) >> 31 and (nk * hkv * d) >> 31
    o = ssd.ssd_attn_prefill(q, k, v, [0, n, n + L], kv_starts=[0, nk], kv_lens=[0, L])
    check_attn("bf16", o[n:], host(q[n:]), host(k[nk:]), host(v[nk:]), d ** -0.5, "the last rows")
    assert not o[:n].any()
