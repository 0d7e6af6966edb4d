"""Calls of the attention layers that are allowed but rare: unaligned tokens, shared
keys, the same tensor twice, batches of odd strides, several calls at once."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import F, U, host, lin_bounds, randn, within
from oracle import attention as att
from test_gpu_attn import check as check_attn, prompt, step_inputs
from test_gpu_linattn import check as check_lin, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_linear_step_on_unaligned_tokens(io):
    """q, k, v one element off and odd elements apart; o one element off."""
    B, hk, hv, dk, dv = 3, 2, 4, 64, 128
    q, k, v, g, S0 = inputs(1, io, (B,), hk, hv, dk, dv, B)

    def rows(x):
        n = x[0].numel()
        buf = torch.zeros(1 + B * (n + 7), dtype=x.dtype, device="cuda")
        t = buf[1:].view(B, n + 7)[:, :n].unflatten(1, x.shape[1:])
        t.copy_(x)
        assert t.data_ptr() % 16 and not t.is_contiguous()
        return t

    st = S0[0].clone()
    o = torch.zeros(1 + v[0].numel(), dtype=v[0].dtype, device="cuda")[1:].view(v[0].shape)
    ssd.ssd_linattn_decode_step(rows(q[0]), rows(k[0]), rows(v[0]), g[0], st, o=o, scale=0.5)
    for b in range(B):
        ro, rS, ao, A = att.linattn(q[1][b:b + 1], k[1][b:b + 1], v[1][b:b + 1], g[1], S0[1][b], 0.5)
        _, bS = lin_bounds(io, ro, ao, A, 1, dk)
        within(o[b:b + 1], ro, (dk + 16) * F * ao + U[io] * np.abs(ro) + 1e-30, f"b={b}: o")
        within(st[b], rS, bS, f"b={b}: state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,L", [(3, 1), (1, 40), (2, 33)])
def test_linear_scan_of_batches_of_slices(io, B, L):
    """Batch rows and tokens evenly apart, in batches and prompts of one."""
    q, k, v, g, S0 = inputs(B + L, io, (B, L), 1, 2, 64, 64, B, sliced=True)
    o, fin = ssd.ssd_linattn_chunk_scan(q[0], k[0], v[0], g[0], initial_state=S0[0])
    for b in range(B):
        check_lin(io, o[b], fin[b], q[1][b], k[1][b], v[1][b], g[1], S0[1][b], 1.0, f"b={b}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_one_tensor_as_query_key_and_value(io):
    gen = torch.Generator().manual_seed(5)
    x = randn(gen, 90, 2, 64, io=io, scale=0.3)
    g = torch.tensor([-0.1, -0.01], device="cuda")
    o, fin = ssd.ssd_linattn_chunk_scan_varlen(x[0], x[0], x[0], g, [0, 90])
    check_lin(io, o, fin[0], x[1], x[1], x[1], host(g), None, 1.0, "scan")
    check_attn(io, ssd.ssd_attn_prefill(x[0], x[0], x[0], [0, 90]), x[1], x[1], x[1], 0.125, "prefill")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sequences_that_share_keys(io):
    """Several continuations of one cached prefix, and key ranges that overlap."""
    lq, starts, lens = [20, 33, 1, 7], [10, 10, 0, 50], [120, 100, 150, 60]
    cu = np.concatenate([[0], np.cumsum(lq)])
    q, k, v = prompt(6, io, int(cu[-1]), 150, 4, 2, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], cu, kv_starts=starts, kv_lens=lens)
    for i in range(4):
        s = slice(starts[i], starts[i] + lens[i])
        check_attn(io, o[cu[i]:cu[i + 1]], q[1][cu[i]:cu[i + 1]], k[1][s], v[1][s], 0.125, f"seq {i}")


def test_steps_and_prefills_at_once():
    """Calls in flight on two streams, each with its own caches and workspace, several
    times over; the softmax step's chunks and the scan's segments among them."""
    cases = [step_inputs(40 + i, "bf16", 3, 1500, 8, 2, 128) for i in range(2)]
    pr = [prompt(50 + i, "bf16", 400, 400, 8, 2, 128) for i in range(2)]
    n = torch.tensor([1400, 700, 3], dtype=torch.int32, device="cuda")

    def run(c, p, kc, vc, stream=None):
        return (ssd.ssd_attn_decode_step(c[0][0], c[1][0], c[2][0], kc, vc, n, stream=stream),
                ssd.ssd_attn_prefill(p[0][0], p[1][0], p[2][0], [0, 150, 400], stream=stream))

    want = [run(c, p, c[3][0].clone(), c[4][0].clone()) for c, p in zip(cases, pr)]
    caches = [(c[3][0].clone(), c[4][0].clone()) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[run(c, p, *m, stream=s) for c, p, m, s in zip(cases, pr, caches, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_of_one_step():
    """Two captured steps with workspaces of their own, replayed in turn and after eager
    work between them."""
    q, k, v, kc, vc = step_inputs(70, "bf16", 2, 900, 4, 2, 64)
    n = torch.tensor([880, 100], dtype=torch.int32, device="cuda")
    want = ssd.ssd_attn_decode_step(q[0], k[0], v[0], kc[0], vc[0], n)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ssd.ssd_attn_decode_step(q[0], k[0], v[0], kc[0], vc[0], n))
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)
            assert torch.equal(ssd.ssd_attn_decode_step(q[0], k[0], v[0], kc[0], vc[0], n), want)


def test_other_types_are_refused_by_name():
    x, g = torch.zeros(2, 8, 1, 64, dtype=torch.float16, device="cuda"), torch.zeros(1, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: ssd.ssd_linattn_chunk_scan(x, x, x, g),
                 lambda: ssd.ssd_linattn_decode_step(x[:, 0], x[:, 0], x[:, 0], g, torch.zeros(2, 1, 64, 64, device="cuda")),
                 lambda: ssd.ssd_attn_prefill(x[0], x[0], x[0], [0, 8]),
                 lambda: ssd.ssd_attn_decode_step(x[:, 0], x[:, 0], x[:, 0], x, x.clone(), n),
                 lambda: ssd.ssd_gdn_decode_step(*(x[:, 0].contiguous(),) * 3, g.expand(2, 1).contiguous(),
                                                 g.expand(2, 1).contiguous(), torch.zeros(2, 1, 64, 64, device="cuda"))):
        with pytest.raises(TypeError, match="q/k/v must be bfloat16 or float32"):
            call()
