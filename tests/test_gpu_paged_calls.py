"""The paged-cache calls together, as a serving program makes them, and calls that are
allowed but rare: captured and replayed, at once on two streams, refused."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import DT, F, U, host, randn
from oracle import paged as orc
from paged_cases import Cache, check_decode, turn_bound

pytestmark = pytest.mark.gpu


class Layer:
    """A small softmax layer's inputs: prompts and then one token at a time, normed and rotated."""

    def __init__(self, seed, io, lens, steps, Hq=6, Hkv=2, D=64, page=16):
        gen = torch.Generator().manual_seed(seed)
        self.io, self.lens, self.Hq, self.Hkv, self.D, self.page = io, lens, Hq, Hkv, D, page
        B, T = len(lens), sum(lens)
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        self.prompt = [randn(gen, T, h, D, io=io) for h in (Hq, Hkv, Hkv)]
        self.tokens = [[randn(gen, B, h, D, io=io) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
        self.f = (1e4 ** (-2 * np.arange(D // 2) / D)).astype(np.float32)
        self.w = [(1 + 0.2 * np.random.default_rng(seed + i).standard_normal(D)).astype(np.float32) for i in (0, 1)]
        self.width = -(-(max(lens) + steps) // page)
        self.n = B * self.width
        self.table = np.random.default_rng(seed).permutation(self.n).reshape(B, -1).astype(np.int32)
        self.turn = dict(inv_freq=torch.from_numpy(self.f).cuda(), q_weight=torch.from_numpy(self.w[0]).cuda(),
                         k_weight=torch.from_numpy(self.w[1]).cuda())

    def cache(self, bits):
        shape = (self.n, self.Hkv, self.page, self.D)
        if bits == 4:
            c = [torch.zeros(shape[:3] + (self.D // 2,), dtype=torch.uint8, device="cuda") for _ in "kv"]
            s = [torch.zeros(shape[:3] + (self.D // 64, 2), dtype=torch.half, device="cuda") for _ in "kv"]
            return (*c, torch.from_numpy(self.table).cuda()), dict(k_scales=s[0], v_scales=s[1])
        return (*(torch.zeros(shape, dtype=DT[self.io], device="cuda") for _ in "kv"), torch.from_numpy(self.table).cuda()), {}

    def lengths(self):
        return torch.zeros(len(self.lens), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prompts_then_steps_match_the_padded_cache(io):
    """The same layer over a paged cache and over a padded one (rotated by
    ssd_attn_qk_norm_rope): queries, keys and prompts to the bit, steps up to rounding."""
    L = Layer(1, io, [40, 1, 90, 17], 5)
    B = len(L.lens)
    pages, sc = L.cache(16)
    n = L.lengths()
    ko = torch.empty_like(L.prompt[1][0])
    q = ssd.ssd_attn_paged_append(*(x[0] for x in L.prompt), *pages, n, cu_seqlens=L.cu, k_out=ko, **L.turn)
    pos = torch.from_numpy(np.concatenate([np.arange(m) for m in L.lens]).astype(np.int32)).cuda()
    q2, k2 = ssd.ssd_attn_qk_norm_rope(L.prompt[0][0], L.prompt[1][0], pos, **L.turn)
    assert torch.equal(q, q2) and torch.equal(ko, k2)
    o = ssd.ssd_attn_prefill(q, ko, L.prompt[2][0], L.cu)
    kr, vr = ssd.ssd_attn_paged_gather(*pages, L.cu)
    assert torch.equal(kr, ko) and torch.equal(vr, L.prompt[2][0])
    assert torch.equal(o, ssd.ssd_attn_prefill(q, kr, vr, L.cu))
    M = L.width * L.page
    kc, vc = (torch.zeros(B, M, L.Hkv, L.D, dtype=DT[io], device="cuda") for _ in "kv")
    for b in range(B):
        kc[b, :L.lens[b]], vc[b, :L.lens[b]] = kr[L.cu[b]:L.cu[b + 1]], vr[L.cu[b]:L.cu[b + 1]]
    n = torch.tensor(L.lens, dtype=torch.int32, device="cuda")
    for qt, kt, vt in L.tokens:
        qs = ssd.ssd_attn_paged_append(qt[0], kt[0], vt[0], *pages, n, **L.turn)
        o = ssd.ssd_attn_paged_decode_step(qs, *pages, n)
        q2, k2 = ssd.ssd_attn_qk_norm_rope(qt[0], kt[0], n, **L.turn)
        assert torch.equal(qs, q2)
        o2 = ssd.ssd_attn_decode_step(q2, k2, vt[0], kc, vc, n)
        # two sums of the same terms, each rounded once to the output type; fp32 sums and scores
        # of a hundred terms of size 64 (D) in other orders
        tol = 2 * U[io] * o2.float().abs().max().item() + (2.0 ** -15 if io == "bf16" else 2000 * F) * 4
        assert (o.float() - o2.float()).abs().max().item() <= tol
        n += 1


@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_in_parts(bits):
    """A prompt appended in two parts, the second attending the first as it lies in the pages."""
    io = "bf16"
    L = Layer(2, io, [100], 0, D=128)
    pages, sc = L.cache(bits)
    cut, n = 37, L.lengths()
    q, k, v = (x[0] for x in L.prompt)
    ssd.ssd_attn_paged_append(q[:cut], k[:cut], v[:cut], *pages, n, cu_seqlens=[0, cut], **sc, **L.turn)
    qo = ssd.ssd_attn_paged_append(q[cut:], k[cut:], v[cut:], *pages, n + cut, cu_seqlens=[0, 100 - cut], **sc, **L.turn)
    kr, vr = ssd.ssd_attn_paged_gather(*pages, [0, 100], **sc)
    o = ssd.ssd_attn_prefill(qo, kr, vr, [0, 100 - cut], kv_starts=[0], kv_lens=[100])
    whole, sc2 = L.cache(bits)
    qa = ssd.ssd_attn_paged_append(q, k, v, *whole, n, cu_seqlens=[0, 100], **sc2, **L.turn)
    ka, va = ssd.ssd_attn_paged_gather(*whole, [0, 100], **sc2)
    assert torch.equal(qo, qa[cut:]) and torch.equal(kr, ka) and torch.equal(vr, va)
    # (other row blocks: the tiles' sums are rounded in other orders)
    want = ssd.ssd_attn_prefill(qa, ka, va, [0, 100])[cut:]
    assert (o.float() - want.float()).abs().max().item() <= 4 * U[io] * want.float().abs().max().item()
    # a step at the last token attends what the prefill's last query did
    last = ssd.ssd_attn_paged_decode_step(qo[-1:], *pages, n + 99, **sc)
    assert (last.float() - o[-1:].float()).abs().max().item() <= 4 * U[io] * o[-1].float().abs().max().item()


@pytest.mark.parametrize("io,bits", [("bf16", 16), ("bf16", 4), ("f32", 16)])
def test_a_captured_step(io, bits):
    """Append and attention of one token captured once and replayed for the following tokens,
    the lengths counted up by the graph; eager work on another cache in between."""
    L = Layer(3, io, [30, 5], 6)
    pages, sc = L.cache(bits)
    eager, sce = L.cache(bits)
    n = L.lengths()
    for c, s in ((pages, sc), (eager, sce)):
        ssd.ssd_attn_paged_append(*(x[0] for x in L.prompt), *c, n, cu_seqlens=L.cu, **s, **L.turn)
    start = torch.tensor(L.lens, dtype=torch.int32, device="cuda")
    n, ne = start.clone(), start.clone()
    buf = [torch.zeros_like(x[0]) for x in L.tokens[0]]

    def one(c, s, n):
        q = ssd.ssd_attn_paged_append(*buf, *c, n, **s, **L.turn)
        o = ssd.ssd_attn_paged_decode_step(q, *c, n, **s)
        n += 1
        return o

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = one(pages, sc, n)
    n.copy_(start)
    for tok in L.tokens:
        for b, x in zip(buf, tok):
            b.copy_(x[0])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = one(eager, sce, ne)
        assert torch.equal(out, want) and torch.equal(n, ne)
    for a, b in zip((*pages, *sc.values()), (*eager, *sce.values())):
        assert torch.equal(a, b)


def test_two_graphs_and_two_streams():
    """Steps of two layers captured apart and replayed in turn, and in flight at once on two
    streams: each has a workspace of its own."""
    caches = [Cache(30 + i, "bf16", bits, [3000, 200], 2, 128, 16) for i, bits in enumerate((16, 4))]
    qs = [randn(torch.Generator().manual_seed(40 + i), 2, 8, 128, io="bf16")[0] for i in range(2)]
    n = torch.tensor([2999, 150], dtype=torch.int32, device="cuda")

    def run(c, q, stream=None):
        pos, kw = c.args()
        return ssd.ssd_attn_paged_decode_step(q, *pos, n, stream=stream, **kw)

    want = [run(c, q) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[run(c, q, s) for c, q, s in zip(caches, qs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    graphs, outs = [], []
    for c, q in zip(caches, qs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(c, q))
        graphs.append(g)
    for _ in range(3):
        for g, o, w, c, q in zip(graphs, outs, want, caches, qs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w) and torch.equal(run(c, q), w)


def test_rows_on_a_stream():
    """Append, gather and norm on a stream of the caller's."""
    L = Layer(5, "bf16", [50, 20], 0)
    s = torch.cuda.Stream()
    pages, _ = L.cache(16)
    other, _ = L.cache(16)
    n = L.lengths()
    q = ssd.ssd_attn_paged_append(*(x[0] for x in L.prompt), *pages, n, cu_seqlens=L.cu, **L.turn)
    torch.cuda.synchronize()
    q2 = ssd.ssd_attn_paged_append(*(x[0] for x in L.prompt), *other, n, cu_seqlens=L.cu, stream=s, **L.turn)
    k2, v2 = ssd.ssd_attn_paged_gather(*other, L.cu, stream=s)
    pos = torch.from_numpy(np.concatenate([np.arange(m) for m in L.lens]).astype(np.int32)).cuda()
    torch.cuda.synchronize()
    q3, k3 = ssd.ssd_attn_qk_norm_rope(L.prompt[0][0], L.prompt[1][0], pos, stream=s, **L.turn)
    s.synchronize()
    assert torch.equal(q, q2) and torch.equal(q, q3) and torch.equal(k2, k3) and torch.equal(v2, L.prompt[2][0])


@pytest.mark.parametrize("bits", [16, 4])
def test_prompts_captured_and_given_outputs(bits):
    """Append of prompts and reading back captured in a graph with all outputs given, replayed on
    other inputs; the same calls eagerly in between."""
    L = Layer(7, "bf16", [33, 0, 70], 0, D=128)
    cu = L.cu
    (kp, vp, tab), sc = L.cache(bits)
    (ke, ve, _), sce = L.cache(bits)
    n = L.lengths()
    q, k, v = (x[0].clone() for x in L.prompt)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kr, vr = torch.empty_like(k), torch.empty_like(k)

    def run(kp, vp, sc, qo, ko, kr, vr):
        ssd.ssd_attn_paged_append(q, k, v, kp, vp, tab, n, cu_seqlens=cu, q_out=qo, k_out=ko, **sc, **L.turn)
        return ssd.ssd_attn_paged_gather(kp, vp, tab, cu, k=kr, v=vr, **sc)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(kp, vp, sc, qo, ko, kr, vr)
    assert got[0] is kr and got[1] is vr
    gen = torch.Generator(device="cuda").manual_seed(8)
    for _ in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(x) for x in (qo, ko, kr, vr)]
        run(ke, ve, sce, *want)
        assert all(torch.equal(x, y) for x, y in zip((qo, ko, kr, vr), want))
    for a, b in zip((kp, vp, *sc.values()), (ke, ve, *sce.values())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [16, 4])
def test_empty_batches_and_prompts(bits):
    L = Layer(9, "bf16", [5], 0, D=128)
    (kp, vp, tab), sc = L.cache(bits)
    before = [x.clone() for x in (kp, vp, *sc.values())]
    q, k, v = (x[0] for x in L.prompt)
    none = tab[:0]
    n = L.lengths()
    ssd.ssd_attn_paged_append(q[:0], k[:0], v[:0], kp, vp, none, n[:0], **sc, **L.turn)
    ssd.ssd_attn_paged_append(q[:0], k[:0], v[:0], kp, vp, tab, n, cu_seqlens=[0, 0], **sc, **L.turn)
    assert ssd.ssd_attn_paged_decode_step(q[:0], kp, vp, none, n[:0], **sc).shape == (0, L.Hq, L.D)
    kr, vr = ssd.ssd_attn_paged_gather(kp, vp, none, [0], **sc)
    assert kr.shape == vr.shape == (0, L.Hkv, L.D)
    o = ssd.ssd_attn_paged_decode_step(q[:1], kp, vp, tab, n - 1, **sc)
    assert not o.any() and all(torch.equal(x, y) for x, y in zip((kp, vp, *sc.values()), before))


def test_refusals():
    """Wrong types, shapes and devices are refused by name before anything runs."""
    L = Layer(6, "bf16", [4], 0)
    (kp, vp, tab), _ = L.cache(16)
    (k4, v4, _), s4 = L.cache(4)
    q, k, v = (x[0] for x in L.prompt)
    n, f = L.lengths(), L.turn["inv_freq"]
    half = q.half()
    step, app = ssd.ssd_attn_paged_decode_step, ssd.ssd_attn_paged_append
    for err, match, call in (
            (TypeError, "q/k must be bfloat16 or float32", lambda: ssd.ssd_attn_qk_norm_rope(half, half)),
            (ValueError, "positions is required", lambda: ssd.ssd_attn_qk_norm_rope(q, k, inv_freq=f)),
            (TypeError, "positions must be torch.int32", lambda: ssd.ssd_attn_qk_norm_rope(q, k, n.long().expand(4).contiguous(), f)),
            (ValueError, "k has shape", lambda: ssd.ssd_attn_qk_norm_rope(q, k[:3])),
            (TypeError, "q_weight must be torch.float32", lambda: ssd.ssd_attn_qk_norm_rope(q, k, q_weight=q[0, 0])),
            (ssd.SsdError, "SSD_ERR_ALIAS|overlap", lambda: ssd.ssd_attn_qk_norm_rope(q, k, q_out=q, k_out=q[:, :2])),
            (TypeError, "lengths must be torch.int32", lambda: step(q[:1], kp, vp, tab, n.long())),
            (ValueError, "lengths is on cpu", lambda: step(q[:1], kp, vp, tab, n.cpu())),
            (ValueError, "block_table has shape", lambda: step(q[:2], kp, vp, tab, n)),
            (TypeError, "block_table must be torch.int32", lambda: step(q[:1], kp, vp, tab.long(), n)),
            (TypeError, "k_pages must be torch.uint8", lambda: step(q[:1], kp, vp, tab, n, **s4)),
            (TypeError, "k_pages must be torch.bfloat16", lambda: step(q[:1], k4, v4, tab, n)),
            (ValueError, "k_pages has shape", lambda: step(q[:1], kp[..., :32].contiguous(), vp, tab, n)),
            (ValueError, "v_scales is required", lambda: step(q[:1], k4, v4, tab, n, k_scales=s4["k_scales"])),
            (ValueError, "v_pages has shape", lambda: step(q[:1], kp, vp[:, :, :8].contiguous(), tab, n)),
            (ValueError, "q_out needs q", lambda: app(None, k[:1], v[:1], kp, vp, tab, n, q_out=q[:1])),
            (ValueError, "block_table has shape", lambda: app(q, k, v, kp, vp, tab, n)),
            (ssd.SsdError, "failed", lambda: app(q, k, v, kp, vp, tab, n, cu_seqlens=[0, 3])),
            (ssd.SsdError, "failed", lambda: ssd.ssd_attn_paged_gather(kp, vp, tab, [0, L.width * 16 + 1])),
            (ssd.SsdError, "failed", lambda: ssd.ssd_attn_paged_gather(kp, vp, tab, [0, 4], starts=[-1])),
            (TypeError, "rows of", lambda: ssd.ssd_attn_paged_gather(kp, vp, tab, [0, 4], dtype=torch.float32)),
            (TypeError, "float32, got", lambda: ssd.ssd_attn_paged_gather(k4, v4, tab, [0, 4], dtype=torch.half, **s4))):
        with pytest.raises(err, match=match):
            call()
