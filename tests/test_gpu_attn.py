"""GPU parity of the softmax-attention operators against the fp64 oracle."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import attn_bound, fused, host, randn, within
from oracle import attention as att

pytestmark = pytest.mark.gpu


def prompt(seed, io, lq, lk, hq, hkv, d, sliced=False):
    gen = torch.Generator().manual_seed(seed)
    q = randn(gen, lq, hq, d, io=io)
    if sliced:
        k, v = fused(gen, (lk,), [(hkv, d), (hkv, d)], io, (1.0, 1.0))
    else:
        k, v = randn(gen, lk, hkv, d, io=io), randn(gen, lk, hkv, d, io=io)
    return q, k, v


def check(io, o, q, k, v, scale, what):
    ro, ao, big = att.attn(q, k, v, scale)
    within(o, ro, attn_bound(io, ro, ao, big, k.shape[0], q.shape[2]), what)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 64, 65, 130, 257])
def test_lengths(io, L):
    q, k, v = prompt(L, io, L, L, 2, 1, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], [0, L])
    check(io, o, q[1], k[1], v[1], 0.125, f"L={L}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (6, 2, 128), (7, 1, 64), (4, 4, 256), (33, 1, 64), (8, 1, 256)])
def test_head_layouts(io, hq, hkv, d):
    q, k, v = prompt(hq + d, io, 75, 75, hq, hkv, d, sliced=True)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], [0, 75])
    check(io, o, q[1], k[1], v[1], d ** -0.5, f"{hq}/{hkv} x {d}")


@pytest.mark.parametrize("io,hq,hkv,d", [("bf16", 32, 32, 64), ("bf16", 66, 22, 128), ("bf16", 32, 32, 256),
                                         ("f32", 50, 50, 64), ("f32", 100, 25, 128), ("f32", 50, 50, 256)])
def test_many_rows(io, hq, hkv, d):
    """Enough rows for the kernel of large row blocks (the small cases take the
    one that splits the keys): several sequences, some on cached prefixes, one that
    sees nothing at first, ragged everywhere."""
    lq, lk = [300, 1, 64, 33, 150, 129], [300, 50, 64, 97, 100, 129]
    starts = [0, 300, 350, 414, 511, 611]
    cu = np.concatenate([[0], np.cumsum(lq)])
    q, k, v = prompt(hq + d, io, int(cu[-1]), 740, hq, hkv, d, sliced=True)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], cu, kv_starts=starts, kv_lens=lk)
    for i in range(len(lq)):
        s = slice(starts[i], starts[i] + lk[i])
        check(io, o[cu[i]:cu[i + 1]], q[1][cu[i]:cu[i + 1]], k[1][s], v[1][s], d ** -0.5, f"seq {i}")


def test_many_rows_growing_scores():
    """The large-block kernel's running maximum over 10 tiles."""
    L, h, d = 600, 32, 64
    q, k, v = prompt(5, "bf16", L, L, h, h, d)
    kk = (torch.ones(L, h, d) * torch.arange(L)[:, None, None] / 8).to(torch.bfloat16)
    qq = torch.ones(L, h, d, dtype=torch.bfloat16)
    for kx in (kk, kk.flip(0).contiguous()):
        o = ssd.ssd_attn_prefill(qq.cuda(), kx.cuda(), v[0], [0, L])
        for j in (0, h - 1):
            check("bf16", o[:, j:j + 1], qq[:, :1].double().numpy(), kx[:, j:j + 1].double().numpy(),
                  v[1][:, j:j + 1], d ** -0.5, f"head {j}")


@pytest.mark.parametrize("scale", [0.0, 1e-40, -0.3, 2.0])
def test_scales(scale):
    q, k, v = prompt(3, "f32", 70, 70, 2, 2, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], [0, 70], scale=scale)
    check("f32", o, q[1], k[1], v[1], scale, f"scale {scale}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_growing_scores(io):
    """The running maximum grows by far more than the slack at every tile."""
    L, d = 300, 64
    q, k, v = prompt(4, io, L, L, 1, 1, d)
    kk = (torch.ones(L, 1, d) * torch.arange(L)[:, None, None] / 8).to(k[0].dtype)
    qq = torch.ones(L, 1, d).to(q[0].dtype)
    o = ssd.ssd_attn_prefill(qq.cuda(), kk.cuda(), v[0], [0, L])
    check(io, o, qq.double().numpy(), kk.double().numpy(), v[1], d ** -0.5, "growing")
    o = ssd.ssd_attn_prefill(qq.cuda(), kk.flip(0).contiguous().cuda(), v[0], [0, L])
    check(io, o, qq.double().numpy(), kk.flip(0).double().numpy(), v[1], d ** -0.5, "shrinking")


def test_scores_far_below_zero():
    """Every score of a row near -1e34: still a softmax, in both prefill kernels and
    the decode step."""
    for hkv in (1, 40):
        q, k, v = prompt(8, "f32", 512, 512, hkv, hkv, 64)
        qq, kk = torch.full_like(q[0], 1e16), torch.full_like(k[0], -1e16)
        kk *= (1 + torch.arange(512, device="cuda") / 64)[:, None, None]    # the first key scores highest by far
        o = ssd.ssd_attn_prefill(qq, kk, v[0], [0, 512])
        assert torch.equal(o, v[0][:1].expand(512, -1, -1))
    o = ssd.ssd_attn_decode_step(qq[:1], kk[511:], v[0][511:], kk[None].clone(), v[0][None].clone(),
                                 torch.tensor([511], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, v[0][:1])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_packed_on_cached_prefixes(io):
    """Sequences of all sizes, in any order, some empty, some on cached keys, some
    with fewer keys than queries (rows that see none)."""
    lq = [40, 0, 1, 100, 65, 3, 30, 1]
    lk = [40, 5, 1, 180, 65, 0, 20, 333]
    starts = [500, 0, 499, 0, 700, 9, 300, 160]
    cu = np.concatenate([[0], np.cumsum(lq)])
    q, k, v = prompt(6, io, int(cu[-1]), 800, 4, 2, 128, sliced=True)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], cu, kv_starts=starts, kv_lens=lk, scale=0.1)
    for i, n in enumerate(lq):
        if n:
            s = slice(starts[i], starts[i] + lk[i])
            check(io, o[cu[i]:cu[i + 1]], q[1][cu[i]:cu[i + 1]], k[1][s], v[1][s], 0.1, f"seq {i}")
    assert not o[cu[5]:cu[6]].any() and not o[cu[6]:cu[6] + 10].any()


def test_many_sequences():
    """More sequences than one launch takes."""
    lens = [(5 * i) % 7 for i in range(300)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = prompt(7, "bf16", int(cu[-1]), int(cu[-1]), 2, 1, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], cu)
    for i, n in enumerate(lens):
        if n:
            s = slice(cu[i], cu[i + 1])
            check("bf16", o[s], q[1][s], k[1][s], v[1][s], 0.125, f"seq {i}")


def test_nothing_outside_the_sequences_is_read_or_written():
    nan = float("nan")
    L, M = 70, 200
    q, k, v = prompt(8, "bf16", L, L, 2, 1, 64)
    kb, vb = (torch.full((M, 1, 64), nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb[50:50 + L], vb[50:50 + L] = k[0], v[0]
    ob = torch.full((M, 2, 64), nan, dtype=torch.bfloat16, device="cuda")
    ssd.ssd_attn_prefill(q[0], kb, vb, [0, L], kv_starts=[50], kv_lens=[L], o=ob[10:10 + L])
    check("bf16", ob[10:10 + L], q[1], k[1], v[1], 0.125, "inside")
    assert ob[:10].isnan().all() and ob[10 + L:].isnan().all()


@pytest.mark.parametrize("io,hq", [("bf16", 2), ("bf16", 66), ("f32", 2), ("f32", 80)])
def test_non_finite_keys_and_values(io, hq):
    """A bad value reaches its own sequence from at most 63 queries before its token
    on, a bad key only queries that see it."""
    cu = [0, 260, 520]
    q, k, v = prompt(21, io, 520, 520, hq, hq, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], cu)
    for bad in (float("inf"), float("nan")):
        kx, vx = k[0].clone(), v[0].clone()
        kx[100], vx[100] = bad, bad
        assert torch.equal(ssd.ssd_attn_prefill(q[0], kx, v[0], cu)[:100], o[:100])
        ox = ssd.ssd_attn_prefill(q[0], k[0], vx, cu)
        assert torch.equal(ox[:37], o[:37]) and torch.equal(ox[260:], o[260:])
        assert not ox[100:260].isfinite().any()


def test_prefill_no_rows():
    z = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert ssd.ssd_attn_prefill(z, z[:, :1], z[:, :1], [0]).shape == z.shape
    assert ssd.ssd_attn_prefill(z, z[:, :1], z[:, :1], [0, 0, 0]).shape == z.shape


def step_inputs(seed, io, B, M, hq, hkv, d):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = fused(gen, (B,), [(hq, d), (hkv, d), (hkv, d)], io, (1.0, 1.0, 1.0))
    kc, vc = randn(gen, B, M, hkv, d, io=io), randn(gen, B, M, hkv, d, io=io)
    return q, k, v, kc, vc


def check_step(io, q, k, v, kc, vc, lengths, scale=None):
    """A step over caches whose rows from lengths[b] on hold NaN."""
    B, M, hkv, d = kc[1].shape
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kg, vg = kc[0].clone(), vc[0].clone()
    for b, at in enumerate(lengths):
        if 0 <= at < M:
            kg[b, at:], vg[b, at:] = float("nan"), float("nan")
    kw, vw = kg.clone(), vg.clone()
    o = ssd.ssd_attn_decode_step(q[0], k[0], v[0], kg, vg, n, scale=scale)
    s = d ** -0.5 if scale is None else scale
    for b, at in enumerate(lengths):
        if not 0 <= at < M:
            assert not o[b].any()
            continue
        kw[b, at], vw[b, at] = k[0][b], v[0][b]
        kk = np.concatenate([kc[1][b, :at], k[1][b:b + 1]])
        vv = np.concatenate([vc[1][b, :at], v[1][b:b + 1]])
        check(io, o[b:b + 1], q[1][b:b + 1], kk, vv, s, f"b={b} at={at}")
    # the new rows are in the caches, and nothing else has changed
    assert torch.equal(kg.nan_to_num(123.0), kw.nan_to_num(123.0))
    assert torch.equal(vg.nan_to_num(123.0), vw.nan_to_num(123.0))
    assert torch.equal(n.cpu(), torch.tensor(lengths, dtype=torch.int32))
    return o


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_step_lengths(io):
    M = 300
    lengths = [0, 1, 31, 32, 33, 127, 128, 129, 255, 256, 298, 299, 300, -1, 2 ** 31 - 1, -2 ** 31]
    q, k, v, kc, vc = step_inputs(1, io, len(lengths), M, 4, 2, 64)
    check_step(io, q, k, v, kc, vc, lengths)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (6, 2, 128), (3, 3, 256), (40, 1, 64), (70, 1, 128), (16, 2, 256)])
def test_step_head_layouts(io, hq, hkv, d):
    q, k, v, kc, vc = step_inputs(hq + d, io, 2, 150, hq, hkv, d)
    check_step(io, q, k, v, kc, vc, [149, 77], scale=-0.2)


def test_step_short_capacities():
    """A cache within one work-group's chunk (no join), and one just past it."""
    for M in (1, 5, 128, 129):
        q, k, v, kc, vc = step_inputs(M, "bf16", 3, M, 2, 1, 64)
        check_step("bf16", q, k, v, kc, vc, [M - 1, 0, M])


def test_step_without_capacity():
    q, k, v, _, _ = step_inputs(3, "bf16", 2, 1, 4, 2, 64)
    c = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    assert not ssd.ssd_attn_decode_step(q[0], k[0], v[0], c, c.clone(), n).any()


def test_step_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last sequence's rows lie past it."""
    B, M, hkv, d = 3, 1 << 20, 8, 128                     # 3 x 2^30 elements
    gen = torch.Generator().manual_seed(5)
    q, k, v = (randn(gen, B, h, d, io="bf16") for h in (16, hkv, hkv))
    kc = torch.zeros(B, M, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    at = M - 2
    kt, vt = randn(gen, 40, hkv, d, io="bf16"), randn(gen, 40, hkv, d, io="bf16")
    kc[2, at - 40:at], vc[2, at - 40:at] = kt[0] * 4, vt[0]
    # the zero keys before score 0 and have value 0: they only add to the sum
    n = torch.tensor([-1, 3, at], dtype=torch.int32, device="cuda")
    o = ssd.ssd_attn_decode_step(q[0], k[0], v[0], kc, vc, n)
    assert torch.equal(kc[2, at], k[0][2]) and torch.equal(vc[2, at], v[0][2])
    assert not kc[2, at + 1:].any() and not kc[0].any() and not o[0].any()
    kk = np.concatenate([host(kc[2, at - 40:at]), k[1][2:3]])
    vv = np.concatenate([vt[1], v[1][2:3]])
    for h in (0, 15):
        a = d ** -0.5 * (kk[:, h // 2] @ q[1][2, h])
        p = np.exp(a - a.max())
        rest = (at - 40) * np.exp(-a.max())
        want = p @ vv[:, h // 2] / (p.sum() + rest)
        size = p @ np.abs(vv[:, h // 2]) / (p.sum() + rest)
        # bf16 roundings as in attn_bound; a sum of 2^20 equal terms in fp32 over 4096
        # partial sums of 256 each is off by some 2^-15 at most
        assert (np.abs(host(o[2, h]) - want) <= 2.0 ** -8 * (np.abs(want) + 1.01 * size) + 2.0 ** -12 * size).all()


def test_step_long_cache():
    q, k, v, kc, vc = step_inputs(77, "bf16", 2, 9000, 8, 2, 64)
    check_step("bf16", q, k, v, kc, vc, [8999, 4100])


def test_prefill_then_steps_agree():
    """A prompt whose keys are in the padded cache, then single tokens: every row
    against the oracle of the whole sequence."""
    L, n, M, hq, hkv, d = 90, 4, 128, 4, 2, 128
    q, k, v = prompt(17, "bf16", L + n, L + n, hq, hkv, d)
    kc = torch.full((2, M, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    kc[1, :L], vc[1, :L] = k[0][:L], v[0][:L]
    flat = lambda c: c.view(2 * M, hkv, d)
    o = [ssd.ssd_attn_prefill(q[0][:50], flat(kc), flat(vc), [0, 50], kv_starts=[M], kv_lens=[50]),
         ssd.ssd_attn_prefill(q[0][50:L], flat(kc), flat(vc), [0, L - 50], kv_starts=[M], kv_lens=[L])]
    lengths = torch.tensor([-1, L], dtype=torch.int32, device="cuda")
    for t in range(L, L + n):
        rows = [x[0][t:t + 1].expand(2, -1, -1).contiguous() for x in (q, k, v)]
        o.append(ssd.ssd_attn_decode_step(*rows, kc, vc, lengths)[1:])
        lengths[1] += 1
    check("bf16", torch.cat(o), q[1], k[1], v[1], d ** -0.5, "prompt in parts + steps")


def test_replayed_on_another_stream():
    """Captured together; replays follow the lengths on the device."""
    q, k, v, kc, vc = step_inputs(23, "bf16", 2, 400, 4, 2, 128)
    pq, pk, pv = prompt(24, "bf16", 100, 100, 4, 2, 128)
    lengths = torch.tensor([10, 390], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    po = ssd.ssd_attn_prefill(pq[0], pk[0], pv[0], [0, 30, 100], stream=s)
    torch.cuda.synchronize()
    want_p = ssd.ssd_attn_prefill(pq[0], pk[0], pv[0], [0, 30, 100])
    torch.cuda.synchronize()
    assert torch.equal(po, want_p)
    want, ke, ve, n = [], kc[0].clone(), vc[0].clone(), lengths.clone()
    for _ in range(3):
        want.append(ssd.ssd_attn_decode_step(q[0], k[0], v[0], ke, ve, n).clone())
        n += 1
    ws = torch.empty(ssd.ssd_attn_decode_workspace_size(2, 400, 4, 2, 128), dtype=torch.uint8, device="cuda")
    o, kg, vg = torch.empty_like(want[0]), kc[0].clone(), vc[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_attn_prefill(pq[0], pk[0], pv[0], [0, 30, 100], o=po)
        ssd.ssd_attn_decode_step(q[0], k[0], v[0], kg, vg, lengths, o=o, workspace=ws)
    for i in range(3):
        po.zero_(), o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i]) and torch.equal(po, want_p)
        lengths += 1
    assert torch.equal(kg, ke) and torch.equal(vg, ve)


def test_refusals():
    q, k, v = prompt(31, "bf16", 16, 16, 4, 2, 64)
    q, k, v = q[0], k[0], v[0]
    pre = ssd.ssd_attn_prefill

    def code(fn, *a, **kw):
        with pytest.raises(ssd.SsdError) as e:
            fn(*a, **kw)
        return e.value.code

    for cu in ([0, 15], [1, 16], [0, 9, 8, 16], [0, 17, 16]):
        assert code(pre, q, k, v, cu) == 2
    for st, ln in (([-1], [4]), ([0], [-1]), ([0], [17]), ([10], [7]), ([17], [0]), ([2 ** 62], [2 ** 62])):
        assert code(pre, q, k, v, [0, 16], kv_starts=st, kv_lens=ln) == 2
    assert code(pre, q, k, v, [0, 16], kv_starts=[0]) == 1
    assert code(pre, q, k[:8], v[:8], [0, 16]) == 2
    assert code(pre, q, k, v, [0, 16], o=q) == 4
    assert code(pre, q, k, v, [0, 16], scale=float("inf")) == 3
    assert code(pre, q[:, :3].contiguous(), k, v, [0, 16]) == 2
    assert code(pre, *(t[..., :32].contiguous() for t in (q, k, v)), [0, 16]) == 3
    with pytest.raises(ValueError):
        pre(q, k, v[:8], [0, 16])
    with pytest.raises(ValueError):
        pre(q, k, v, [0, 16], kv_starts=[0, 1], kv_lens=[1, 1])
    with pytest.raises(TypeError):
        pre(q, k.float(), v, [0, 16])
    with pytest.raises(ValueError):
        pre(q, k, v, [])
    kc = torch.zeros(16, 256, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    n = torch.zeros(16, dtype=torch.int32, device="cuda")
    step = ssd.ssd_attn_decode_step
    assert code(step, q, k, v, kc, kc, n) == 4
    assert code(step, q, k, v, kc, vc, n, o=q) == 4
    assert code(step, q, k, v, kc, vc, n, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")) == 5
    with pytest.raises(TypeError):
        step(q, k, v, kc, vc, n.long())
    with pytest.raises(ValueError):
        step(q, k, v, kc, vc[:, :8], n)
    with pytest.raises(ValueError):
        step(q, k, v, kc, vc, n[:4])
    assert not kc.any() and not vc.any()
