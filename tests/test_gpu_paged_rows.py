"""Norm and rotation of queries and keys, appending to pages and reading back, against
oracle/paged.py."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import DT, F, U, fused, host, randn, within
from oracle import paged as orc
from paged_cases import NAN, Cache, turn_bound

pytestmark = pytest.mark.gpu


def freqs(R, base=10000.0):
    return (base ** (-2 * np.arange(R // 2) / R)).astype(np.float32) if R else None


def dev(x, dtype=None):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def weights(seed, D, which):
    rng = np.random.default_rng(seed)
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in "qk"]
    return [x if n in which else None for x, n in zip(w, "qk")]


def turned(x, w, pos, f, inter, eps=1e-6):
    return orc.turn_rows(x, w, eps, pos, None if f is None else f.astype(np.float64), inter)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D,R,inter,which", [(64, 64, False, "qk"), (64, 16, True, ""), (64, 0, False, "qk"),
                                             (128, 128, False, "q"), (128, 32, False, "qk"), (128, 128, True, "k"),
                                             (256, 256, False, "qk"), (256, 64, True, "qk"), (256, 8, False, "")])
@pytest.mark.parametrize("T,Hq,Hkv,sliced", [(1, 8, 2, True), (37, 5, 5, False), (3, 12, 4, True)])
def test_norm_rope(io, D, R, inter, which, T, Hq, Hkv, sliced):
    gen = torch.Generator().manual_seed(D + R + T)
    if sliced:
        q, k, _ = fused(gen, (T,), [(Hq, D), (Hkv, D), (Hkv, D)], io, (3.0, 0.2, 1.0))
    else:
        q, k = randn(gen, T, Hq, D, io=io, scale=3.0), randn(gen, T, Hkv, D, io=io, scale=0.2)
    f, (qw, kw) = freqs(R), weights(T, D, which)
    pos = np.random.default_rng(T).integers(0, 200000, T).astype(np.int32)
    qo, ko = ssd.ssd_attn_qk_norm_rope(q[0], k[0], dev(pos) if R else None, dev(f), dev(qw), dev(kw), eps=1e-5,
                                       interleaved=inter)
    assert qo.is_contiguous() and ko.is_contiguous()
    for got, x, w, what in ((qo, q[1], qw, "q"), (ko, k[1], kw, "k")):
        out, size = turned(x, w, pos, f, inter, 1e-5)
        within(got, out, turn_bound(io, out, size, pos), what)


@pytest.mark.parametrize("inter", [False, True])
def test_sines_and_cosines(inter):
    """Pairs (1, 0) become (cos, sin).  Off by the last addition's half a step, and by what goes
    into it: 2^-24 of its smaller term (at most half the result) from each of about three roundings,
    less than a step altogether; the angle's own error in fp64 stands in front of its zeros."""
    D, T = 128, 4096
    rng = np.random.default_rng(5)
    pos = rng.integers(-2 ** 17, 2 ** 17, T).astype(np.int32)
    pos[:4] = 0, 1, -1, 131071
    f = (1e6 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    f[1], f[2] = 0.0, np.float32(np.pi / 2)                           # no turn, and almost quarter turns
    x = np.zeros((T, 1, D), dtype=np.float32)
    x[..., slice(0, None, 2) if inter else slice(0, D // 2)] = 1
    t = torch.from_numpy(x).cuda()
    got = ssd.ssd_attn_qk_norm_rope(t, t, dev(pos), torch.from_numpy(f).cuda(), interleaved=inter)[0].cpu().numpy()[:, 0]
    cos, sin = (got[:, 0::2], got[:, 1::2]) if inter else (got[:, :D // 2], got[:, D // 2:])
    angle = pos.astype(np.longdouble)[:, None] * f.astype(np.longdouble)
    for y, want in ((cos, np.cos(angle)), (sin, np.sin(angle))):
        size = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64)
        # (an angle of up to 2^17 2 radians in fp64 turns: two roundings of 2^-53 of it)
        assert (np.abs(y - want) <= size + 2.0 ** -53 * 4 * np.abs(angle)).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_far_and_negative_positions(io):
    pos = np.array([2 ** 31 - 1, -(2 ** 31), -5, 0, 1, 131071, 1 << 24], dtype=np.int32)
    gen = torch.Generator().manual_seed(1)
    q, k = randn(gen, 7, 2, 128, io=io), randn(gen, 7, 1, 128, io=io)
    f = freqs(128)
    qo, ko = ssd.ssd_attn_qk_norm_rope(q[0], k[0], dev(pos), dev(f))
    for got, x in ((qo, q[1]), (ko, k[1])):
        out, size = turned(x, None, pos, f, False)
        within(got, out, turn_bound(io, out, size, pos), "far")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_in_place_on_slices(io):
    """q and k turned where they lie in one projection; v between other rows stays."""
    gen = torch.Generator().manual_seed(2)
    (q, qv), (k, kv), (v, vv) = fused(gen, (50,), [(6, 64), (2, 64), (2, 64)], io, (1.0, 1.0, 1.0))
    pos, f, (qw, kw) = np.arange(50, dtype=np.int32), freqs(64), weights(3, 64, "qk")
    a, b = ssd.ssd_attn_qk_norm_rope(q, k, dev(pos), dev(f), dev(qw), dev(kw), q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and b.data_ptr() == k.data_ptr()
    for got, x, w in ((q, qv, qw), (k, kv, kw)):
        out, size = turned(x, w, pos, f, False)
        within(got, out, turn_bound(io, out, size, pos), "in place")
    assert np.array_equal(host(v), vv)


def test_zero_rows_and_zero_heads_of_values():
    """A head of zeros stays 0 (eps > 0); no tokens do nothing."""
    q = torch.zeros(4, 2, 64, device="cuda")
    qo, ko = ssd.ssd_attn_qk_norm_rope(q, q[:, :1].contiguous(), q_weight=torch.ones(64, device="cuda"),
                                       k_weight=torch.ones(64, device="cuda"))
    assert not qo.any() and not ko.any()
    qo, ko = ssd.ssd_attn_qk_norm_rope(q[:0], q[:0, :1])
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)


def test_many_tokens():
    """More work items than waves of one launch's first pass, and heads that fill no wave."""
    gen = torch.Generator().manual_seed(3)
    T = 9000
    q, k = randn(gen, T, 7, 64, io="bf16"), randn(gen, T, 1, 64, io="bf16")
    f, pos = freqs(64), np.arange(T, dtype=np.int32)
    qo, ko = ssd.ssd_attn_qk_norm_rope(q[0], k[0], dev(pos), dev(f))
    x = np.concatenate([q[1], k[1]], axis=1)
    z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * pos[:, None, None] * f.astype(np.float64))
    want, size = np.concatenate([z.real, z.imag], axis=-1), np.tile(np.abs(x[..., :32]) + np.abs(x[..., 32:]), 2)
    within(torch.cat([qo, ko], dim=1), want, turn_bound("bf16", want, size, pos), "many")


# --------------------------------------------------------------------------
# Appending
# --------------------------------------------------------------------------
def empty_cache(seed, io, bits, B, width, page, Hkv, D, spare=2):
    """A cache of B full tables, all NaN (4 bits: bytes 255 with NaN scales)."""
    n = B * width + spare
    table = np.random.default_rng(seed).permutation(n)[:B * width].reshape(B, width).astype(np.int32)
    c = dict(table=table, n=n, page=page)
    for x in ("k", "v"):
        if bits == 4:
            c[x] = torch.full((n, Hkv, page, D // 2), 255, dtype=torch.uint8, device="cuda")
            c[x + "s"] = torch.full((n, Hkv, page, D // 64, 2), NAN, dtype=torch.half, device="cuda")
        else:
            c[x] = torch.full((n, Hkv, page, D), NAN, dtype=DT[io], device="cuda")
            c[x + "s"] = None
    return c


def check_append(io, bits, c, lens, start, q, k, v, qw, kw, f, inter, qo, pos=None, ko=None):
    """q_out and every line of the pages after an append of lens[b] tokens at rows start[b]."""
    cu = np.concatenate([[0], np.cumsum(lens)])
    row = np.concatenate([s + np.arange(n) for s, n in zip(start, lens)] + [[]]).astype(np.int64)
    at = row if pos is None else pos
    out, size = turned(q, qw, at, f, inter)
    within(qo, out, turn_bound(io, out, size, at), "q_out")
    kt, ks = turned(k, kw, at, f, inter)
    kb = turn_bound(io, kt, ks, at)
    if ko is not None:
        within(ko, kt, kb, "k_out")
    got = {x: host(c[x]) for x in ("k", "v")}
    hit = np.zeros((c["n"], c["page"]), dtype=bool)
    for b in range(len(lens)):
        for t in range(cu[b], cu[b + 1]):
            place = None if start[b] < 0 else orc.page_line(c["table"][b], c["page"], c["n"], int(row[t]))
            if place is None:
                continue
            p, l = place
            hit[p, l] = True
            if bits == 16:
                within(got["k"][p, :, l], kt[t], kb[t], f"k row {row[t]} of {b}")
                assert np.array_equal(got["v"][p, :, l], v[t])
            else:
                check4(c["k"][p, :, l], c["ks"][p, :, l], kt[t], (24 * F + abs(at[t]) * 2.0 ** -51) * ks[t])
                check4(c["v"][p, :, l], c["vs"][p, :, l], v[t], 0 * v[t])
    for x in ("k", "v"):                      # nothing else was written
        rest = got[x].transpose(0, 2, 1, 3)[~hit]
        assert (rest == 255).all() if bits == 4 else np.isnan(rest).all()
        if bits == 4:
            assert np.isnan(host(c[x + "s"]).transpose(0, 2, 1, 3, 4)[~hit]).all()


def check4(codes, scales, x, err):
    """A row's codes: its least value and step are the half-precision roundings (2^-11 of the
    value, or half of 2^-24 below 2^-14) of those of x, which the kernel knows up to err, and
    each code is the nearest one up to that and the roundings of its quotient."""
    codes, scales = codes.cpu().numpy(), host(scales)
    for h in range(x.shape[0]):
        for g in range(x.shape[1] // 64):
            part, e = x[h, 64 * g:64 * g + 64], err[h, 64 * g:64 * g + 64].max()
            s, m = scales[h, g]
            lo, step = part.min(), (part.max() - part.min()) / 15
            assert abs(m - lo) <= 2.0 ** -11 * abs(lo) + 2.0 ** -25 + 1.01 * e
            assert abs(s - step) <= (2.0 ** -11 + 4 * F) * step + 2.0 ** -25 + e
            b = codes[h, 32 * g:32 * g + 32]
            code = np.stack([b & 15, b >> 4], axis=-1).reshape(-1)
            if s == 0:
                assert not code.any()
                continue
            ideal = (part - m) / s
            off = np.abs(code - np.clip(ideal, 0, 15))
            assert (off <= 0.5 + (e + 4 * F * np.abs(part - m)) / s + 1e-9).all(), off.max()


@pytest.mark.parametrize("io,bits", [("bf16", 16), ("f32", 16), ("bf16", 4), ("f32", 4)])
@pytest.mark.parametrize("D,R,inter,which,Hq,Hkv", [(64, 64, False, "qk", 4, 2), (128, 64, True, "k", 5, 1),
                                                    (128, 128, False, "", 3, 3), (256, 256, False, "qk", 8, 2),
                                                    (64, 0, False, "", 2, 1), (256, 32, True, "q", 1, 1)])
@pytest.mark.parametrize("page,lens,start", [(16, [5, 0, 17, 1], [14, 3, 0, 31]), (64, [70], [60]),
                                             (32, [1, 1, 1], [0, 63, 95])])
def test_append(io, bits, D, R, inter, which, Hq, Hkv, page, lens, start):
    T = sum(lens)
    gen = torch.Generator().manual_seed(D + page + Hq)
    q, k, v = fused(gen, (T,), [(Hq, D), (Hkv, D), (Hkv, D)], io, (1.0, 2.0, 0.5))
    f, (qw, kw) = freqs(R), weights(page, D, which)
    c = empty_cache(1, io, bits, len(lens), -(-160 // page), page, Hkv, D)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = torch.tensor(start, dtype=torch.int32, device="cuda")
    ko = torch.empty(T, Hkv, D, dtype=DT[io], device="cuda")
    qo = ssd.ssd_attn_paged_append(q[0], k[0], v[0], c["k"], c["v"], dev(c["table"]), n,
                                   cu_seqlens=None if lens == [1, 1, 1] else cu, k_scales=c["ks"], v_scales=c["vs"],
                                   inv_freq=dev(f), q_weight=dev(qw), k_weight=dev(kw), interleaved=inter, k_out=ko)
    check_append(io, bits, c, lens, start, q[1], k[1], v[1], qw, kw, f, inter, qo, ko=ko)
    assert n.tolist() == start


@pytest.mark.parametrize("bits", [16, 4])
def test_append_where_there_is_no_page(bits):
    """Unused slots, tables that end, entries that are no page: nothing is written for those
    tokens, and q_out is as for any row."""
    io, D, page = "bf16", 64, 16
    lens, start = [3, 20, 2, 8, 4], [-1, 40, 48, 12, -3]
    gen = torch.Generator().manual_seed(9)
    T = sum(lens)
    q, k, v = (randn(gen, T, h, D, io=io) for h in (2, 1, 1))
    c = empty_cache(2, io, bits, 5, 3, page, 1, D)
    c["table"][1, 2] = c["n"]                 # just past the pages
    c["table"][3] = [-1, 2 ** 31 - 1, 0]
    c["table"][c["table"] == 0] = c["n"] + 7
    f = freqs(64)
    qo = ssd.ssd_attn_paged_append(q[0], k[0], v[0], c["k"], c["v"], dev(c["table"]),
                                   torch.tensor(start, dtype=torch.int32, device="cuda"),
                                   cu_seqlens=np.concatenate([[0], np.cumsum(lens)]), k_scales=c["ks"],
                                   v_scales=c["vs"], inv_freq=dev(f))
    check_append(io, bits, c, lens, start, q[1], k[1], v[1], None, None, f, False, qo)


@pytest.mark.parametrize("bits", [16, 4])
def test_append_to_many_sequences(bits):
    """More sequences than one launch takes, some without tokens; positions of their own."""
    io, D, page, B = "bf16", 64, 16, 250
    rng = np.random.default_rng(3)
    lens, start = rng.integers(0, 4, B), rng.integers(0, 30, B)
    T = int(lens.sum())
    gen = torch.Generator().manual_seed(4)
    q, k, v = (randn(gen, T, h, D, io=io) for h in (1, 1, 1))
    pos = rng.integers(0, 5000, T).astype(np.int32)
    c, f = empty_cache(5, io, bits, B, 3, page, 1, D), freqs(32)
    qo = ssd.ssd_attn_paged_append(q[0], k[0], v[0], c["k"], c["v"], dev(c["table"]), dev(start.astype(np.int32)),
                                   cu_seqlens=np.concatenate([[0], np.cumsum(lens)]), k_scales=c["ks"],
                                   v_scales=c["vs"], inv_freq=dev(f), positions=dev(pos))
    check_append(io, bits, c, lens, start, q[1], k[1], v[1], None, None, f, False, qo, pos=pos)


def test_append_without_queries_and_in_place():
    io, D, page = "bf16", 128, 32
    gen = torch.Generator().manual_seed(6)
    (q, qv), (k, kv), (v, vv) = fused(gen, (40,), [(4, D), (2, D), (2, D)], io, (1.0, 1.0, 1.0))
    f, n = freqs(D), torch.zeros(1, dtype=torch.int32, device="cuda")
    c = empty_cache(7, io, 16, 1, 2, page, 2, D)
    got = ssd.ssd_attn_paged_append(None, k, v, c["k"], c["v"], dev(c["table"]), n, cu_seqlens=[0, 40], inv_freq=dev(f))
    assert got is None
    first = c["k"].clone()
    qo = ssd.ssd_attn_paged_append(q, k, v, c["k"], c["v"], dev(c["table"]), n, cu_seqlens=[0, 40], inv_freq=dev(f),
                                   q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr() and torch.equal(first.nan_to_num(7), c["k"].nan_to_num(7))
    check_append(io, 16, c, [40], [0], qv, kv, vv, None, None, f, False, q, ko=k)
    assert np.array_equal(host(v), vv)


@pytest.mark.parametrize("dt,it", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
def test_values_are_copied_bit_by_bit(dt, it):
    """Any bits of v reach the pages as they are: subnormal numbers, signed zeros, infinities, NaN."""
    gen = torch.Generator().manual_seed(10)
    bits = torch.randint(torch.iinfo(it).min, torch.iinfo(it).max, (30, 2, 64), generator=gen, dtype=torch.int64).to(it)
    bits[0, 0, :8] = torch.tensor([0, -(1 << (15 if it is torch.int16 else 31)), 1, 2, 3, 4, 5, 6]).to(it)
    v = bits.cuda().view(dt)
    k = torch.zeros_like(v)
    c = empty_cache(11, "bf16" if dt is torch.bfloat16 else "f32", 16, 1, 2, 16, 2, 64)
    ssd.ssd_attn_paged_append(None, k, v, c["k"], c["v"], dev(c["table"]), torch.zeros(1, dtype=torch.int32, device="cuda"),
                              cu_seqlens=[0, 30])
    _, back = ssd.ssd_attn_paged_gather(c["k"], c["v"], dev(c["table"]), [0, 30])
    assert torch.equal(back.view(it).cpu(), bits)


def test_four_bit_rows_of_special_values():
    """Constant rows, values past half precision's range, tiny values, one outlier."""
    D, page = 64, 16
    x = np.zeros((6, 1, D), dtype=np.float32)
    x[0], x[1, 0, ::2], x[2, 0, :2] = 2.5, 3e38, (-1e5, 1e5)
    x[3] = np.linspace(0, 1e-9, D)
    x[4, 0, 5], x[5] = 1000.0, np.arange(D) % 16 * 0.5 - 3
    x[1, 0, 1::2] = -3e38
    c = empty_cache(8, "f32", 4, 1, 1, page, 1, D)
    t = torch.from_numpy(x).cuda()
    ssd.ssd_attn_paged_append(None, t, t, c["k"], c["v"], dev(c["table"]), torch.zeros(1, dtype=torch.int32, device="cuda"),
                              cu_seqlens=[0, 6], k_scales=c["ks"], v_scales=c["vs"])
    p = int(c["table"][0, 0])
    for name in ("k", "v"):
        for r in range(6):
            codes, s = c[name][p, 0, r].cpu().numpy(), c[name + "s"][p, 0, r].cpu().numpy()
            wc, ws = orc.store4(x[r, 0].astype(np.float64))
            if r == 3:
                continue
            assert np.array_equal(s.view(np.int16), ws.view(np.int16)) and np.array_equal(codes, wc), (name, r)
    k, v = ssd.ssd_attn_paged_gather(c["k"], c["v"], dev(c["table"]), [0, 6], k_scales=c["ks"], v_scales=c["vs"],
                                     dtype=torch.float32)
    assert torch.isfinite(k).all() and torch.equal(k, v)
    assert torch.equal(k[0], t[0]) and torch.equal(k[5], t[5]) and (k[3] - t[3]).abs().max() <= 2.0 ** -24


def test_four_bit_codes_beside_ties():
    """Values in the middle between two codes go to the even one, and four fp32 steps beside it
    (further than a rounded quotient is off) to the nearer; steps of every size, tiny ones too."""
    D, rows = 64, 200
    rng = np.random.default_rng(3)
    s = (2.0 ** rng.uniform(-24, 11.9, rows)).astype(np.float16)
    s[:4] = 2.0 ** -24, 3 * 2.0 ** -24, 2.0 ** -14, 4096
    tie = (np.arange(15, dtype=np.float64) + 0.5) * s.astype(np.float64)[:, None]
    tie = tie.astype(np.float32)                                      # (exact: 11 + 5 bits)
    step = 4 * np.spacing(tie)
    x = np.zeros((rows, 1, D), dtype=np.float32)
    x[:, 0, 1], x[:, 0, 2:17], x[:, 0, 20:35], x[:, 0, 40:55] = 15 * s.astype(np.float32), tie, tie - step, tie + step
    c = empty_cache(8, "f32", 4, 1, 16, 16, 1, D)
    t = torch.from_numpy(x).cuda()
    ssd.ssd_attn_paged_append(None, t, t, c["k"], c["v"], dev(c["table"]), torch.zeros(1, dtype=torch.int32, device="cuda"),
                              cu_seqlens=[0, rows], k_scales=c["ks"], v_scales=c["vs"])
    for r in range(rows):
        page, line = int(c["table"][0, r // 16]), r % 16
        wc, ws = orc.store4(x[r, 0].astype(np.float64))
        for name in ("k", "v"):
            codes, sc = c[name][page, 0, line].cpu().numpy(), c[name + "s"][page, 0, line].cpu().numpy()
            assert np.array_equal(sc.view(np.int16), ws.view(np.int16)) and np.array_equal(codes, wc), (name, r, s[r])


# --------------------------------------------------------------------------
# Reading back
# --------------------------------------------------------------------------
@pytest.mark.parametrize("io,bits", [("bf16", 16), ("f32", 16), ("bf16", 4), ("f32", 4)])
@pytest.mark.parametrize("D,Hkv,page", [(64, 3, 16), (128, 1, 64), (256, 2, 32)])
def test_gather(io, bits, D, Hkv, page):
    rows = [70, 0, 1, 33, 130]
    c = Cache(D + page, io, bits, rows, Hkv, D, page)
    for starts, lens in ((None, rows), ([3, 0, 0, 16, 129], [60, 0, 1, 17, 1]), ([69, 0, 0, 0, 0], [1, 0, 0, 5, 130])):
        cu = np.concatenate([[0], np.cumsum(lens)])
        pos, kw = c.args()
        k, v = ssd.ssd_attn_paged_gather(*pos, cu, starts=starts, dtype=DT[io], **kw)
        for got, x in ((k, "k"), (v, "v")):
            want = np.concatenate([orc.rows_of(c.val[x], c.table[b], 0 if starts is None else starts[b], n)[0]
                                   for b, n in enumerate(lens)])
            if bits == 16:
                assert np.array_equal(host(got), want)
            else:
                within(got, want, (U[io] * 1.01 + F) * np.abs(want), x)


@pytest.mark.parametrize("bits", [16, 4])
def test_gather_of_no_pages_and_of_many_sequences(bits):
    rows = [20] * 300
    c = Cache(3, "bf16", bits, rows, 1, 64, 16)
    c.table[5, 1], c.table[299] = -7, 2 ** 31 - 1
    c.table[17, 0] = c.n
    lens = [i % 4 * 6 for i in range(300)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    pos, kw = c.args()
    k, v = ssd.ssd_attn_paged_gather(pos[0], pos[1], dev(c.table), cu, **kw)
    for got, x in ((k, "k"), (v, "v")):
        want = np.concatenate([orc.rows_of(c.val[x], c.table[b], 0, n)[0] for b, n in enumerate(lens)])
        within(got, want, U["bf16"] * 1.01 * np.abs(want), x)
    k, v = ssd.ssd_attn_paged_gather(pos[0], pos[1], dev(c.table), [0] * 301, **kw)
    assert k.shape == v.shape == (0, 1, 64)


# --------------------------------------------------------------------------
# More work than one pass of the largest launch, arrays past 2^31 elements
# --------------------------------------------------------------------------
def test_norm_rope_of_millions_of_tokens():
    T = 4_200_000
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, 1, 64, generator=gen, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(T, 1, 64, generator=gen, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    f = dev(freqs(8))
    qo, ko = ssd.ssd_attn_qk_norm_rope(q, k, pos, f)
    a = pos.double()[:, None] * f.double()
    c, s = torch.cos(a), torch.sin(a)
    for x, y in ((q, qo), (k, ko)):
        assert torch.equal(x[:, 0, 8:], y[:, 0, 8:])
        u, v = x[:, 0, :4].double(), x[:, 0, 4:8].double()
        for want, got in ((u * c - v * s, y[:, 0, :4]), (v * c + u * s, y[:, 0, 4:8])):
            # (24 F of the two values and one rounding, as turn_bound)
            tol = (24 * F + pos.double()[:, None] * 2.0 ** -51) * (u.abs() + v.abs()) * 1.01 + U["bf16"] * want.abs() + 1e-30
            assert ((got.double() - want).abs() <= tol).all()


def test_gather_past_2_to_31_elements():
    rows, Hkv, D, page = 540_000, 64, 64, 1024
    n = -(-rows // page)
    gen = torch.Generator(device="cuda").manual_seed(2)
    kp = torch.randint(0, 1 << 15, (n, Hkv, page, D), generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    vp = kp.flip(0).contiguous()
    table = torch.randperm(n, generator=gen, device="cuda").int()[None]
    k, v = ssd.ssd_attn_paged_gather(kp, vp, table, [0, rows])
    assert k.numel() > 2 ** 31
    for got, p in ((k, kp), (v, vp)):
        for i in range(0, n, 16):
            want = p[table[0, i:i + 16].long()].transpose(1, 2).reshape(-1, Hkv, D)
            at = slice(i * page, min(rows, (i + 16) * page))
            assert torch.equal(got[at].view(torch.int16), want[:at.stop - at.start].view(torch.int16))
