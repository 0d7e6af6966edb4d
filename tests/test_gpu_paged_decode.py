"""One query token per sequence over paged caches in the input type and in 4 bits,
against oracle/paged.py.  Every line that no row uses is NaN."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import host, randn
from paged_cases import Cache, check_decode

pytestmark = pytest.mark.gpu

FORMATS = [("bf16", 16), ("f32", 16), ("bf16", 4), ("f32", 4)]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def step(c, q, lengths, **kw):
    pos, sc = c.args()
    return ssd.ssd_attn_paged_decode_step(q, *pos, ints(lengths), **sc, **kw)


def queries(seed, B, Hq, D, io):
    return randn(torch.Generator().manual_seed(seed), B, Hq, D, io=io)


@pytest.mark.parametrize("io,bits", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 16), (8, 2, 64), (17, 1, 32), (32, 2, 16), (40, 1, 128), (9, 3, 1024)])
def test_sizes(io, bits, D, Hq, Hkv, page):
    """Lengths around tiles, work units and pages, and unused slots."""
    lengths = [0, 14, 15, 16, 31, 32, -1, 63, 64, 127, 128, 255, 256, 300, 1 << 30]
    c = Cache(D + Hq, io, bits, [n + 1 if 0 <= n < 1000 else 0 for n in lengths], Hkv, D, page)
    q = queries(Hq, len(lengths), Hq, D, io)
    check_decode(c, step(c, q[0], lengths), q[1], lengths, D ** -0.5, f"{io} {bits} {D}")


@pytest.mark.parametrize("io,bits", FORMATS)
@pytest.mark.parametrize("D,rows,width", [(64, [9000], None), (128, [5000, 3, 2500], 5000), (256, [1, 3000], 190)])
def test_long_sequences(io, bits, D, rows, width):
    """Items cut between many work-groups; tables far wider than the sequences are long."""
    page = 16
    c = Cache(5, io, bits, rows, 2, D, page, width=width)
    lengths = [n - 1 for n in rows]
    q = queries(6, len(rows), 6, D, io)
    check_decode(c, step(c, q[0], lengths), q[1], lengths, D ** -0.5, "long")


@pytest.mark.parametrize("io,bits", [("bf16", 16), ("f32", 4)])
def test_many_sequences(io, bits):
    """More sequences than a work-group has threads, runs of unused slots among them."""
    rng = np.random.default_rng(7)
    rows = [int(n) for n in rng.integers(0, 40, 700)]
    rows[100:400] = [0] * 300
    c = Cache(8, io, bits, rows, 1, 64, 16)
    lengths = [n - 1 for n in rows]
    q = queries(9, 700, 2, 64, io)
    check_decode(c, step(c, q[0], lengths), q[1], lengths, 0.125, "many")


@pytest.mark.parametrize("io,bits", FORMATS)
def test_more_items_than_work_groups(io, bits):
    """600 items of 2 key heads, a few of them cut between work-groups."""
    rng = np.random.default_rng(23)
    rows = [int(n) for n in rng.integers(1, 30, 300)]
    rows[7], rows[8], rows[150], rows[299] = 1500, 0, 2100, 900
    c = Cache(24, io, bits, rows, 2, 64, 32)
    lengths = [n - 1 for n in rows]
    q = queries(25, 300, 6, 64, io)
    check_decode(c, step(c, q[0], lengths), q[1], lengths, 0.125, "items")


@pytest.mark.parametrize("io,bits", FORMATS)
@pytest.mark.parametrize("D", [128, 256])
def test_one_long_sequence_of_many_heads(io, bits, D):
    """Two tiles of query heads (32 and 8) of a key head, cut between work-groups."""
    c = Cache(26, io, bits, [2500, 40], 1, D, 64)
    q = queries(27, 2, 40, D, io)
    check_decode(c, step(c, q[0], [2499, 39]), q[1], [2499, 39], D ** -0.5, "heads")


@pytest.mark.parametrize("io,bits", FORMATS)
def test_entries_that_are_no_page(io, bits):
    """Rows on no page are left out, at the start, in the middle and at the end of a table; a
    sequence with no page at all gets 0.  (Page 0, which stands in for them, is NaN.)"""
    rows = [300, 300, 64, 20, 1]
    c = Cache(10, io, bits, rows, 2, 128, 32, first_page=1)
    pages = c.table.copy()
    pages[0, [0, 3]], pages[1, 9] = (-1, c.n), 2 ** 31 - 1
    pages[2, :], pages[4, 0] = -5, c.n + 1
    c.dev["block_table"] = torch.from_numpy(pages).cuda()
    lengths = [n - 1 for n in rows]
    q = queries(11, 5, 4, 128, io)
    o = step(c, q[0], lengths)
    check_decode(c, o, q[1], lengths, 128 ** -0.5, "bad pages", table=pages)
    assert not o[2].any() and not o[4].any() and o[3].any()


@pytest.mark.parametrize("io,bits", FORMATS)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 3.0])
def test_scales(io, bits, scale):
    c = Cache(12, io, bits, [200, 45], 1, 64, 16)
    q = queries(13, 2, 3, 64, io)
    check_decode(c, step(c, q[0], [199, 44], scale=scale), q[1], [199, 44], scale, "scale")


@pytest.mark.parametrize("io,bits", FORMATS)
def test_strided_queries_given_outputs_and_shared_pages(io, bits):
    """q a slice of a projection, o and the workspace given, two sequences on the same pages."""
    D, Hq = 128, 4
    c = Cache(14, io, bits, [100, 0, 100], 2, D, 16)
    c.table[1] = c.table[0]
    c.dev["block_table"] = torch.from_numpy(c.table).cuda()
    wide = queries(15, 3, 3 * Hq, D, io)
    q = wide[0][:, Hq:2 * Hq]
    o = torch.full((3, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    fmt = ssd.SSD_PAGES_4BIT if bits == 4 else ssd.SSD_PAGES_IO
    need = ssd.ssd_attn_paged_decode_workspace_size(3, Hq, 2, D, c.n, 16, c.width,
                                                    ssd.SSD_BF16 if io == "bf16" else ssd.SSD_F32, fmt)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    got = step(c, q, [99, 50, 80], o=o, workspace=ws[:need])
    assert got is o and (ws[need:] == 255).all()
    check_decode(c, o, wide[1][:, Hq:2 * Hq], [99, 50, 80], D ** -0.5, "strided")


@pytest.mark.parametrize("io,bits", FORMATS)
def test_scores_far_from_zero(io, bits):
    """Scores that grow along the sequence (the running maximum is raised again and again) and
    reach thousands: a softmax that is one row."""
    c = Cache(16, io, bits, [400], 1, 64, 16)
    q = (torch.full((1, 2, 64), 1.0)).to(torch.bfloat16 if io == "bf16" else torch.float32)
    lines = [(int(c.table[0, r // 16]), r % 16) for r in range(400)]
    for r, (p, l) in enumerate(lines):
        if bits == 4:
            c.dev["k_scales"][p, 0, l] = torch.tensor([[0.0, r / 8]])
            c.val["k"][p, 0, l] = r / 8
            c.size["k"][p, 0, l] = r / 8
        else:
            c.dev["k_pages"][p, 0, l] = float(r // 2)
            c.val["k"][p, 0, l] = c.size["k"][p, 0, l] = float(r // 2)
    check_decode(c, step(c, q.cuda(), [399], scale=1.0), q.double().numpy(), [399], 1.0, "far")


@pytest.mark.parametrize("io,bits", [("bf16", 16), ("f32", 16), ("bf16", 4)])
def test_infinite_scores_and_values(io, bits):
    """All scores -infinity: 0.  An infinity in a value row reaches its own sequence only."""
    c = Cache(17, io, bits, [40, 40, 40], 1, 64, 16)
    q = queries(18, 3, 2, 64, io)
    want = step(c, q[0], [39, 39, 39])
    if bits == 16:
        v = c.dev["v_pages"].clone()
        v[int(c.table[1, 1]), 0, 3, 5] = float("inf")
        pos, kw = c.args()
        o = ssd.ssd_attn_paged_decode_step(q[0], pos[0], v, pos[2], ints([39, 39, 39]), **kw)
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2]) and not torch.isfinite(o[1, :, 5]).any()
        big = torch.full_like(q[0], 3e38)
        k = torch.where(c.dev["k_pages"].isnan(), c.dev["k_pages"], torch.full_like(c.dev["k_pages"], -3e38))
        o = ssd.ssd_attn_paged_decode_step(big, k, pos[1], pos[2], ints([39, 39, 39]))
        assert not o.any()
    else:
        s = c.dev["v_scales"].clone()
        s[int(c.table[1, 1]), 0, 3, 0, 1] = float("inf")
        pos, kw = c.args()
        o = ssd.ssd_attn_paged_decode_step(q[0], *pos, ints([39, 39, 39]), k_scales=kw["k_scales"], v_scales=s)
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2]) and not torch.isfinite(o[1]).any()


@pytest.mark.parametrize("io,bits", FORMATS)
def test_a_sequence_in_any_batch(io, bits):
    """The same sequences alone and in a batch that cuts them elsewhere agree up to rounding,
    and the same call gives the same bits."""
    rows = [3000, 1, 700, 0, 128, 2049]
    c = Cache(19, io, bits, rows, 2, 64, 16)
    q = queries(20, 6, 4, 64, io)
    lengths = [n - 1 for n in rows]
    o = step(c, q[0], lengths)
    assert torch.equal(o, step(c, q[0], lengths))
    for b in range(6):
        alone = step(c, q[0], [n if i == b else -1 for i, n in enumerate(lengths)])
        check_decode(c, alone[b:b + 1], q[1][b:b + 1], [lengths[b]], 0.125, f"alone {b}", table=c.table[b:b + 1])


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_past_32_bits(bits):
    """Caches of more than 2^31 values (and bytes), the sequence's pages at their far end."""
    D, page, n = 256, 1024, 9000
    io, rows = "bf16", [1500]
    gen = torch.Generator().manual_seed(21)
    small = Cache(22, io, bits, rows, 1, D, page)
    dev = {}
    for x in ("k", "v"):
        for name in (x + "_pages", x + "_scales"):
            if name in small.dev:
                t = small.dev[name]
                m = n if bits == 16 else 2 * n
                dev[name] = torch.empty((m,) + t.shape[1:], dtype=t.dtype, device="cuda")
                dev[name][-t.shape[0]:] = t
    m = dev["k_pages"].shape[0]
    assert dev["k_pages"].numel() > 2 ** 31
    table = np.where(small.table >= 0, small.table + (m - small.n), -1).astype(np.int32)
    q = randn(gen, 1, 4, D, io=io)
    kw = {x: dev[x] for x in dev if "scales" in x}
    o = ssd.ssd_attn_paged_decode_step(q[0], dev["k_pages"], dev["v_pages"], torch.from_numpy(table).cuda(), ints([1499]),
                                       **kw)
    check_decode(small, o, q[1], [1499], D ** -0.5, "far pages")
    k, v = ssd.ssd_attn_paged_gather(dev["k_pages"], dev["v_pages"], torch.from_numpy(table).cuda(), [0, 1500], **kw)
    pos, skw = small.args()
    ks, vs = ssd.ssd_attn_paged_gather(*pos, [0, 1500], **skw)
    assert torch.equal(k, ks) and torch.equal(v, vs)
    new = randn(gen, 1, 1, D, io=io)
    ssd.ssd_attn_paged_append(None, new[0], new[0], dev["k_pages"], dev["v_pages"], torch.from_numpy(table).cuda(),
                              ints([1400]), **kw)
    k, v = ssd.ssd_attn_paged_gather(dev["k_pages"], dev["v_pages"], torch.from_numpy(table).cuda(), [0, 1], starts=[1400], **kw)
    if bits == 16:
        assert torch.equal(k, new[0]) and torch.equal(v, new[0])
    else:
        assert (k.float() - new[0].float()).abs().max() < 0.3 and torch.equal(k, v)
