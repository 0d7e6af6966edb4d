"""Shared by the GPU tests of the paged key/value cache: caches whose every unread line
is NaN, and error bounds.

F = 2^-24 is the largest relative error of one fp32 rounding, U that of one to the input
type.  Norm and rotation, of an element that is a sum of products of sizes `size`: the sum
of squares is off by 16 F (8 products and 5 additions, rounded), its root by half of that,
the reciprocal root and the two products by 5 F, cosine and sine by 6 F (2 of their own,
the reduced angle's rounding times pi), the rotation's products and sum by 3 F: 22 F with
the norm, 24 F taken; angles of position t are off by t 2^-51 in fp64 (kernel and oracle).
"""
import numpy as np
import torch

from attention_cases import DT, F, U, attn_bound, host
from oracle import paged as orc

NAN = float("nan")


def turn_bound(io, out, size, positions):
    far = np.abs(np.asarray(positions, dtype=np.float64)).reshape(-1, 1, 1) * 2.0 ** -51
    return (24 * F + far) * size * (1 + U[io]) + U[io] * np.abs(out) + 1e-30


class Cache:
    """A paged cache whose sequences have `rows` rows in randomly placed pages; all other
    lines are NaN (4 bits: random codes with NaN scales) and all other table entries -1."""

    def __init__(self, seed, io, bits, rows, Hkv, D, page, width=None, spare=3, first_page=0, num_pages=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in rows]
        self.width = max(max(need, default=1), 1) if width is None else width
        n = first_page + sum(need) + spare if num_pages is None else num_pages
        ids = first_page + rng.permutation(n - first_page)
        self.table = np.full((len(rows), self.width), -1, dtype=np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        self.rows, self.io, self.bits, self.page, self.D, self.Hkv, self.n = rows, io, bits, page, D, Hkv, n
        gen = torch.Generator().manual_seed(seed)
        self.dev = {"block_table": torch.from_numpy(self.table).cuda()}
        self.val, self.size = {}, {}
        for x in ("k", "v"):
            shape = (n, Hkv, page, D)
            if bits == 4:
                codes = torch.randint(0, 256, (n, Hkv, page, D // 2), generator=gen, dtype=torch.int32).to(torch.uint8)
                step = 0.05 + 0.4 * torch.rand(n, Hkv, page, D // 64, generator=gen)
                sc = torch.stack([step, -7.5 * step + 0.2 * torch.randn(step.shape, generator=gen)], dim=-1).half()
                sc[~np.broadcast_to(self.live(), shape[:3])] = NAN
                self.dev[x + "_pages"], self.dev[x + "_scales"] = codes.cuda(), sc.cuda()
                self.val[x] = orc.load4(codes.numpy(), sc.numpy())
                # 16 + code and the least value: what the kernel's terms are made of
                s = np.abs(np.repeat(sc.double().numpy(), 64, axis=-2))
                self.size[x] = 31 * s[..., 0] + s[..., 1]
            else:
                t = torch.randn(shape, generator=gen).to(DT[io])
                t[~np.broadcast_to(self.live(), shape[:3])] = NAN
                self.dev[x + "_pages"] = t.cuda()
                self.val[x] = t.double().numpy()
                self.size[x] = np.abs(self.val[x])

    def live(self):
        """[n, 1, page]: the lines that hold rows."""
        out = np.zeros((self.n, 1, self.page), dtype=bool)
        for b, n in enumerate(self.rows):
            for r in range(n):
                at = orc.page_line(self.table[b], self.page, self.n, r)
                if at is not None:
                    out[at[0], 0, at[1]] = True
        return out

    def args(self):
        """The cache's arguments of ssd_attn_paged_decode_step and _gather."""
        pos = (self.dev["k_pages"], self.dev["v_pages"], self.dev["block_table"])
        kw = {x: self.dev[x] for x in ("k_scales", "v_scales") if x in self.dev}
        return pos, kw


def check_decode(cache, o, q, lengths, scale, what="", table=None):
    """o [B, Hq, D] of a step against the oracle.  Scores: a sum of D products of the terms'
    sizes; probabilities enter the second product as bf16 terms, off by 2^-16 in bf16 and 2^-24
    in fp32 (4 bits: times steps, in fp32), so that every term there is off by that and by the
    sums' roundings; the output is rounded once."""
    io, D = cache.io, cache.D
    o = host(o)
    table = cache.table if table is None else table
    assert np.isfinite(o).all(), f"{what}: non-finite values"
    for b, n in enumerate(lengths):
        want, _, _ = orc.decode(q[b], cache.val["k"], cache.val["v"], table[b], n, scale)
        if not want.any():
            assert not o[b].any(), (what, b)
            continue
        size, _ = orc.rows_of(cache.size["v"], table[b], 0, n + 1)
        ks, _ = orc.rows_of(cache.size["k"], table[b], 0, n + 1)
        grp = q.shape[1] // cache.Hkv
        p = weights(q[b], cache, table[b], n, scale)
        ao = np.stack([p[h] @ size[:, h // grp] for h in range(q.shape[1])])
        big = np.stack([abs(scale) * (ks[:, h // grp] @ np.abs(q[b, h])).max(keepdims=True) for h in range(q.shape[1])])
        bound = attn_bound("f32", want, ao, big, n + 1 + 16, D + 16) + (2.0 ** -16 if io == "bf16" else 4 * F) * 1.01 * ao
        bound = bound + U[io] * np.abs(want) * 1.01
        bad = np.abs(o[b] - want) > bound
        assert not bad.any(), (what, b, n, int(bad.sum()), float(np.abs(o[b] - want)[bad].max()), float(bound[bad].min()))


def weights(q, cache, table, n, scale):
    """Probabilities [Hq, n + 1], 0 for rows on no page."""
    k, there = orc.rows_of(cache.val["k"], table, 0, n + 1)
    grp = q.shape[0] // cache.Hkv
    p = np.zeros((q.shape[0], n + 1))
    for h in range(q.shape[0]):
        a = scale * (k[there, h // grp] @ q[h])
        e = np.exp(a - a.max())
        p[h, there] = e / e.sum()
    return p
