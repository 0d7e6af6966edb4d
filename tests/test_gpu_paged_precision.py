"""One-token attention over paged caches in bf16 is as near its formula as fp32 sums and
probabilities are, beside the output's one rounding.

F = 2^-24.  Two kinds of inputs make errors visible that the output's rounding hides elsewhere:

Two kinds of rows whose weighted values nearly cancel.  The output is small beside p |v|, and
its rounding small beside the errors of p.  One live row B with score -a (0.25 <= a <= 2.5) and
others A with score 0, so that the numerator is p v - c with p = e^-a, p |v| = c up to the
rounding of c.  Scores are exact (one query value times one key value).  p: the factor log2 e
of the exponent (|exponent| < 4) is off by F of itself, the exponent's one rounding by 2^-23,
2.8 F + 1.4 F of p; the exponential by one unit in its last place, 2 F.  In the second product
p enters as three bf16 numbers, off by 2^-27 at most, and is rounded once more with 4-bit steps
(F).  Each of the few additions of the numerator is off by F of what it adds up, at most twice
c in 4 bits (codes of 8 and more, counted from either end): three terms and the least values'
sum in two pieces, 2 (3 + 2) F.  In all 6.2 + 1 + 10 + 0.1 < 18 F of c, the sum in the denominator 4 F of the
small output.  Two terms instead of three would be off by up to 64 F.

Rows of random weights whose values come in pairs v, -v of the same weight, in random order.
The output is the roundings of the sums alone.  Adding values of size s one by one, L to a wave,
with r roundings to a tile of K rows, each F / sqrt(3) of a sum that has wandered off by
s sqrt(t): F s L sqrt(r / (6 K)) for L rows, that is F sqrt(L r / (6 K)) of the size of a random
sum of them, s sqrt(L).  r <= 15 (three terms, five roundings each at most), K >= 32, L <= 300
below: 5 F; and each weight off by up to 8 F by itself (as above; |exponent| < 6): 13 F.  32 F
taken.  (Sums that grow with the number of rows, because codes of one sign and least values of
the other are summed apart, would be off by about F L of it, 100 F and more.)"""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import F

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("grp", [1, 20])
@pytest.mark.parametrize("bits", [4, 16])
def test_probabilities_of_values_that_cancel(bits, D, grp):
    B, Hkv, page = 48, 2, 16
    rng = np.random.default_rng(D + grp + bits)
    a = rng.uniform(0.25, 2.5, (B, Hkv))
    a = torch.from_numpy(a).to(BF).double().numpy()              # (a key value: bf16 or half alike)
    p = np.exp(-a)
    where = np.stack([rng.permutation(16)[:3] for _ in range(B)])  # rows of B, A, A' among 16
    k = np.full((B, Hkv, page, D), 0.0)
    v = np.zeros((B, Hkv, page, D))
    k[..., 0] = -20000.0                                         # rows that weigh nothing
    q = torch.zeros(B, Hkv * grp, D, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    seq = np.arange(B)
    for i, s in ((0, -a), (1, 0 * a), (2, 0 * a)):
        k[seq, :, where[:, i], 0] = s
    if bits == 16:
        # v of B any bf16 number, -c as the sum of two
        vb = torch.from_numpy(rng.uniform(1, 2, (B, Hkv, D))).to(BF).double().numpy()
        c = p[..., None] * vb
        c1 = torch.from_numpy(c).to(BF).double().numpy()
        c2 = torch.from_numpy(c - c1).to(BF).double().numpy()
        v[seq, :, where[:, 0]], v[seq, :, where[:, 1]], v[seq, :, where[:, 2]] = vb, -c1, -c2
        kp, vp = (torch.from_numpy(x).to(BF).cuda() for x in (k, v))
        o = ssd.ssd_attn_paged_decode_step(q, kp, vp, table, ints([15] * B), scale=1.0)
    else:
        # keys: their first group's least value (a query of one value sees it), no steps; B: code
        # n and step s everywhere, A and A' the least values -c and 0
        G = D // 64
        half = lambda x: torch.from_numpy(np.ascontiguousarray(x)).half()
        n = rng.integers(8, 16, (B, Hkv, G))
        s = half(rng.uniform(0.25, 2.0, (B, Hkv, G)))
        c = half(p[..., None] * n * s.double().numpy())
        ks = torch.zeros(B, Hkv, page, G, 2, dtype=torch.half)
        ks[..., 0, 1] = half(k[..., 0])
        vs = torch.zeros_like(ks)
        codes = torch.zeros(B, Hkv, page, G, 32, dtype=torch.uint8)
        for b in range(B):
            rb, ra = where[b, 0], where[b, 1]
            codes[b, :, rb] = torch.from_numpy(n[b] * 17).to(torch.uint8)[..., None]
            vs[b, :, rb, :, 0], vs[b, :, ra, :, 1] = s[b], -c[b]
            v[b, :, rb] = np.repeat(n[b] * s[b].double().numpy(), 64, axis=-1)
            v[b, :, ra] = np.repeat(-c[b].double().numpy(), 64, axis=-1)
        zero = torch.zeros(B, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
        # (a key is its least value in all of its group; the query sees the first value of it)
        o = ssd.ssd_attn_paged_decode_step(q, zero, codes.flatten(-2).cuda(), table, ints([15] * B), scale=1.0,
                                           k_scales=ks.cuda(), v_scales=vs.cuda())
    w = np.exp(k[..., 0])
    want = np.einsum("bhr,bhrd->bhd", w, v) / w.sum(axis=-1)[..., None]
    size = np.repeat((p[..., None] * np.abs(v).max(axis=2)) / w.sum(axis=-1)[..., None], grp, axis=1)
    want = np.repeat(want, grp, axis=1)
    off = np.abs(o.double().cpu().numpy() - want)
    bound = 18 * F * size + (U + 16 * F) * np.abs(want)
    assert (np.abs(want) < 2.0 ** -9 * size).all()               # (they cancel)
    assert (off <= bound).all(), (float((off / bound).max()), int((off > bound).sum()))


@pytest.mark.parametrize("D,Hkv,grp,B,rows", [(64, 2, 4, 32, 8192), (128, 2, 4, 32, 8192), (256, 2, 4, 24, 8192),
                                              (64, 1, 20, 64, 8192), (128, 1, 20, 32, 8192), (128, 2, 4, 1, 1024)])
@pytest.mark.parametrize("order", ["random", "halves"])
def test_sums_of_values_that_cancel(D, Hkv, grp, B, rows, order):
    page, G = 64, D // 64
    gen = torch.Generator(device="cuda").manual_seed(D + grp)
    half = rows // 2
    codes = torch.randint(0, 256, (B, half, Hkv, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
    codes = torch.cat([codes, 255 - codes], dim=1)               # 15 - code
    s = 0.25 + torch.rand(B, half, Hkv, G, generator=gen, device="cuda")
    s = (s * 64).round() / 64                                    # seven bits: 7.5 s is a half-precision number
    scales = torch.stack([s, -7.5 * s], dim=-1).repeat(1, 2, 1, 1, 1)
    least = 0.5 * torch.randn(B, half, Hkv, generator=gen, device="cuda").clamp(-3, 3).repeat(1, 2, 1)
    keys = torch.zeros(B, rows, Hkv, G, 2, device="cuda")
    keys[..., 0, 1] = least.half().float()                       # a row's score, for a query of one value
    if order == "random":
        at = torch.randperm(rows, generator=gen, device="cuda")
        codes, scales, keys = codes[:, at], scales[:, at], keys[:, at]
    assert torch.equal(scales.half().float(), scales)
    lay = lambda x: x.reshape(B * rows // page, page, *x.shape[2:]).transpose(1, 2).contiguous()
    vp, vs, ks = lay(codes), lay(scales.half()), lay(keys.half())
    table = torch.arange(B * rows // page, dtype=torch.int32, device="cuda").view(B, -1)
    q = torch.zeros(B, Hkv * grp, D, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    o = ssd.ssd_attn_paged_decode_step(q, torch.zeros_like(vp), vp, table, ints([rows - 1] * B), scale=1.0,
                                       k_scales=ks, v_scales=vs).double()
    # the size of a sum of such values with random signs
    p = keys[..., 0, 1].double().exp()
    v2 = sum((x - 7.5) ** 2 for x in range(16)) / 16 * scales[..., 0].double().square().mean(dim=-1)
    size = float(((p * p * v2).sum(dim=1) / p.sum(dim=1) ** 2).mean().sqrt())
    assert float(o.square().mean().sqrt()) <= 32 * F * size, float(o.square().mean().sqrt()) / (F * size)
