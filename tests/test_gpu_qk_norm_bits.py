"""The norm of queries and keys in fp32, to the last bit.

The reciprocal root.  Heads of small whole numbers have a sum of squares that is exact in fp32
however it is added up, its mean is exact (D is a power of two), and with eps = 0 and weights of
1 a value 1 of the head becomes the reciprocal root of the mean z.  y, the hardware's estimate,
is off by at most one unit in its last place, 2^-23 of it.  A Newton step from it has the error
3/8 (2^-22)^2 < 2^-45 of y; the residual 1 - z y^2, of size 2^-22, is formed from exact products
with one rounding, 2^-46; and the result is rounded once: half a unit and 2^-20 of one.  (The
estimate alone exceeds half a unit for many z.)

Whole heads, bounds for what the kernel does: every square rounded, F = 2^-24, and 3 additions
to a sum of four, one to eight, log2(D / 8) to all: 5 + log2(D / 8) F of the sum, half of that of
its root; the addition of eps, F / 2; the root, F; two products, F each.  (With the rotation's
sines and cosines, off by one unit in their last place at most, 2 F, its products and its sum,
12.5 F of a pair's sizes: paged_cases.turn_bound takes 24 F, which it derives for sums in another
order and for sines and cosines from the library.)"""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import F, host

pytestmark = pytest.mark.gpu

# rotated values of a head of D, neighbours paired: none, all, and parts of a head
TURNS = [(0, False), (1, False), (0.5, False), (0.25, False), (1, True), (0.5, True)]


def turn(D, part):
    return None if part == 0 else torch.full((int(D * part) // 2,), 0.37, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("part,inter", TURNS)
def test_reciprocal_roots(D, part, inter):
    T, H = 500, 5
    rng = np.random.default_rng(D)
    x = rng.integers(-30, 31, (T, H, D)).astype(np.float32)
    x[..., 1:] *= rng.random((T, H, 1)) < 0.9                    # (some heads of one value)
    x *= rng.random((T, H, D)) < rng.random((T, H, 1))
    one = rng.integers(0, D, (T, H))
    np.put_along_axis(x, one[..., None], 1.0, axis=-1)
    t = torch.from_numpy(x).cuda()
    w = torch.ones(D, device="cuda")
    q, k = ssd.ssd_attn_qk_norm_rope(t, t, torch.zeros(T, dtype=torch.int32, device="cuda"), turn(D, part), w, w, eps=0.0,
                                     interleaved=inter)          # (position 0: cosines 1, sines 0)
    z = (x.astype(np.float64) ** 2).sum(axis=-1) / D
    want = 1 / np.sqrt(z)
    unit = np.spacing(want.astype(np.float32)).astype(np.float64)
    unit = np.where(want < want.astype(np.float32), np.spacing(np.nextafter(want.astype(np.float32), 0)), unit)
    for got in (q, k):
        y = np.take_along_axis(host(got), one[..., None], axis=-1)[..., 0]
        off = np.abs(y - want) / unit
        assert (off <= 0.5 + 2.0 ** -20).all(), (float(off.max()), int((off > 0.5).sum()))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("part,inter", TURNS)
def test_norms(D, part, inter):
    T, H, eps = 200, 5, 1e-5
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(T, H, D, generator=gen) * torch.exp(3 * torch.randn(T, H, 1, generator=gen))
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    t = x.cuda()
    q, k = ssd.ssd_attn_qk_norm_rope(t, t, torch.zeros(T, dtype=torch.int32, device="cuda"), turn(D, part), w.cuda(),
                                     w.cuda(), eps=eps, interleaved=inter)
    x = x.double().numpy()
    want = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * w.double().numpy()
    bound = ((5 + np.log2(D // 8)) / 2 + 0.5 + 1 + 2) * F * (1 + 16 * F) * np.abs(want)
    for got in (q, k):
        assert (np.abs(host(got) - want) <= bound).all()
