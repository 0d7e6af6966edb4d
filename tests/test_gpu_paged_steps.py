"""Steps of 4-bit groups: half((max - min) r), r the fp32 number next to 1 / 15, bit by bit; and
how often that is not half((max - min) / 15)."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd

pytestmark = pytest.mark.gpu


def test_steps_bit_by_bit():
    T, D, page = 4000, 256, 1024
    rng = np.random.default_rng(1)
    x = rng.standard_normal((T, 2, D)).astype(np.float32) * np.exp(rng.standard_normal((T, 2, 1))).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    n = -(-T // page)
    c = {}
    for name in ("k", "v"):
        c[name + "_pages"] = torch.zeros(n, 2, page, D // 2, dtype=torch.uint8, device="cuda")
        c[name + "_scales"] = torch.zeros(n, 2, page, D // 64, 2, dtype=torch.half, device="cuda")
    ssd.ssd_attn_paged_append(None, t, t, c["k_pages"], c["v_pages"],
                              torch.arange(n, dtype=torch.int32, device="cuda")[None],
                              torch.zeros(1, dtype=torch.int32, device="cuda"), cu_seqlens=[0, T],
                              k_scales=c["k_scales"], v_scales=c["v_scales"])
    g = x.reshape(T, 2, D // 64, 64)
    span = g.max(axis=-1) - g.min(axis=-1)                       # fp32, rounded
    want = (span * (np.float32(1) / np.float32(15))).astype(np.float16)
    for name in ("k", "v"):
        s = c[name + "_scales"].transpose(1, 2).reshape(n * page, 2, D // 64, 2)[:T].cpu().numpy()
        assert np.array_equal(s[..., 0].view(np.int16), want.view(np.int16))
        assert np.array_equal(s[..., 1].view(np.int16), g.min(axis=-1).astype(np.float16).view(np.int16))
    # a product with r is off by 2^-24 for r and 2^-24 for itself, at most; a quotient lies that
    # near the middle of two half-precision numbers, 2^-11 of it apart or more, once in 2^11 at most
    off = want != (span.astype(np.float64) / 15).astype(np.float16)
    assert off.mean() < 2.0 ** -11
    assert (np.abs(want.view(np.int16).astype(int) - (span.astype(np.float64) / 15).astype(np.float16).view(np.int16)) <= 1).all()
