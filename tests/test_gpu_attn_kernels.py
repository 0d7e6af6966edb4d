"""Softmax attention: the prefill kernel of large row blocks at scales and scores where
it can go wrong, and the same sequence through every path."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import U, attn_bound, within
from oracle import attention as att
from test_gpu_attn import check, prompt, step_inputs

pytestmark = pytest.mark.gpu

# Work-groups of 32 rows (of a key head) far above any limit up to which the kernel
# for few rows is chosen: what follows runs the one of large row blocks.
MANY = 4096


# the limit, in work-groups of 32 rows
FEW = {("bf16", 64): 512, ("bf16", 128): 512, ("bf16", 256): 512, ("f32", 64): 1024, ("f32", 128): 768,
       ("f32", 256): 512}


def heads_for(L):
    return -(-MANY // (-(-L // 32)))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1e-40, -0.3, 2.0])
def test_scales_many_rows(io, scale):
    L, h = 70, heads_for(70)
    q, k, v = prompt(3, io, L, L, h, h, 64)
    o = ssd.ssd_attn_prefill(q[0], k[0], v[0], [0, L], scale=scale)
    for j in (0, 1, h // 2, h - 1):
        s = slice(j, j + 1)
        check(io, o[:, s], q[1][:, s], k[1][:, s], v[1][:, s], scale, f"scale {scale}, head {j}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_below_zero_many_rows(io, d):
    """Every score of a row near -1e33 and below: the first key's by far the highest."""
    L, h = 512, heads_for(512)
    q, k, v = prompt(8, io, L, L, h, h, d)
    qq, kk = torch.full_like(q[0], 2.0 ** 53), torch.full_like(k[0], -2.0 ** 53)
    kk *= (1 + torch.arange(L, device="cuda") / 64)[:, None, None].to(kk.dtype)
    o = ssd.ssd_attn_prefill(qq, kk, v[0], [0, L])
    assert torch.equal(o, v[0][:1].expand(L, -1, -1))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scores_far_above_zero_many_rows(io):
    """Scores that grow far past 2^24 with each key: each query takes its own value."""
    L, h = 300, heads_for(300)
    q, k, v = prompt(9, io, L, L, h, h, 64)
    qq = torch.full_like(q[0], 2.0 ** 20)
    kk = torch.full_like(k[0], 2.0 ** 20) * (2.0 ** (torch.arange(L, device="cuda") // 8 - 18))[:, None, None].to(q[0].dtype)
    kk = kk * (1 + torch.arange(L, device="cuda") % 8 / 8)[:, None, None].to(kk.dtype)     # (exact, and growing)
    o = ssd.ssd_attn_prefill(qq, kk, v[0], [0, L])
    assert torch.equal(o, v[0])


@pytest.mark.parametrize("io,d", list(FEW))
def test_on_both_sides_of_the_limit(io, d):
    """One work-group of 32 rows more or less: the other kernel, the same answers."""
    for h in (FEW[io, d] // 2, FEW[io, d] // 2 + 1):       # two row blocks a head
        q, k, v = prompt(d + h, io, 45, 78, h, h, d)
        o = ssd.ssd_attn_prefill(q[0], k[0], v[0], [0, 45], kv_starts=[3], kv_lens=[75])
        for j in (0, h // 3, h - 1):
            s = slice(j, j + 1)
            check(io, o[:, s], q[1][:, s], k[1][3:, s], v[1][3:, s], d ** -0.5, f"{h} heads, head {j}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scores_of_minus_infinity(io):
    """Products that overflow to -infinity weigh nothing: beside other keys as if they
    were masked, and where a query has no others its output is 0, in the prefill
    kernels and in the step, whatever the cache's capacity."""
    L, d, hq, hkv = 90, 64, 4, 2
    q, k, v = prompt(11, io, L, L, hq, hkv, d)
    qq, kk = torch.full_like(q[0], 1e20), torch.full_like(k[0], -1e20)
    zero = torch.zeros_like(q[0])
    assert torch.equal(ssd.ssd_attn_prefill(qq, kk, v[0], [0, L]), zero)
    h = heads_for(L)
    wide = lambda x: x[:, :1].expand(-1, h, -1).contiguous()
    assert not ssd.ssd_attn_prefill(wide(qq), wide(kk), wide(v[0]), [0, L]).any()
    for M in (L, 128, 129, 1000, 5000):
        kc = torch.zeros(1, M, hkv, d, dtype=q[0].dtype, device="cuda")
        vc = torch.zeros_like(kc)
        kc[0, :L - 1], vc[0, :L - 1] = kk[:-1], v[0][:-1]
        at = torch.tensor([L - 1], dtype=torch.int32, device="cuda")
        o = ssd.ssd_attn_decode_step(qq[-1:], kk[-1:], v[0][-1:], kc, vc, at)
        assert torch.equal(o, zero[:1]), f"capacity {M}"
        kc[0, 40] = 0                                      # one key with scores of 0
        o = ssd.ssd_attn_decode_step(qq[-1:], kk[-1:], v[0][-1:], kc, vc, at)
        want = v[0][40].repeat_interleave(hq // hkv, dim=0)
        assert torch.equal(o[0], want), f"capacity {M}"


@pytest.mark.parametrize("scale", [3.4e38, -3.4e38])
def test_largest_scales(scale):
    """Scores of 0 are 0 at every finite scale: equal weights."""
    L, hq, hkv, d = 40, 4, 2, 64
    q, k, v = prompt(12, "f32", L, L, hq, hkv, d)
    zero = torch.zeros_like(k[0])
    n = torch.arange(1, L + 1, device="cuda")[:, None, None]
    want, size = (x.cumsum(0).repeat_interleave(2, dim=1) / n for x in (v[0].double(), v[0].double().abs()))
    o = ssd.ssd_attn_prefill(q[0], zero, v[0], [0, L], scale=scale)
    # L terms of weight 1 and their sum in fp32, a division, a product
    assert ((o - want).abs() <= (L + 4) * 2.0 ** -24 * size).all()
    kc, vc = zero[None].clone(), v[0][None].clone()
    at = torch.tensor([L - 1], dtype=torch.int32, device="cuda")
    o = ssd.ssd_attn_decode_step(q[0][-1:], zero[-1:], v[0][-1:], kc, vc, at, scale=scale)
    assert ((o[0] - want[-1]).abs() <= (L + 4) * 2.0 ** -24 * size[-1]).all()


def test_heads_of_no_width_are_refused():
    x = torch.empty(4, 2, 0, dtype=torch.bfloat16, device="cuda")
    c = torch.empty(4, 8, 2, 0, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ssd.ssd_attn_prefill(x, x, x, [0, 4]),
                 lambda: ssd.ssd_attn_decode_step(x, x, x, c, c, torch.zeros(4, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ssd.SsdError) as e:
            call()
        assert e.value.code == 3


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (4, 4, 256), (40, 1, 128)])
@pytest.mark.parametrize("M", [100, 2000])
def test_step_rounds_once(hq, hkv, d, M):
    """The bf16 step's only rounding to 8 bits is the output's: its probabilities enter
    as two bf16 numbers, off by up to 2^-17 of each."""
    q, k, v, kc, vc = step_inputs(M + d, "bf16", 3, M, hq, hkv, d)
    lengths = [M - 1, M // 3, 0]
    o = ssd.ssd_attn_decode_step(q[0], k[0], v[0], kc[0], vc[0],
                                 torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lengths):
        kk, vv = (np.concatenate([c[1][b, :n], x[1][b:b + 1]]) for c, x in ((kc, k), (vc, v)))
        ro, ao, big = att.attn(q[1][b:b + 1], kk, vv, d ** -0.5)
        bound = attn_bound("f32", ro, ao, big, n + 1, d) + U["bf16"] * np.abs(ro) * 1.01 + 1.01 * 2.0 ** -17 * ao
        within(o[b:b + 1], ro, bound, f"{n} rows")
