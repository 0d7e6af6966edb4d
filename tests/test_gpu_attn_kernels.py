"""Softmax attention: the same sequence through every path (both prefill kernels, the
step with and without chunks to join)."""
import pytest
import torch

import state_space_model_mamba_amd as ssd
from test_gpu_attn import prompt

pytestmark = pytest.mark.gpu

# Work-groups of 32 rows (of a key head) far above any limit up to which the kernel
# for few rows is chosen: what follows runs the one of large row blocks.
MANY = 4096


def heads_for(L):
    return -(-MANY // (-(-L // 32)))


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
