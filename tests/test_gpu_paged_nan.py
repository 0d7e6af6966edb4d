"""NaN and infinities on their way into 4-bit pages: a group of 64 values with a NaN among them,
or of infinities of one sign alone, comes back as NaN, as its formula has it (the step is NaN),
and nothing else does."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import DT

pytestmark = pytest.mark.gpu

PAGE, ROWS, HKV = 16, 40, 2


def append(k, v, **kw):
    """k, v [ROWS, HKV, D] in 4-bit pages, read back in fp32: (codes and scales, k, v)."""
    D = k.shape[-1]
    n = -(-ROWS // PAGE)
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    c = {}
    for x in ("k", "v"):
        c[x + "_pages"] = torch.full((n, HKV, PAGE, D // 2), 255, dtype=torch.uint8, device="cuda")
        c[x + "_scales"] = torch.zeros(n, HKV, PAGE, D // 64, 2, dtype=torch.half, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.ssd_attn_paged_append(None, k, v, c["k_pages"], c["v_pages"], table, zero, cu_seqlens=[0, ROWS],
                              k_scales=c["k_scales"], v_scales=c["v_scales"], **kw)
    back = ssd.ssd_attn_paged_gather(c["k_pages"], c["v_pages"], table, [0, ROWS], k_scales=c["k_scales"],
                                     v_scales=c["v_scales"], dtype=torch.float32)
    return c, table, back[0], back[1]


def inputs(io, D, seed=1):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(ROWS, HKV, D, generator=gen).to(DT[io]).cuda() for _ in "kv"]


def groups(x):
    return x.unflatten(-1, (-1, 64))


# (row, head, group, which of its values, what they are): one NaN at every place in the work of
# a lane and of a group, all NaN, NaN with a sign, NaN beside infinities and huge values
SPECIAL = [(0, 0, 0, [0], "nan"), (3, 1, 0, [63], "nan"), (7, 0, 0, [13], "-nan"), (15, 1, 0, list(range(64)), "nan"),
           (16, 0, 0, list(range(0, 64, 2)), "nan"), (21, 1, 0, [5, 6], "nan inf"), (30, 0, 0, [40, 9], "nan -inf")]


def put(x, D, special):
    """x with the values put in, and [ROWS, HKV, D / 64]: which groups hold one."""
    x, hit = x.clone(), torch.zeros(ROWS, HKV, D // 64, dtype=torch.bool, device=x.device)
    for r, h, g, at, what in special:
        g = (r + g) % (D // 64)
        values = [float(s.replace("-nan", "nan")) for s in what.split()]
        for i, e in enumerate(at):
            value = torch.tensor(values[i % len(values)])
            x[r, h, 64 * g + e] = torch.copysign(value, torch.tensor(-1.0 if "-" in what.split()[i % len(values)] else 1.0))
        hit[r, h, g] = True
    return x, hit


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_takes_its_group(io, D):
    k, v = inputs(io, D)
    kn, hit = put(k, D, SPECIAL)
    vn, vhit = put(v, D, [(r + 1, 1 - h, g, at, what) for r, h, g, at, what in SPECIAL])
    clean, _, k0, v0 = append(k, v)
    c, table, k1, v1 = append(kn, vn)
    for before, after, h in ((k0, k1, hit), (v0, v1, vhit)):
        assert torch.equal(groups(after).isnan().all(dim=-1), h)
        assert torch.equal(groups(after)[~h], groups(before)[~h])
    # the scales of those groups are NaN, both, and their codes 0; all others are as without them
    for x, h in (("k", hit), ("v", vhit)):
        row = torch.arange(ROWS, device="cuda")
        page, line = table[0, row // PAGE].long(), row % PAGE
        s, s0 = (y[x + "_scales"][page, :, line] for y in (c, clean))
        b, b0 = (groups(y[x + "_pages"][page, :, line].repeat_interleave(2, dim=-1))[..., ::2] for y in (c, clean))
        assert s[h].isnan().all() and not b[h].any()
        assert torch.equal(s[~h], s0[~h]) and torch.equal(b[~h], b0[~h])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_key_that_its_norm_makes_nan(io, D, what):
    """A NaN or an infinity in a key is NaN in the whole normed key or where it stood."""
    k, v = inputs(io, D, 2)
    k[5, 1, 7] = float(what)
    kw = dict(inv_freq=torch.full((D // 2,), 0.01, device="cuda"), k_weight=torch.ones(D, device="cuda"))
    c, table, k1, v1 = append(k, v, **kw)
    ko = torch.empty_like(k)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.ssd_attn_paged_append(None, k, v, c["k_pages"], c["v_pages"], table, zero, cu_seqlens=[0, ROWS], k_out=ko,
                              k_scales=c["k_scales"], v_scales=c["v_scales"], **kw)
    want = groups(ko).isnan().any(dim=-1)
    assert want[5, 1].any() and want.sum() == want[5, 1].sum() and (what == "inf" or want[5, 1].all())
    assert torch.equal(groups(k1).isnan().any(dim=-1), want) and torch.equal(groups(k1).isnan().all(dim=-1), want)
    assert torch.isfinite(v1).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_over_a_nan(io):
    """A NaN in a key reaches the outputs of its sequence and key head, one in a value those of its
    group; the other heads' outputs stay as they were."""
    D = 128
    k, v = inputs(io, D, 3)
    q = torch.randn(1, 2 * HKV, D, generator=torch.Generator().manual_seed(4)).to(DT[io]).cuda()
    at = torch.full((1,), ROWS - 1, dtype=torch.int32, device="cuda")

    def step(k, v):
        c, table, _, _ = append(k, v)
        return ssd.ssd_attn_paged_decode_step(q, c["k_pages"], c["v_pages"], table, at, k_scales=c["k_scales"],
                                              v_scales=c["v_scales"])

    o = step(k, v)
    kn, vn = k.clone(), v.clone()
    kn[11, 0, 3], vn[17, 1, 70] = float("nan"), float("nan")
    a, b = step(kn, v), step(k, vn)
    assert a[:, :2].isnan().all() and torch.equal(a[:, 2:], o[:, 2:])
    assert torch.equal(b[:, :2], o[:, :2]) and torch.equal(b[:, 2:, :64], o[:, 2:, :64]) and b[:, 2:, 64:].isnan().all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_infinities(io):
    """Infinities beside finite values are held within the scales' range; of one sign alone in a
    group they have no step."""
    D, inf = 64, float("inf")
    k, v = inputs(io, D, 5)
    v[0], v[1], v[2, :, 5], v[3, :, 6] = inf, -inf, inf, -inf
    v[4, :, :32], v[4, :, 32:] = inf, -inf
    c, table, k1, v1 = append(k, v)
    assert v1[:2].isnan().all() and torch.isfinite(v1[2:]).all() and torch.isfinite(k1).all()
    m = v[2].float().masked_fill(v[2].isinf(), 0).amin(dim=-1, keepdim=True).half().float()
    assert torch.equal(v1[2], torch.where(v[2].isinf(), 15 * 65504.0 + m, m).float())
    assert torch.equal(v1[3], torch.where(v[3].isinf(), -65504.0, 0.0))
    assert torch.equal(v1[4], torch.where(v[4] > 0, 14 * 65504.0, -65504.0))
