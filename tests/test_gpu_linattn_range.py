"""Linear attention at the ends of the number range: large and small values, states of
which little is left."""
import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import host, lin_bounds, within
from oracle import attention as att
from test_gpu_linattn import inputs

pytestmark = pytest.mark.gpu

# forgetting at every speed: from 3 powers of two in 1500 tokens to 5 in each token
DECAYS = [-0.0014, -0.03, -0.1, -0.3, -0.5, -0.8, -1.3, -3.5]


@pytest.mark.parametrize("io,dk,dv", [("bf16", 64, 64), ("bf16", 128, 128), ("bf16", 256, 64), ("f32", 64, 128),
                                      ("f32", 128, 64), ("f32", 256, 64)])
@pytest.mark.parametrize("power", [115, 70, -60])
def test_large_and_small_values(io, dk, dv, power):
    """Values (and states) scaled by a power of two: what the recurrence can hold, the
    scan can, whatever the head's decay.  (S and o stay below 2^115 64 sqrt(1500).)"""
    L, hv, f = 1500, len(DECAYS), 2.0 ** power
    q, k, v, g, S0 = inputs(dk + dv + power, io, (1, L), 2, hv, dk, dv, 1, g=DECAYS)
    vx, Sx = v[0] * f, S0[0] * f                           # (exact)
    o, fin = ssd.ssd_linattn_chunk_scan(q[0], k[0], vx, g[0], initial_state=Sx)
    ro, rS, ao, A = att.linattn(q[1][0], k[1][0], v[1][0], g[1], S0[1][0])
    bo, bS = lin_bounds(io, ro, ao, A, L, dk)
    within(host(o[0]) / f, ro, bo, "o")
    within(host(fin[0]) / f, rS, bS, "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-110, 115])
def test_large_and_small_scales(io, power):
    """Outputs near the ends of the range by their scale: no factor on the way leaves it.
    (Values of the inverse size are not tried: q . S must stay above 2^-60, since the
    products behind it carry weights down to 2^-40 and fp32 ends at 2^-126.)"""
    L, hv, dk, dv, f = 400, len(DECAYS), 64, 64, 2.0 ** power
    q, k, v, g, S0 = inputs(power + 200, io, (1, L), 2, hv, dk, dv, 1, g=DECAYS)
    o, _ = ssd.ssd_linattn_chunk_scan(q[0], k[0], v[0], g[0], initial_state=S0[0], scale=f)
    ro, _, ao, A = att.linattn(q[1][0], k[1][0], v[1][0], g[1], S0[1][0])
    bo, _ = lin_bounds(io, ro, ao, A, L, dk)
    within(host(o[0]) / f, ro, bo, "o")


def one_token_state(dev, g, n, k, v, L):
    """A state whose only term is lambda^n k v, against the formula.

    Roundings, relative, in units of 2^-22 (a power of the decay: the exponential's
    last place and its exponent's fraction in fp32, 1.5 2^-23; a product or sum
    2^-24): the token's weight and product 1, the partial sums it enters 1, the end
    factor 1, a segment's power and its sum into the next ones 3, and a rescale every
    256 tokens or after 2^-32 at most.  Beside these, in bf16, 2^-24 of the token's
    own product, however much of it is left."""
    size = np.abs(k[..., :, None] * v[..., None, :])
    want = np.exp(g * n)[..., None, None] * k[..., :, None] * v[..., None, :]
    off = np.abs(host(dev) - want) - ((7 + L / 256 + np.abs(g * n)[..., None, None] / 22) * 2.0 ** -22 * np.abs(want)
                                      + 2.0 ** -24 * size)
    assert (off <= 0).all(), f"past the bound by {(off / (size + 1e-30)).max():.2e} of the product"


@pytest.mark.parametrize("io,dk,dv", [("bf16", 64, 64), ("bf16", 128, 128), ("bf16", 128, 64), ("bf16", 256, 64),
                                      ("f32", 64, 64)])
@pytest.mark.parametrize("L,at", [(200, 20), (3000, 20), (3000, 2500)])
def test_states_of_quiet_ends(io, dk, dv, L, at):
    """One token that matters, before keys of 0 (padding) by whose end it is forgotten
    to 2^-3 to 2^-28: the end state is off by no more than fp32 roundings of it and of
    what it was."""
    gs = np.log(2.0) * -np.array([3.0, 5.2, 6.5, 9.0, 28.0]) / (L - 1 - at)
    q, k, v, g, _ = inputs(L + at + dk, io, (1, L), 1, 5, dk, dv, 1, init=False, g=gs)
    k[0][:, :at], k[0][:, at + 1:] = 0, 0
    _, fin = ssd.ssd_linattn_chunk_scan(q[0], k[0], v[0], g[0])
    one_token_state(fin[0], g[1], L - 1 - at, np.repeat(k[1][0, at], 5, axis=0), v[1][0, at], L)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128), (256, 64)])
def test_states_handed_between_segments(dk, dv):
    """As above with enough heads that segments are long: the token that matters is
    forgotten within its own segment, all of whose later keys are 0."""
    B, L, hv, at = 8, 2048, 24, 10
    gs = -np.linspace(0.003, 0.012, hv)
    q, k, v, g, _ = inputs(dk + dv, "bf16", (B, L), 8, hv, dk, dv, B, init=False, g=gs)
    k[0][:, :at], k[0][:, at + 1:] = 0, 0
    _, fin = ssd.ssd_linattn_chunk_scan(q[0], k[0], v[0], g[0])
    one_token_state(fin, g[1][None], L - 1 - at, np.repeat(k[1][:, at], 3, axis=1), v[1][:, at], L)


def test_the_same_layer_through_the_ssd_scan():
    """128 keys by 64 values in bf16 are an SSD layer with dt = 1, A = g, D = 0: the
    same recurrence through the other kernels, its state transposed."""
    B, L, hk, hv, dk, dv = 2, 700, 2, 4, 128, 64
    q, k, v, g, _ = inputs(3, "bf16", (B, L), hk, hv, dk, dv, B, init=False, g=[-0.003, -0.05, -0.3, -1.0])
    o, fin = ssd.ssd_linattn_chunk_scan(q[0], k[0], v[0], g[0])
    y, H = ssd.ssd_chunk_scan(v[0], torch.ones(B, L, hv, device="cuda"), g[0], k[0], q[0],
                              torch.zeros(hv, device="cuda"), 256)
    for a, b in ((y, o), (H.transpose(2, 3), fin)):       # the SSD scan's bound in bf16: 2e-2
        e = torch.linalg.vector_norm((a - b).double()) / torch.linalg.vector_norm(b.double())
        assert e < 2e-2, f"off by {e:.2e}"
