"""Linear attention at the ends of the number range."""
import pytest

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
