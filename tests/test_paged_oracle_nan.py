"""The oracle's 4-bit rows of NaN and infinities: the step of a group with a NaN, or of infinities of
one sign alone, is NaN, its codes 0, and all its values come back as NaN; other groups stay."""
import numpy as np
import pytest

from oracle import paged as orc


@pytest.mark.parametrize("put", [{5: np.nan}, {i: np.nan for i in range(64)}, {0: np.nan, 63: np.inf},
                                 {i: np.inf for i in range(64)}, {i: -np.inf for i in range(64)}])
@pytest.mark.filterwarnings("error")
def test_groups_without_a_step(put):
    x = np.random.default_rng(1).standard_normal(128)
    clean = orc.load4(*orc.store4(x))
    y = x.copy()
    for i, v in put.items():
        y[64 + i] = v
    codes, scales = orc.store4(y)
    assert np.isnan(scales[1, 0]) and not codes[32:].any()
    back = orc.load4(codes, scales)
    assert np.isnan(back[64:]).all() and np.array_equal(back[:64], clean[:64])
