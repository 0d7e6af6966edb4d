"""The usage example of the paged cache, run as it stands for two prompts and a step, gives what the
formulas give: prompts and generated tokens normed and rotated alike, once each, at their
rows, and no row of a prompt overwritten."""
import pathlib
import re

import numpy as np
import pytest
import torch

import state_space_model_mamba_amd as ssd
from attention_cases import F, host, randn
from oracle import paged as orc
from oracle.attention import attn

README = pathlib.Path(__file__).resolve().parents[1] / "README.md"


def example():
    """The example's lines from the append of prompts on (with what they name)."""
    blocks = re.findall(r"```python\n(.*?)```", README.read_text(), re.S)
    (block,) = [b for b in blocks if "ssd_attn_paged_append" in b]
    lines = block.splitlines()
    first = next((i for i, x in enumerate(lines) if x.startswith("turn =")), None)
    if first is None:
        first = next(i for i, x in enumerate(lines) if "ssd_attn_paged_append" in x)
    return "\n".join(lines[first:])


def test_the_example_is_found():
    assert "ssd_attn_paged_decode_step" in example() and "ssd_attn_paged_gather" in example()


@pytest.mark.gpu
def test_the_example_gives_what_the_formulas_give():
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    lens = [5, 37]
    T = sum(lens)
    gen = torch.Generator().manual_seed(1)
    (q, qv), (k, kv), (v, vv) = (randn(gen, T, h, D) for h in (Hq, Hkv, Hkv))
    (q_t, qtv), (k_t, ktv), (v_t, vtv) = (randn(gen, B, h, D) for h in (Hq, Hkv, Hkv))
    f = (1e4 ** (-2 * np.arange(D // 2) / D)).astype(np.float32)
    rng = np.random.default_rng(2)
    qw, kw = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in "qk")
    cu = np.concatenate([[0], np.cumsum(lens)])
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    names = dict(ssd=ssd, q=q, k=k, v=v, q_t=q_t, k_t=k_t, v_t=v_t, inv_freq=dev(f), qw=dev(qw), kw=dev(kw),
                 kp=torch.full((8, Hkv, page, D), float("nan"), device="cuda"),
                 vp=torch.full((8, Hkv, page, D), float("nan"), device="cuda"),
                 table=dev(np.array([[5, 0, 2, 7], [1, 6, 3, 4]], dtype=np.int32)),
                 lengths=torch.zeros(B, dtype=torch.int32, device="cuda"), cu_seqlens=cu,
                 prompt_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 cu_rows=np.concatenate([[0], np.cumsum([n + 1 for n in lens])]))
    exec(example(), names)
    o, o_t, rows = host(names["o"]), host(names["o_t"]), host(names["k"])
    # a score is off by (24 + 24 + D + 3) F of the sum of its products' sizes (a normed head's
    # length is below 2 sqrt(D), so at most 4 D scale = 32), a probability and the sum it is
    # divided by by that each; sums over 38 keys add less: 2^-11 of the largest value
    tol = 2 * (51 + D) * F * 32 + 2 * 46 * F
    assert tol < 2.0 ** -11
    at = 0
    for b, n in enumerate(lens):
        s = slice(cu[b], cu[b + 1])
        turned = lambda x, w, p: orc.turn_rows(x, w, 1e-6, p, f.astype(np.float64), False)[0]
        kk = turned(np.concatenate([kv[s], ktv[b:b + 1]]), kw, np.arange(n + 1))
        vals = np.concatenate([vv[s], vtv[b:b + 1]])
        qq = turned(np.concatenate([qv[s], qtv[b:b + 1]]), qw, np.arange(n + 1))
        assert max(np.linalg.norm(x, axis=-1).max() for x in (qq, kk)) < 2 * D ** 0.5
        want = np.stack([attn(qq[i:i + 1], kk[:i + 1], vals[:i + 1], D ** -0.5)[0][0] for i in range(n + 1)])
        assert np.abs(o[s] - want[:-1]).max() <= tol * np.abs(vals).max()
        assert np.abs(o_t[b] - want[-1]).max() <= tol * np.abs(vals).max()
        # the rows read back: normed and rotated once, within 24 F of a pair's sizes
        assert np.abs(rows[at:at + n + 1] - kk).max() <= 24 * F * 2 * np.abs(kk).max() + 64 * 2.0 ** -51
        at += n + 1
    assert names["lengths"].tolist() == [n + 1 for n in lens]
