"""min-p beside top-p without top-k, and at high temperatures, against the fp64
oracle (tolerances and marks as in test_gpu_sample.py)."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_attn_gb300 as bdsa  # noqa: F401
from test_gpu_sample import DEV, check, params, run

pytestmark = pytest.mark.gpu


def both(l, u, **kw):
    t, p = run(l, u, **kw)
    check(l, u, t, p, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 33, 300, 1000, 5003, 40001, 151936])
@pytest.mark.parametrize("which", [("top_p", "min_p"), ("temperature", "top_p", "min_p"),
                                   ("top_k", "min_p")])
def test_pairs_of_filters(dtype, V, which):
    rng = np.random.default_rng(V + len(which))
    bs, B = 4, 3
    for std in (0.3, 3.0):
        l = torch.from_numpy(rng.normal(size=(bs, B, V)).astype(np.float32) * std)
        u = rng.random((bs, B), dtype=np.float32)
        both(l.to(DEV).to(dtype), u, **params(rng, bs, V, which))


def test_a_bin_of_part_maxima_that_holds_the_cut():
    """100 logits just below the largest and 20 behind them, over a bulk far below:
    the nucleus ends among the 20, min-p keeps them all."""
    V, T = 5003, 0.05
    l = np.full(V, -25.0, np.float32)
    l[40:440:4] = -1.95 * T
    l[1000:1080:4] = -2.5 * T
    l[8] = 0.0
    for dtype in (torch.float32, torch.bfloat16):
        lt = torch.from_numpy(l).to(DEV).to(dtype).view(1, 1, V)
        for tp in (0.9, 0.95, 0.99, 0.999):
            both(lt, [[0.7]], temperature=[T], top_p=[tp], min_p=[0.05])
            both(lt, [[0.7]], temperature=[T], top_p=[tp], min_p=[1e-4])


@pytest.mark.parametrize("mask", [-100.0, -1000.0, -1e4])
@pytest.mark.parametrize("V", [2003, 5003, 40001])
def test_finite_masks(mask, V):
    """Half the vocabulary at a finite mask value: the parts' maxima span a wide
    range, and a bin of it many tokens."""
    rng = np.random.default_rng(V)
    bs, B = 16, 4
    l = rng.normal(size=(bs, B, V)).astype(np.float32) * 3
    l[rng.random((bs, B, V)) < 0.5] = mask
    # whole parts masked, so that the smallest part maximum is the mask
    l[:, :, V // 4:V // 2] = mask
    u = rng.random((bs, B), dtype=np.float32)
    for T in (0.05, 0.3, 1.0, 2.0):
        kw = dict(temperature=np.full(bs, T, np.float32),
                  top_p=rng.uniform(0.5, 0.999, bs).astype(np.float32))
        for dtype in (torch.float32, torch.bfloat16):
            lt = torch.from_numpy(l).to(DEV).to(dtype)
            both(lt, u, **kw, min_p=rng.uniform(1e-4, 0.1, bs).astype(np.float32))
            both(lt, u, **kw)
