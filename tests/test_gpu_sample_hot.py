"""min-p near one at high temperatures: the logit the weight m belongs to, T ln m
below the largest, is a small difference of it (fp64 oracle, marks and tolerances as
in test_gpu_sample.py)."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DEV, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [30.0, 1000.0, 3e4])
@pytest.mark.parametrize("others", [(), ("top_k",), ("top_p",)])
def test_logits_around_the_cut(T, others):
    """Logits from 4e-9 to 1e-6 T to either side of the cut, the largest at 0."""
    rng = np.random.default_rng(int(T))
    bs, V = 96, 5003
    m = np.concatenate([rng.uniform(0.9, 0.9999, bs - 4),
                        [0.5, 0.99999, 0.999999, 0.9]]).astype(np.float32)
    d = 10.0 ** rng.uniform(np.log10(4e-9), -6, (bs, 200)) * rng.choice([-1.0, 1.0], (bs, 200))
    l = np.full((bs, 1, V), -T, np.float32)
    at = rng.choice(V - 1, 200, replace=False)
    l[:, 0, at] = np.minimum(T * (np.log(m.astype(np.float64))[:, None] + d), 0.0)
    l[:, 0, V - 1] = 0.0
    kw = dict(temperature=np.full(bs, T, np.float32), min_p=m)
    if "top_k" in others:
        kw["top_k"] = np.full(bs, 150, np.int32)
    if "top_p" in others:
        kw["top_p"] = np.full(bs, 0.9, np.float32)
    u = rng.random((bs, 1), dtype=np.float32)
    lt = torch.from_numpy(l).to(DEV)
    t, p = run(lt, u, **kw)
    near = check(lt, u, t, p, **kw)
    assert near.mean() < 0.5
