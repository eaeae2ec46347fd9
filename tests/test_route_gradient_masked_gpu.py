"""The routing gradient of places that name a masked expert: their weight does not
depend on the logits, so their gradient, whatever it holds, counts for nothing."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_b200 as fq
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [8, 60, 256, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("mask", [float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_at_masked_experts_count_for_nothing(E, score, renorm, mask, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(E)
    T, k = 12, 4
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dtype)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    clean = g.copy()
    for t in range(T - 1):
        at = ids[t, t % k]
        l[t, at] = mask
        g[t, t % k] = (np.nan, np.inf, -np.inf, 3e38)[t % 4]
        clean[t, t % k] = 0.0
    l[5, torch.from_numpy(ids[5]).long()] = mask             # all of a row's places
    g[5] = np.nan
    clean[5] = 0.0
    got = fq.fp8_moe_route_bwd(l.to(dev), torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev), score=score,
                               renorm=renorm).double().cpu().numpy()
    host = l.double().numpy()
    ref, mag = moe.route_bwd(host, ids, clean, score=score, renorm=renorm)
    # weights within (2 R + 64) u, R the spread of the logits (below 10), their gradients within twice that of the terms
    tol = 2 * (2 * 10 + 64) * 2.0 ** -24 * mag + 1e-35
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol)
    assert np.all(got[~(host > -np.inf)] == 0)
