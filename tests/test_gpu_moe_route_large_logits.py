"""Routing where logits are as large as their type holds: exponents of such logits
overflow fp32 long before the sigmoid or softmax does.  Few tokens (one a wave) and many
(four a wave) against the oracle; tolerances as in test_gpu_moe_route_many.py."""
import numpy as np
import pytest
import torch

import block_scaled_precision_04_amd as bs
from oracle import route
from tests.test_gpu_moe_route import _bias
from tests.test_gpu_moe_route_many import _check, _close

pytestmark = pytest.mark.gpu


def _rows(E, dtype, sigmoid):
    """Ordinary logits with one to E of them at +-the values around which log2(e) times
    them passes fp32, up to the type's largest."""
    g = np.random.default_rng(E)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    top = torch.finfo(t).max
    far = [2.3e38, 2.36e38, 2.4e38, 3.3e38, top]
    x = g.standard_normal((60, E)) * 1.5
    for r in range(60):
        n = min(E, (1, 2, 5, 20, E)[r % 5])
        at = g.permutation(E)[:n]
        big = g.choice(far, n)
        # (one sign a row: where both are there, a softmax keeps one choice and zeros)
        x[r, at] = big if r % 3 == 0 else (-big if r % 3 == 1 else big * g.choice([-1.0, 1.0], n))
    x = torch.tensor(np.clip(x, -top, top)).to(t)
    assert x.isfinite().all()
    return x.cuda(), x.double().numpy()


@pytest.mark.parametrize("E,groups,keep", [(8, 1, 1), (64, 1, 1), (256, 1, 1), (16, 4, 2), (64, 8, 3), (256, 8, 4), (256, 8, 1), (512, 16, 5)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_logits(E, groups, keep, sigmoid, dtype):
    x, xo = _rows(E, dtype, sigmoid)
    b, bo = _bias(E, E)
    k = min(8, keep * (E // groups))
    for top in (1, 2) if groups > 1 else (1,):
        for renorm in (True, False):
            ids, w = bs.moe_route(x, k, bias=b, score=int(sigmoid), groups=groups, topk_groups=keep, group_top=top,
                                  renorm=renorm, scale=2.5)
            io, wo = route.route(xo, k, bo, sigmoid, groups, keep, top, renorm, 2.5)
            bad = np.argwhere((ids.cpu().numpy() != io).any(1))
            assert not len(bad), (len(bad), int(bad[0, 0]), ids[int(bad[0, 0])].tolist(), io[bad[0, 0]])
            _close(w, wo)
            _check(x, xo, k, b, bo, sigmoid, groups, keep, top, renorm, 2.5)
