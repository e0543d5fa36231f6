"""The router's gradient of tokens whose logits hold NaN or, under softmax,
+inf: the same whatever kernel the number of experts chooses. The chosen
experts get NaN, and with softmax scores that are not renormalised, where every
logit has a part in every weight, the whole row."""
import math

import pytest
import torch

from test_gpu_route import gpu_route, gpu_route_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [60, 64, 256, 512, 1024, 1028, 4096])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_rows_of_nan_and_infinity(E, renorm, sigmoid, kind):
    g = torch.Generator().manual_seed(31)
    T, k = 7, 5
    z = torch.randn(T, E, generator=g)
    z[1, 7] = math.nan
    z[3, E - 1] = math.inf
    z[4] = math.nan
    z[5] = -math.inf
    z[5, 2] = math.nan
    z = z.to(kind)
    _, ids, w = gpu_route([z], sigmoid, None, 1, 1, 1, k, renorm, 1.0)
    st, (got,) = gpu_route_grad([z], ids, w, [torch.randn(T, k, generator=g)], sigmoid, renorm, 1.0)
    assert st == 0
    full = not sigmoid and not renorm
    for t in range(T):
        bad = t in (1, 4, 5) or (t == 3 and not sigmoid)
        want = torch.zeros(E, dtype=torch.bool)
        if bad and full:
            want[:] = True
        elif bad:
            want[ids[0][t].long()] = True
        assert torch.equal(torch.isnan(got[t]), want), t
