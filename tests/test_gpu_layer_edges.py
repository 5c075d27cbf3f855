"""Edges of the layer around retention that the sizes of test_gpu_layer.py do not
reach, against the float64 definitions of oracle/layer.py; tolerances as there
unless stated."""
import numpy as np
import pytest

from oracle import layer as ol
from tests.gpu_util import down, note, torch_dev
from tests.test_gpu_layer import EPS, U, _msr, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d", [(3001, 1000), (2048, 256)])
def test_weight_gradient_rounding(rows, d):
    """The size of dweight's rounding, not its bound.  One fp32 rounding is uniform over +-2^-24 of the binade, rms
    s = 2^-24 / sqrt(3) * 0.74 = 2.5e-8 of a value spread evenly over it in the logarithm.  Of N random terms a partial sum
    of k has k / N of the result's square, so in units of s^2 the variance is: a term's product 1 and its row's rstd 3
    (mean 4 / 4, root, reciprocal); a team's turns 3.5 (6 of them, 502 teams, 3001 rows; 1 for 2048 x 256), the teams of
    a workgroup 1 (3.3), four parts in a slice 2.3, 64 slices in pairs 6: 16.8 (16.6).  That is 4.1 s = 1.04e-7; a quarter
    more is allowed.  A chain over the slices has 32 in place of 6: 1.7e-7."""
    torch, dev = torch_dev()
    msr = _msr()
    h, hf = values(torch, dev, (rows, d), "f32", 61, spread=False)
    dy, dyf = values(torch, dev, (rows, d), "f32", 62, spread=False)
    _, dw = msr.msr_add_rmsnorm_backward(h, None, dy, eps=EPS)
    want = ol.add_rmsnorm_backward(hf, None, dyf, None, EPS)[1]
    err = np.linalg.norm(down(dw) - want) / np.linalg.norm(want)
    note(f"dweight {rows}x{d}: {err:.3g} of its norm")
    assert err <= 1.3e-7
