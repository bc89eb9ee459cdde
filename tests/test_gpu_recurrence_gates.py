"""The gated linear recurrence's raw gates where a gate is nearly closed or open: what is left of a gradient there
is held to a relative bound."""
import pytest
import torch

from gpu_common import dev
from layer_common import DTYPES, Recurrence

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [68, 1700])
@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_of_open_and_closed_input_gates(dtype, sign, unit, C):
    """b from 4 to 30: sigmoid(b) (1 - sigmoid(b)) falls to 1e-13, of which 1 less a rounded sigmoid would keep nothing."""
    case = Recurrence([90, 1, 40], C, dtype, unit=unit, seed=21)
    b = 4 + 26 * torch.rand(case.b.shape, generator=torch.Generator("cpu").manual_seed(22))
    case.b.copy_((sign * b).to(dtype).to(dev()))
    y, final, chk = case.forward(return_checkpoints=True)
    case.check_forward(y, final)
    case.check_backward(case.backward(chk))
