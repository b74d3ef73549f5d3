"""What the residual blocks' layers refuse before anything is launched."""

import pytest
import torch

from amsgrad_optimizer_step_gb300 import layers


@pytest.mark.parametrize("coefs", [dict(z_coef=0.1), dict(balance_coef=0.01)])
def test_a_route_without_a_loss_takes_no_coefficients(coefs):
    with pytest.raises(ValueError):
        layers.route(torch.zeros(2, 8), 2, loss=False, **coefs)
