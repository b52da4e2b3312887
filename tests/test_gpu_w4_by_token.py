"""The 4-bit expert layer on both sides of the bound up to which L2 runs by token, for few and many slots, one
expert for all tokens among them."""
import pytest
import torch

from test_gpu_w4 import check_experts, experts_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k,EL", [(1, 1), (1, 4), (2, 2), (8, 8), (9, 12)])
@pytest.mark.parametrize("T,H", [(32, 256), (33, 256), (4, 2048), (5, 2048), (1, 8192), (2, 8192), (64, 128), (65, 128)])
def test_experts_at_the_bound(T, H, k, EL):
    check_experts(*experts_inputs(T, H, 128, EL, EL, k, 64, torch.bfloat16, True, seed=T + k))
