"""device_status by every name of the current device."""
import pytest
import torch

import log_space_sum_gb300 as pc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", [lambda i: None, lambda i: i, lambda i: f"cuda:{i}", lambda i: "cuda",
                                  lambda i: torch.device("cuda"), lambda i: torch.device("cuda", i)])
def test_device_status(name):
    pc.device_status(name(torch.cuda.current_device()))
