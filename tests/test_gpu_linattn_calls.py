"""Calls of linear attention that its documentation allows and whose answers are
easy to lose. Tolerances as in test_gpu_linattn.py unless stated."""
import pytest
import torch

import selective_state_space_42_b200 as ss

from test_gpu_linattn import DEV, DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 0, 3, 8), (0, 4, 3, 8)], ids=str)
def test_empty_decays_have_an_empty_gradient(dtype, shape):
    z = torch.zeros(shape, device=DEV, dtype=DT[dtype])
    g = ss.selscan_linattn_bwd(z, z, z, z[..., 0].contiguous(), dy=z)
    assert g["dlog_decay"] is not None and g["dlog_decay"].shape == shape[:3]
    assert ss.selscan_linattn_bwd(z, z, z, torch.zeros(3, device=DEV), dy=z)["dlog_decay"] is None
