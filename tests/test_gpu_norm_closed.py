"""Closed lists of tensors are refused: a closed `out` is not the same as none, which clips in place."""
import pytest
import torch

from _gpu import need_gpu

pytestmark = pytest.mark.gpu


def test_closed_lists_are_refused():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    x, y = torch.ones(100, device="cuda"), torch.zeros(100, device="cuda")
    norm = torch.empty(1, device="cuda")
    lst, out = ofrl.TensorList([x]), ofrl.TensorList([y])
    out.close()
    with pytest.raises(ValueError, match="closed"):
        ofrl.global_norm_clip(lst, 1.0, norm, out=out)
    torch.cuda.synchronize()
    assert (x == 1).all() and (y == 0).all()
    lst.close()
    with pytest.raises(ValueError, match="closed"):
        ofrl.global_norm(lst, norm)
    with pytest.raises(ValueError, match="closed"):
        ofrl.global_norm_clip(lst, 1.0, norm)
    with pytest.raises(TypeError):
        ofrl.global_norm_clip(ofrl.TensorList([x]), 1.0, norm, out=[y])
