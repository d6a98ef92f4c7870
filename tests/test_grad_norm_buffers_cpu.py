"""What grad_norm and clip_grad_norm say of a norm's buffer where there are no gradients to take
the GPU from."""
import os

import pytest

import cfc_recurrent_cell_amd as C
from cfc_recurrent_cell_amd import _lib

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH),
                                reason="libcfc_amd.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("call", [C.grad_norm, lambda grads, norm: C.clip_grad_norm(grads, 1.0, norm=norm)])
def test_norms_that_are_refused(call):
    for bad in (torch.zeros(()), torch.zeros(1), torch.zeros((), dtype=torch.float64)):
        with pytest.raises(ValueError, match="norm must be a contiguous torch.float32 tensor on a GPU"):
            call([], norm=bad)
    with pytest.raises(TypeError, match="norm must be a torch.Tensor"):
        call([], norm=1.0)
