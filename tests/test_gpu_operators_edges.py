"""Linear attention and the norm where paths, magnitudes and workspaces meet
their limits, on the GPU against the float64 oracle.  Tolerances are those of
test_gpu_linear_attention.py and test_gpu_qk_norm.py, derived there."""
import ctypes

import numpy as np
import pytest
import torch

from tests import operators_oracle as O
from tests import test_gpu_linear_attention as LA

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def P():
    from linear_recurrent_sequence_shortconv_amd import prism
    return prism


# ------------------------------------------------------------ empty batches
@pytest.mark.parametrize("packed", [False, True])
def test_dg_of_one_decay_a_head_without_sequences(packed):
    """No sequence adds to it: zeros, written without a workspace."""
    L = P().lib()
    desc = P().LinearAttentionDesc(B=0, T=5, H=4, Hk=2, dk=32, dv=32, dtype=P().PRISM_BF16, scale=1.0)
    for n, H in (("q", 4), ("k", 2), ("v", 2), ("o", 4)):
        setattr(desc, n, P().Strides(5 * H * 32, H * 32, 32))
    desc.g = P().Strides(0, 0, 1)
    g = torch.full((4,), -0.1, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    dg = torch.full((4,), float("nan"), device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    st = L.prism_linear_attention_backward(
        ctypes.byref(desc), None, None, None, ptr(g), None, ptr(cu) if packed else None, None, None, None, None,
        None, ptr(dg), None, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and dg.tolist() == [0.0] * 4
