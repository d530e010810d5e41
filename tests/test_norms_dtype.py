"""What `rms_norm` takes as its result's type: a torch.dtype or None, nothing else without a word (CPU)."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu


@pytest.mark.parametrize("dtype", ["bf16", "torch.bfloat16", 5, True, torch.zeros(1), [torch.bfloat16]])
def test_what_is_no_type_is_refused(dtype):
    with pytest.raises(TypeError, match="dtype: expected a torch.dtype or None"):
        # (an entry of 0 would be a fault if it were ever called)
        mu.training._describe().residual_norm(0, 0, 0, (torch.zeros(4, 8), None, None, None, None, None), False, True, 1e-6, dtype)


@pytest.mark.parametrize("dtype", [None, torch.bfloat16, torch.float32])
def test_types_are_taken(dtype):
    with pytest.raises(ValueError, match="x: expected a tensor on GPU 0"):
        mu.training._describe().residual_norm(0, 0, 0, (torch.zeros(4, 8), None, None, None, None, None), False, True, 1e-6, dtype)
