"""Refusals of the many-adapter binding that need no GPU."""

import pytest
import torch

from bit_nf4_quantized_amd import api


def test_host_gradients_are_refused_as_such():
    for grads in ([torch.zeros(8)], [torch.zeros(8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.bfloat16)]):
        with pytest.raises(ValueError, match="grads must be a device tensor"):
            api.qlora_clip_grad_norm_batch(grads, 1.0)
