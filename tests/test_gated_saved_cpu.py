"""The tensors a gated block keeps between its passes: any sequence of the four, and
no other number of them reaches the library."""
import pytest
import torch

import bit_nf4_quantized_06_amd as q


@pytest.mark.parametrize("count", [0, 3, 5, 6])
@pytest.mark.parametrize("bwd", [False, True])
def test_saved_of_another_length_is_refused(count, bwd):
    bf = torch.bfloat16
    w = [q.NF4Weight.empty(128, 64, device="cpu") for _ in range(2)]
    x, a, b = torch.zeros(4, 64, dtype=bf), torch.zeros(16, 64, dtype=bf), torch.zeros(128, 16, dtype=bf)
    h, u = torch.zeros(4, 128, dtype=bf), torch.zeros(4, 16, dtype=bf)
    saved = ((h, h, u, u) + (u, u))[:count]
    with pytest.raises(ValueError, match="saved"):
        if bwd:
            q.qlora_gated_linear_bwd(*w, x, h, a, b, a, b, 16.0, saved)
        else:
            q.qlora_gated_linear_fwd(*w, x, a, b, a, b, 16.0, saved=saved)
