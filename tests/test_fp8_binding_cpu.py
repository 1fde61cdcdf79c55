"""What the 8-bit layer's binding refuses on the host, by the name of the
tensor at fault. Nothing here launches a kernel."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("scales,good", [
    ((4, 2, 3), True), ((2, 3), False), ((1, 2, 3), False), ((4, 2, 2), False), ((8, 3), False), ((4, 6), False)])
def test_bank_scales_have_one_matrix_per_expert(scales, good):
    """Scales without the experts' dimension are too short for more than one expert."""
    b = (codes(4, 200, 300), torch.zeros(scales))
    with pytest.raises(ValueError, match="CUDA" if good else "scales"):  # (a good bank: only not on a GPU)
        smr._bank8(b, (4, 200, 300))


@pytest.mark.parametrize("shape,scales,good", [
    ((200, 300), (2, 3), True), ((1, 200, 300), (1, 2, 3), True), ((200, 300), (1, 2, 3), True),
    ((1, 200, 300), (2, 3), True), ((200, 300), (2, 2), False), ((200, 300), (3, 2), False)])
def test_bank_of_one_matrix_may_leave_its_dimension_out(shape, scales, good):
    with pytest.raises(ValueError, match="CUDA" if good else "scales"):
        smr._bank8((codes(*shape), torch.zeros(scales)), (1, 200, 300))
