"""The operators around the layer at the edges of what they take, against 64-bit formulas."""
import pytest
import torch

import moe_megakernel_b200 as mk
from tests.test_gpu_operators import BF, gradient, ortho_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,dtype", [
    ((64, 1032, 520), BF), ((2400, 264, 136), BF), ((2400, 264, 135), BF), ((1200, 264, 136), torch.float32),
    ((2400, 135, 264), torch.float32)])
def test_orthogonalize_batches_with_several_pieces_to_a_warp(shape, dtype):
    """A warp of the scaling pass turns two to six 32 x 32 pieces one after the other through the same
    shared memory: every matrix of a large batch stays as near its 64-bit form as a matrix by itself."""
    G = gradient(*shape, seed=131, dtype=dtype)
    out = mk.orthogonalize(G)
    for at in range(0, shape[0], 400):
        ortho_close(out[at:at + 400], G[at:at + 400])
