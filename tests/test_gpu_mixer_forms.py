"""Short prompts of a batch that fills the GPU, on both sides of the length where
the mixer goes over from single tokens to chunks; bounds as for other prompts."""
import pytest
import torch

from mixer_close import close
from test_gpu_mixer import Inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("L", [5, 7, 8])
@pytest.mark.parametrize("ragged", [False, True])
def test_full_batch(gpu, L, ragged):
    i = Inputs(64, L, 32, 1, 64, 128, 4, BF16)
    lengths = [(3 * b) % (L + 2) for b in range(64)] if ragged else None
    y, S, cs = i.fwd(BF16, lengths)
    torch.cuda.synchronize()
    (ry, rS, rcs), (my, mS) = i.ref(lengths)
    close(y, ry, my, 96 + 4 * L, "y")
    close(S, rS, mS, 96 + 4 * L, "state")
    assert torch.equal(cs.cpu().double(), rcs)
