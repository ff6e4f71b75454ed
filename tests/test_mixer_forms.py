"""Which form a prompt takes, by the workspace that it asks for: token by token
(the convolution's results, fp32) as long as that is no slower than chunks of 64
(CPU)."""
import pytest

import selective_state_space_25_amd as ss


def token_by_token(batch, L, heads, P=64, N=128, dtype=ss.BF16):
    need = ss.mamba2_conv_workspace_bytes(batch, L, heads, P, 1, N, 4, dtype)
    return need == (batch * L * (heads * P + 2 * N) * 4 + 255) // 256 * 256


# heads of 64 x 128: the longest prompt that goes token by token
@pytest.mark.parametrize("dtype", [ss.BF16, ss.F32])
@pytest.mark.parametrize("batch,longest", [(1, 32), (8, 32), (16, 16), (32, 8), (64, 7), (128, 7), (1000, 7)])
def test_by_length_and_heads(batch, longest, dtype):
    for L in range(1, 49):
        assert token_by_token(batch, L, 32, dtype=dtype) == (L <= longest), L


def test_small_heads_do_not_fill_the_gpu():
    assert token_by_token(64, 32, 4, 16, 16) and not token_by_token(64, 33, 4, 16, 16)
