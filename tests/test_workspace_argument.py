"""A workspace that the GPU cannot write, or whose elements are not where its
size says, is refused before its address is passed on (CPU)."""
import pytest
import torch

import selective_state_space_25_amd as ss

HERE = torch.device("cpu")


def test_workspace_on_another_device():
    with pytest.raises(ValueError, match="workspace"):
        ss._ws_arg(torch.empty(1024, dtype=torch.uint8), 512, torch.device("cuda:0"))


def test_workspace_that_is_not_dense():
    with pytest.raises(ValueError, match="workspace"):
        ss._ws_arg(torch.empty(1, dtype=torch.uint8).expand(1 << 20), 1 << 20, HERE)


def test_workspace_that_is_no_tensor():
    with pytest.raises(TypeError, match="workspace"):
        ss._ws_arg(bytearray(1024), 512, HERE)


def test_workspace_taken():
    w = torch.empty(100, dtype=torch.float32)
    assert ss._ws_arg(w, 400, HERE) == (w.data_ptr(), 400, w)
    assert ss._ws_arg(None, 0, HERE) == (None, 0, None)
