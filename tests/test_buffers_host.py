"""Buffers of the host that the distillation from top logits refuses before any
launch (a kernel that reads or writes them may fault)."""
import pytest
import torch

from chunked_lm_head_gb300 import _lib, topk


def test_state_on_the_host():
    n = _lib.flce_topk_kd_state_bytes(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        topk._check_state(torch.zeros(n, dtype=torch.uint8), 4, 8)
    with pytest.raises(ValueError, match="same N and k"):
        topk._check_state(None, 4, 8)
    with pytest.raises(ValueError, match="same N and k"):
        topk._check_state(torch.zeros(n - 256, dtype=torch.uint8), 4, 8)


def test_workspace_on_the_host():
    with pytest.raises(ValueError, match="CUDA"):
        topk._workspace(torch.zeros(1 << 20, dtype=torch.uint8), 1 << 20, None, "cuda")
