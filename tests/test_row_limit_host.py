"""Row counts that the norm and the distillation from top logits refuse before
any launch: their kernels count rows in 32 bits, up to a grid past the last."""
import pytest

from chunked_lm_head_gb300 import _lib

from test_norm_host import INVALID, OK, back, norm, norm8
from test_topk_host import bwd, fb, fwd, teacher

MOST = 2 ** 31 - 1 - 65536


@pytest.mark.parametrize("N", [MOST + 1, 2 ** 31 - 2])
def test_rows_past_the_row_counters(N):
    assert norm(N=N, H=8, ldx=8) == INVALID
    assert norm8(N=N, H=16, ldx=16) == INVALID
    assert back(N=N, H=8, lds=8) == INVALID
    assert _lib.flce_rms_norm_backward_workspace_bytes(N, 8) == 0
    assert fwd(teacher(), N=N, H=8) == INVALID
    assert fb(teacher(), N=N, H=8) == INVALID
    assert bwd(N=N, H=8) == INVALID
    assert _lib.flce_topk_kd_state_bytes(N, 4) == 0
    assert _lib.flce_topk_kd_workspace_bytes(N, 8, 100, 4, 256) == 0


def test_the_most_rows_are_taken():
    assert _lib.flce_rms_norm_backward_workspace_bytes(MOST, 8) > 0
    assert _lib.flce_topk_kd_state_bytes(MOST, 4) > 0
    assert _lib.flce_topk_kd_workspace_bytes(MOST, 8, 100, 4, 256) > 0
    assert norm(N=0) == OK
