"""Workspace of the linear head's losses for few rows (CPU): what the rows that
are there need, and no more of the logits' gradient than the header allows."""
import pytest

import dense_gemm_linear_amd as dg


def _cdiv(a, b):
    return -(-a // b)


@pytest.mark.parametrize("T", [1, 3, 16, 48, 100, 128])
@pytest.mark.parametrize("V", [300, 50257, 131072, 600001, 1 << 24])
@pytest.mark.parametrize("D,slots", [(8, 0), (512, 0), (4096, 7)])
def test_few_rows_take_what_few_rows_need(T, V, D, slots):
    fwd = dg.linear_loss_workspace_bytes(T, V, D, slots)
    bwd = dg.linear_loss_workspace_bytes(T, V, D, slots, backward=True)
    # row tables (of 256 rows: place, row, what the gradient needs, the label's
    # z), X, five tables of targets, and what rounds each part up to 256 bytes
    common = 256 * 28 + 2 * T * D + 20 * T * slots + 8 * T + 20 * 256
    # one pair of floats per row and 64 columns
    assert fwd <= common + 8 * T * _cdiv(V, 64)
    # the logits' gradient in two bf16 halves, at most 256 MiB; dX's planes, at most 64, or as
    # many as give half of 512 workgroups one tile each
    halves = min(4 * T * _cdiv(V, 256) * 256, 256 << 20)
    planes = max(64, 256 // _cdiv(D, 128)) * 4 * T * D
    assert bwd <= max(common + halves + planes, fwd)
