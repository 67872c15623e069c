"""The grouped rows' binding: the import, streams, and arguments that name themselves
when they are refused."""
import subprocess
import sys

import pytest
import torch

import dense_gemm_linear_amd as dg
from conftest import ROOT

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import dense_gemm_linear_amd as dg
print(dg.select_tile(512, 512, 512, num_cus=256).name)
try:
    dg.group_sort(torch.zeros(4, 2, dtype=torch.int64), 4)
except ValueError as e:
    print(e)
"""


def test_import_without_private_names():
    """The host's functions and the refusals need nothing that only some builds of
    torch have."""
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert dg.select_tile(512, 512, 512, num_cus=256).name in r.stdout and "group_sort: ids must be a device tensor" in r.stdout


@pytest.mark.gpu
def test_both_ways_to_the_stream():
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert dg._public_stream(0) == dg._raw_stream(0) == stream.cuda_stream
            assert dg._current_device() == torch.cuda.current_device()


@pytest.mark.parametrize("activation", ["swish", "", ["silu"], 1.0])
def test_activation_names_itself(activation):
    X, W = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="group_linear: activation"):
        dg.group_linear(X, W, torch.zeros(5, dtype=torch.int32), activation=activation)


def test_rows_of_2_gib():
    """Rows of X that span 2 GiB: refused where the loads pick them up by 32-bit offsets."""
    P, K = 0x10000, 1024
    fits = ((1 << 31) - K * 2 - 1) // (K * 2) + 1
    for T, status in ((fits, dg.GEMM_ERR_INVALID_VALUE), (fits + 1, dg.GEMM_ERR_UNSUPPORTED)):
        # (a null pointer elsewhere refuses what the size does not)
        Y = None if status == dg.GEMM_ERR_INVALID_VALUE else P
        assert dg.lib.group_linear(P, K, P, K, 8 * K, P, P, T, 1, 4, 8, K, 0, None, 0, Y, 8, None) == status
        assert dg.lib.linear_adapters(P, K, P, K, P, K, 8 * K, P, 8, 64, None, P, P, T, 8, K, 8, 4, Y, 8, P, 1 << 40,
                                      None) == status
