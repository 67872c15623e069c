"""Infinities in an adapter, and inner values near fp32's largest, give the same on
every path: what the definition gives."""
import pytest
import torch

import dense_gemm_linear_amd as dg
from group_reference import close
from group_tiles import ADAPTER_SIZES
from test_gpu_group import _adapter_reference
from test_gpu_group_tiles import _adapters, _say

pytestmark = pytest.mark.gpu


def _check(got, X, W, A, B, off, order):
    want, err = (t.cpu() for t in _adapter_reference(X, W, A, B, None, off, order))
    assert not bool(torch.isnan(want).any())
    close(got, want, err, "Y")


@pytest.mark.parametrize("form,T,groups,N,K,R", ADAPTER_SIZES)
def test_infinite_entries(form, T, groups, N, K, R):
    """One infinity in some columns of B: its rows get it with the sign of their inner
    value, whatever bits that has; other columns stay finite."""
    _say("infinite", form, T, groups, N, K, R)
    ids, off, order, X, W, A, B, _ = _adapters(T, groups, N, K, R)
    its = int(ids[T - 1])
    # a row whose inner values are exact in bf16, next to those that are not
    X[T - 1] = 0
    X[T - 1, 0] = 1
    B[its, ::3, R // 2] = float("inf")
    B[its, 1::6, 0] = float("-inf")
    got = dg.linear_adapters(X, W, A, B, off, order)
    assert bool(torch.isinf(got[T - 1, ::3]).all())
    _check(got, X, W, A, B, off, order)


@pytest.mark.parametrize("form,T,groups,N,K,R", ADAPTER_SIZES)
def test_largest_inner_values(form, T, groups, N, K, R):
    """An inner value that fp32 holds and bf16 rounds to infinity: (33/32 2^63) (31/16
    2^64) = (2 - 2^-9) 2^127, against columns of zeros and of 2^-120."""
    _say("largest", form, T, groups, N, K, R)
    ids, off, order, X, W, A, B, _ = _adapters(T, groups, N, K, R)
    its, r = int(ids[T - 1]), R // 2
    X[T - 1] = 0
    X[T - 1, 0] = 33 / 32 * 2.0 ** 63
    A[its, :, 0] = 0
    A[its, r, 0] = 31 / 16 * 2.0 ** 64
    X[:T - 1, 0] = 0
    B[its, :, r] = 0
    B[its, 1::2, r] = 2.0 ** -120
    W[:, 0] = 0
    _check(dg.linear_adapters(X, W, A, B, off, order), X, W, A, B, off, order)
