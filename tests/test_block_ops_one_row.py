"""One row (a single decoded token): its row stride means nothing, so the
wrappers around the linears neither hand it on to new tensors nor pass it to
the C entry points.  Host side only; the calls themselves are in
test_gpu_block_ops_edges.py."""
import pytest
import torch

from fine_grained_fp8_act_b200 import layer

BF16 = torch.bfloat16


def _rows(K):
    """[1, K] views of one row whose row stride is not K."""
    return [torch.zeros(3, 2 * K, dtype=BF16)[1:2, :K],           # hidden[:, -1] of a batch of one
            torch.zeros(1, K + 4, dtype=BF16)[:, :K],             # a stride that is no multiple of 8
            torch.zeros(K, 1, dtype=BF16).t()]                    # a stride below the row's length


@pytest.mark.parametrize("which", range(3))
def test_new_tensors_are_row_major(which):
    K = 96
    x = _rows(K)[which]
    assert x.stride(0) != K
    for dtype in (BF16, torch.float8_e4m3fn):
        assert layer._like(x, dtype=dtype).stride() == (K, 1)


@pytest.mark.parametrize("which", range(3))
def test_row_stride_of_one_row_is_its_length(which):
    K = 96
    x = _rows(K)[which]
    assert layer._check_bf16_matrix(x, "x") == (1, K, K)
    assert layer._check_like(x, "x", 1, K, x.device) == K
    assert layer._ld(x) == K


def test_row_stride_of_more_rows_stays():
    x = torch.zeros(4, 200, dtype=BF16)[:, :96]
    assert layer._check_bf16_matrix(x, "x") == (4, 96, 200)
    assert layer._like(x).stride() == (96, 1)
    assert layer._like(x.contiguous()).stride() == (96, 1)
    assert layer._ld(x) == 200
