"""Host-side checks at the edges of what adapts a block.  CPU only."""
import pytest
import torch

import activation_sparse_gemm_amd as rtl
from activation_sparse_gemm_amd import calib
from test_block_abi import Buffers, refused


@pytest.mark.parametrize("M,rows", [(1, 1), (128, 128), (129, 128), (255, 128), (256, 128), (300, 128), (383, 128), (384, 128),
                                    (12, 5), (8191, 4096), (8192, 4096), (12287, 4096), (12288, 4096)])
def test_batches_take_all_rows_alike(M, rows):
    """Consecutive batches are consecutive rows, the first behind the last: after k of them each row was met k rows / M
    times, rounded up or down."""
    X = torch.arange(M).view(M, 1)
    met, at = torch.zeros(M, dtype=torch.long), 0
    for step in range(9):
        batch = calib._batch(X, step, rows).flatten()
        assert torch.equal(batch, (at + torch.arange(rows)) % M)
        at += rows
        met += torch.bincount(batch, minlength=M)
        assert int(met.max()) - int(met.min()) <= 1


@pytest.mark.parametrize("back", (False, True))
@pytest.mark.parametrize("rest", (-1, 2, 2 ** 31 - 1))
def test_rest_is_kept_or_zeros(back, rest):
    b = Buffers()
    M, D, G = 6, 64, 2
    X, Y, dY, stats, groups = b(2 * M * D), b(2 * M * D), b(2 * M * D), b(8 * M), b(16)
    if back:
        need = rtl.rtl_layer_norm_backward_workspace_bytes(M, D, G)
        st = rtl.lib.rtl_layer_norm_backward_ex(rest, rtl.RTL_BF16, M, D, X, D, stats, dY, D, None, None, G, groups, None, 0, Y, D,
                                                None, None, None, None, b(need), need, None)
    else:
        st = rtl.lib.rtl_layer_norm_ex(rest, rtl.RTL_BF16, M, D, X, D, None, None, G, groups, None, 0, None, 0, 1e-6, Y, D, stats,
                                       None)
    refused(st, "RTL_ERR_ARG", b, rest)


@pytest.mark.parametrize("LA,LB", [((48, 16), (16, 64)), ((48, 8), (8, 72)), ((40, 8), (8, 64)), ((48, 8), (64, 8)), ((8, 48), (8, 64))])
def test_trained_fit_starts_from_factors_of_its_rank(LA, LB):
    X, E = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(16, 48, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rank 8"):
        calib.train_lowrank(X, E, 8, LA=torch.zeros(LA), LB=torch.zeros(LB))
