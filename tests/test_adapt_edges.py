"""Host-side checks at the edges of what adapts a block.  CPU only."""
import pytest
import torch

from activation_sparse_gemm_amd import calib


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
