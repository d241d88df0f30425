"""Host-side checks of the layer policy's norm and adapters and of the trained fit.  CPU only."""
import pytest
import torch

from activation_sparse_gemm_amd import calib, policy


def test_norm_takes_one_length():
    with pytest.raises(ValueError):
        policy.AdaptiveNorm(torch.ones(8), torch.zeros(16))
    policy.AdaptiveNorm()
    policy.AdaptiveNorm(torch.ones(8), torch.zeros(8))


@pytest.mark.parametrize("LA,LB", [((2, 40, 8), (2, 8, 64)), ((2, 48, 8), (3, 8, 64)), ((2, 48, 8), (2, 16, 64)),
                                   ((2, 48, 8), (2, 8, 72)), ((48, 8), (8, 64)), ((2, 48, 8), (8, 64))])
def test_adapters_must_fit_the_projection(LA, LB):
    lin = policy.Linear(torch.zeros(48, 64), sparse=False)
    with pytest.raises(ValueError):
        policy.AdaptedLinear(lin, torch.zeros(LA), torch.zeros(LB))


def test_adapters_factors():
    lin = policy.Linear(torch.zeros(48, 64), sparse=False)
    LA, LB = torch.zeros(2, 48, 8), torch.zeros(2, 8, 64)
    policy.AdaptedLinear(lin, LA, LB, torch.ones(2))
    with pytest.raises(ValueError):
        policy.AdaptedLinear(lin, LA, LB, torch.ones(3))


def test_trained_fit_refuses():
    X, E = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(16, 48, dtype=torch.bfloat16)
    for bad in (dict(X=X.float()), dict(E=E.float()), dict(E=E[:8]), dict(X=X[0]), dict(R=0), dict(R=49), dict(rows=0), dict(steps=-1),
                dict(LA=torch.zeros(48, 8))):
        with pytest.raises(ValueError):
            calib.train_lowrank(**{**dict(X=X, E=E, R=8), **bad})
