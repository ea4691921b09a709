"""Shared by the tests of the layer operators: types, seeded inputs and comparisons with the fp64 oracle."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def need_gpu():
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def randn(gen, shape, t, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(TYPES[t]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, tol, what):
    """Every element within its tolerance; where the reference is not finite, the same."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities"
    if not fine.any():
        return
    got, ref, tol = got[fine], ref[fine], np.broadcast_to(tol, fine.shape)[fine]
    over = np.abs(got - ref) - tol
    at = int(np.argmax(over))
    assert over[at] <= 0, f"{what}: {got[at]} against {ref[at]}, {over[at]:.3e} over the tolerance"
