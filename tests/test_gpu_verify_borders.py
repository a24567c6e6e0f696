"""Verification at its borders: more sequences than fit the device at once."""

import numpy as np
import pytest
import torch

from test_gpu_decode import _cuda, _no_device_errors  # noqa: F401
from test_gpu_tree import check_verify, drafted, run_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [304, 305, 1000, 5000])
@pytest.mark.parametrize("mode", ["draft", "point", "greedy"])
def test_more_sequences_than_fit_at_once(mode, R):
    """Four CTAs on each of 152 SMs, a cluster of two CTAs for each sequence: 304 of
    them fit."""
    rng = np.random.default_rng(R)
    sizes = [int(x) for x in rng.integers(0, 6, R)]
    for dtype, V in ((torch.float32, 97), (torch.bfloat16, 40)):
        args = drafted(rng, mode, sizes, V, dtype)
        check_verify(run_verify(*args, 4), *args, 4)
