"""Edges of the paged attention's calls that the tests beside it do not reach."""
import numpy as np
import pytest
import torch

from long_context_sparse_compress_b200 import lib as L
from tests.test_gpu_paged import BF16, Case

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ failure path

@pytest.mark.parametrize("stall", [True, False])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 30, 3], [90, 60, 5]])
def test_waits_that_give_up_at_once(cuda_lib, new, stall):
    """A limit of a nanosecond ends roles while copies and products of their CTA
    are in flight; each CTA waits for those, and the next call is right."""
    c = Case([3000, 400, 7000], new, 8, 2, 128, 64, BF16, seed=30)
    c.run().check()
    for _ in range(20):
        L.set_wait_test(1, stall)
        try:
            c.run()
            torch.cuda.synchronize()
        finally:
            L.set_wait_test(0, False)
        assert c.status.item() in ((L.DEV_TIMEOUT,) if stall else (0, L.DEV_TIMEOUT))
    c.run().check()
