"""The order of the norm's roundings, as include/gq.h states it, bit for bit."""
import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,k,eps", [(1, 2560, 1e-5), (3, 33, 0.0), (200, 4096, 1e-6), (2, 40001, 1e-5)])
def test_norm_order_of_roundings(m, k, eps):
    """Rows of small whole numbers: their squares' sum is exact in any order, so that the rest is determined."""
    gq = need_gpu()
    rng = np.random.default_rng(3)
    h = rng.integers(-13, 14, (m, k)).astype(np.float32)
    w = rng.standard_normal(k).astype(np.float32)
    f = np.float32
    rstd = f(1) / np.sqrt((h * h).sum(-1, keepdims=True, dtype=np.float64).astype(f) / f(k) + f(eps))
    assert rstd.dtype == np.float32
    y = gq.rmsnorm(torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda(), eps).cpu().numpy()
    assert np.array_equal((h * rstd) * w, y)
    assert not np.array_equal((h * w) * rstd, y)
