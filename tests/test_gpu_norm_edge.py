"""Rows of the norm at fp32's upper end, whose factor 1 / sqrt(mean h^2) lies below its normal range: the bounds of
test_gpu_norm hold there too (the factor, s max|u|, its division and y are one rounding each)."""
import numpy as np
import pytest
import torch

from gpu_helpers import banner, dev, to_dev
from test_gpu_norm import check_codes, check_y

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def _large(d):
    """Rows whose root mean square goes from 2^125 to fp32's largest number."""
    r = np.random.default_rng(d)
    most = float(np.finfo(np.float32).max)
    return np.stack([(most * f * (1 - 0.1 * r.random(d)) * r.choice([-1.0, 1.0], d)).astype(np.float32)
                     for f in (1.0, 0.93, 0.7, 0.5, 0.31, 0.26, 0.24, 0.125)])


@pytest.mark.parametrize("d", [64, 1001, 4096, 12000, 16400])
@pytest.mark.parametrize("weights", ["none", "below 1", "tiny"])
def test_largest_rows(G, d, weights):
    banner(f"norm of the largest rows, d {d}, weights {weights}")
    x = _large(d)
    w = {"none": None, "below 1": np.linspace(0.1, 1.0, d).astype(np.float32),
         "tiny": (np.linspace(0.1, 1.0, d) * 2.0 ** -100).astype(np.float32)}[weights]
    wd = None if w is None else to_dev(w)
    y = torch.empty(x.shape, dtype=torch.float32, device=dev())
    rows, _ = G.gptq_norm_tokens(to_dev(x), wd, y=y)
    check_codes(rows, x, w, 1e-6)
    # (y is u s, u one rounding of h w: 2^-126 covers what lies below fp32's normal range)
    check_y(y, x, w, 1e-6)
    with_zeros = to_dev(x)
    _, total = G.gptq_norm_tokens(with_zeros, wd, torch.zeros_like(with_zeros))
    assert torch.equal(total, with_zeros)
