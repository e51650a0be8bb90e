"""Pairs of what changes a score that test_gpu_attention_scores does not take together: a cap or a bias with a prefix, caps past
2^8 with both, slopes that grow with the distance over many tiles of keys (bounds: there)."""
import numpy as np
import pytest
import torch

from gpu_helpers import banner
from test_gpu_attention import Case
from test_gpu_attention_scores import CASES, _call, _prefixes, _slopes, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["cap prefix", "slopes prefix", "wide slopes prefix", "wide slopes"])
@pytest.mark.parametrize("lens,heads,kv,hd,page", CASES)
def test_pairs(G, lens, heads, kv, hd, page, kind, bits):
    banner(f"attention {kind} {lens} {heads}/{kv}x{hd} page {page} int{bits}")
    c = Case(G, lens, heads, kv, hd, page, bits, seed=31)
    cap = 4.0 if "cap" in kind else 900.0 if "wide" in kind else None
    slopes = _slopes(heads) if "slopes" in kind else None
    prefixes = _prefixes(lens, hd + 1) if "prefix" in kind else None
    out = _call(G, c, cap, slopes, prefixes)
    check(c, out, cap, slopes, prefixes)
    assert torch.equal(out, _call(G, c, cap, slopes, prefixes))


@pytest.mark.parametrize("lens", [[(1, 3000), (1, 700)], [(20, 3000)], [(200, 2000), (130, 700)]])
@pytest.mark.parametrize("slope", [-0.5, 0.0, 0.5, 40.0])
@pytest.mark.parametrize("prefix", [None, 900, 3000])
def test_slopes_over_many_keys(G, lens, slope, prefix):
    """Every head alike: the weight lies on the first keys, on all, on the nearest ones, on the nearest alone."""
    banner(f"attention: slope {slope}, prefix {prefix}, {lens}")
    c = Case(G, lens, 4, 2, 64, 16, 8, seed=32)
    slopes = np.full(4, slope, np.float32)
    prefixes = None if prefix is None else np.full(len(lens), prefix, np.int32)
    for cap in (None, 6.0):
        check(c, _call(G, c, cap, slopes, prefixes), cap, slopes, prefixes)
