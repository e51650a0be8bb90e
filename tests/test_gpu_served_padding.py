"""A served block with rows of x behind its last sequence (a padded batch): whatever they hold, NaN too, the sequences' rows and
the cache are the same, and the padding's slots write nothing."""
import pytest
import torch

from gpu_helpers import banner, dev
from test_gpu_served_block import D, HEADS, State, _layers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


@pytest.mark.parametrize("lens,pad", [([1, 1, 1], 5), ([37, 1, 5], 21), ([70, 60], 130)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [{}, {"cap": 20.0}])
def test_padding(G, lens, pad, bits, kw):
    from post_weight_quantization_07_amd.block import serve_block
    banner(f"served block, {lens} and {pad} rows of padding, int{bits} {kw}")
    tensors = {name: layer.dict for name, layer in _layers(True, True).items()}
    n = sum(lens)
    x = torch.randn(n, D, device=dev()).to(torch.bfloat16)
    outs, caches = [], []
    for fill in (0.0, float("nan"), float("inf"), 3.0):
        st = State(G, lens, bits)
        for t in (st.cache.k_codes, st.cache.v_codes):
            t.zero_()
        for t in (st.cache.k_scales, st.cache.v_scales):
            t.fill_(2.5)
        slots, *rest = st.args
        slots = torch.cat([slots, slots.new_full((pad,), -1)])
        xp = torch.cat([x, x.new_full((pad, D), fill)])
        outs.append(serve_block(tensors, xp, st.cache, slots, *rest, n_heads=HEADS, **kw)[:n])
        caches.append([t.clone() for t in (st.cache.k_codes, st.cache.v_codes, st.cache.k_scales, st.cache.v_scales)])
        touched = torch.zeros(st.cache.k_scales.shape[0] * st.cache.k_scales.shape[2], dtype=torch.bool, device=dev())
        touched[st.args[0]] = True
        held = (caches[-1][2] != 2.5).any(dim=1).flatten()               # slots whose scale is another now
        assert not (held & ~touched).any()
    assert torch.isfinite(outs[0]).all()
    for out, cache in zip(outs[1:], caches[1:]):
        assert torch.equal(out, outs[0]) and all(torch.equal(a, b) for a, b in zip(cache, caches[0]))
