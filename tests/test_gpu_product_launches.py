"""The integer products at sizes where the launch changes from one kernel or split to another, against
their 64-bit forms (bounds: test_gpu_epilogue)."""
import pytest
import torch

from gpu_helpers import banner, host
from oracle import serving_oracle as S
from test_gpu_epilogue import Layer, _product64, _x, activated, near

import numpy as np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def check(G, m, d_in, rows, gated, act="silu"):
    """The product alone, with all that may follow it, or gated, for raw tokens and their codes, in both types."""
    d_out = rows // 2 if gated else rows
    banner(f"{m}x{d_in}->{d_out} gated={gated} act={act}")
    x = _x(m, d_in, "bf16", m + d_in)
    first, second = Layer(d_out, d_in, 1, True, True), Layer(d_out, d_in, 2, False, False)
    codes, scales = S.row_codes(host(x), 127)
    inputs = (x, G.gptq_quantize_tokens(x))
    t = first.dict
    a, da = activated(*_product64(first, codes, scales), act)
    if gated:
        z, dz = _product64(second, codes, scales)
        ref, err = a * z, np.abs(z) * da + np.abs(a) * dz + da * dz
        for dtype in (torch.float32, torch.bfloat16):
            y = [G.gptq_integer_gated(inp, first.dict, second.dict, act, out_dtype=dtype) for inp in inputs]
            near(y[0], ref, err)
            assert torch.equal(*y)
        return
    res = torch.randn(m, d_out, device=x.device).to(torch.bfloat16)
    ref, err = a + host(res).astype(np.float64), da + U * np.abs(a)
    plain = Layer(d_out, d_in, 1, True, False)
    plain_ref = _product64(plain, codes, scales)
    for dtype in (torch.float32, torch.bfloat16):
        kw = dict(bias=t["bias"], activation=act, residual=res, out_dtype=dtype)
        y = [G.gptq_integer_matmul(inp, t["w"], t["scales"], t["offsets"], **kw) for inp in inputs]
        near(y[0], ref, err)
        assert torch.equal(*y)
        y = [G.gptq_integer_matmul(inp, t["w"], t["scales"], t["offsets"], out_dtype=dtype) for inp in inputs]
        near(y[0], *plain_ref)
        assert torch.equal(*y)


# the stream kernel with two to five blocks of 64 tokens, the last one full or of few, whole and broken row blocks
BLOCKS = [(65, 256, 4096), (80, 1024, 1024), (128, 768, 770), (129, 1024, 1034), (200, 96, 66), (256, 768, 768), (257, 512, 130),
          (320, 768, 514)]


@pytest.mark.parametrize("m,d_in,rows", BLOCKS)
@pytest.mark.parametrize("gated", [False, True])
def test_blocks_of_tokens(G, m, d_in, rows, gated):
    check(G, m, d_in, rows, gated, ("relu", "gelu", "gelu_tanh", "silu")[(m + d_in) % 4])


# row blocks of one, two and four for few tokens, quantized on the way and given in codes, on both sides of each limit
FEW = [(1, 256, 12288), (1, 256, 12300), (1, 1024, 16390), (1, 1056, 24576), (1, 1056, 24600), (1, 2560, 24600), (1, 4128, 12300),
       (1, 4128, 16400), (1, 4096, 8200), (2, 512, 12400), (2, 544, 12400), (2, 544, 24600), (4, 4096, 8200), (3, 4128, 16400),
       (1, 8192, 12300), (3, 4128, 8200)]


@pytest.mark.parametrize("m,d_in,rows", FEW)
@pytest.mark.parametrize("gated", [False, True])
def test_row_blocks(G, m, d_in, rows, gated):
    check(G, m, d_in, rows, gated)


# sizes whose kernel the estimate chooses by few per cent: streamed, in tiles, in K slices of them
CLOSE = [(8, 11008, 2048), (17, 4096, 6150), (33, 4096, 4100), (40, 4096, 4096), (100, 4128, 1030), (300, 1024, 4100), (17, 10016, 4100)]


@pytest.mark.parametrize("m,d_in,rows", CLOSE)
@pytest.mark.parametrize("gated", [False, True])
def test_close_choices(G, m, d_in, rows, gated):
    check(G, m, d_in, rows, gated, "gelu_tanh")


# Tiles without K slices whose ring of LDS slots turns several times: 128 x 128 (two slots) in 4 to 17 steps, 256 x 256 (two) in 6
# to 16, 64 x 128 (four) in 9 to 17, whole numbers of turns and broken ones, with edges inside a tile
PASSES = [(1100, 1024, 4100), (777, 1056, 8200), (1100, 512, 2200), (700, 2080, 4170),
          (2100, 768, 4200), (2050, 1056, 8200), (4100, 2048, 2100),
          (600, 1568, 2070), (300, 2080, 2100), (100, 1056, 8200)]


@pytest.mark.parametrize("m,d_in,rows", PASSES)
@pytest.mark.parametrize("gated", [False, True])
def test_passes(G, m, d_in, rows, gated):
    assert G.gptq_integer_workspace_size(m, torch.int8, d_in, rows) == 0   # codes given: room for K slices only
    check(G, m, d_in, rows, gated, ("relu", "gelu", "gelu_tanh", "silu")[(m + rows) % 4])
