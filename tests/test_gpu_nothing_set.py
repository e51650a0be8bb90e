"""The calls that change a product's or an attention's values, with nothing set: bit for bit what the plain calls of the
C ABI give.  (The bindings take the plain call there by themselves, so the entries are called directly.)"""
import ctypes

import pytest
import torch

from gpu_helpers import banner, dev
from test_gpu_attention import Case
from test_gpu_epilogue import Layer, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


@pytest.mark.parametrize("m,d_in,d_out", [(1, 4096, 300), (3, 160, 8200), (16, 512, 16500), (40, 768, 500), (100, 1024, 770), (300, 2080, 2100),
                                          (1100, 512, 2200), (2100, 768, 4200), (65, 2048, 100)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_linear_without_anything(G, m, d_in, d_out, out):
    banner(f"linear with nothing set {m}x{d_in}->{d_out} {out}")
    from post_weight_quantization_07_amd import _lib as L
    lib, layer = L._lib(), Layer(d_out, d_in, 7, True, False)
    t = layer.dict
    x = _x(m, d_in, "bf16", m)
    codes, scales, sums = G.gptq_quantize_tokens(x)
    yt = L._type_code("test", out)
    c = L._CLayer(t["w"].data_ptr(), t["scales"].data_ptr(), t["offsets"].data_ptr(), None)
    for inp, code, sc, sm in ((x, L.GPTQ_BF16, None, None), (codes, L.GPTQ_I8, scales.data_ptr(), sums.data_ptr())):
        need = lib.gptq_integer_workspace_size(m, code, d_in, d_out)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev())
        y = [torch.full((m, d_out), fill, dtype=out, device=dev()) for fill in (7.0, -9.0)]   # equal once written
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.gptq_integer_matmul(inp.data_ptr(), code, sc, sm, m, d_in, d_in, t["w"].data_ptr(), t["scales"].data_ptr(),
                                       t["offsets"].data_ptr(), d_out, y[0].data_ptr(), yt, ws.data_ptr(), need, stream) == 0
        assert lib.gptq_integer_linear(inp.data_ptr(), code, sc, sm, m, d_in, d_in, c, d_out, 0, None, 0, 0, y[1].data_ptr(),
                                       yt, ws.data_ptr(), need, stream) == 0
        torch.cuda.synchronize()
        same = torch.equal(*y)
        assert same


@pytest.mark.parametrize("lens", [[(1, 300), (1, 65), (1, 2000)], [(20, 300), (13, 40)], [(200, 300), (130, 130)]])
@pytest.mark.parametrize("bits", [8, 4])
def test_attention_without_anything(G, lens, bits):
    banner(f"attention with nothing set {lens} {bits} bits")
    from post_weight_quantization_07_amd import _lib as L
    lib = L._lib()
    c = Case(G, lens, 4, 2, 64, 16, bits)
    table, starts, kv = c.args
    q = c.q
    n, heads, hd = q.shape
    need = lib.gptq_attention_workspace_size(c.cache._ref, n, heads, len(lens), table.shape[1])
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev())
    out = [torch.full_like(q, fill) for fill in (7.0, -9.0)]   # equal once written
    stream = torch.cuda.current_stream().cuda_stream
    args = (c.cache._ref, q.data_ptr(), L.GPTQ_BF16, n, heads * hd, heads, table.data_ptr(), table.shape[1], starts.data_ptr(),
            kv.data_ptr(), len(lens), ctypes.c_float(hd ** -0.5))
    assert lib.gptq_cache_attention(*args, out[0].data_ptr(), heads * hd, ws.data_ptr(), need, stream) == 0
    assert lib.gptq_cache_attention_scores(*args, L._CScores(0.0, None, None), out[1].data_ptr(), heads * hd, ws.data_ptr(),
                                           need, stream) == 0
    torch.cuda.synchronize()
    same = torch.equal(*out)
    assert same
