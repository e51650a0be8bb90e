"""What the calls take besides the usual tensors: workspaces of any dtype (and
only whole ones), tensors of one head whose head stride says nothing."""
import pytest
import torch

from gpu_helpers import banner, dev
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def whole_and_views(nbytes):
    """A float32 workspace of nbytes, and two views that are not in one piece but count as many elements."""
    n = -(-nbytes // 4)
    return (torch.empty(n, device=dev()), torch.empty(2 * nbytes, dtype=torch.uint8, device=dev())[::2],
            torch.empty(1, dtype=torch.uint8, device=dev()).expand(nbytes))


def test_workspaces(G):
    banner("workspaces: float32 ones count in bytes, views are refused")
    x = torch.randn(40, 256, device=dev()).to(torch.bfloat16)
    w = torch.randint(-127, 128, (90, 256), dtype=torch.int8, device=dev())
    s = torch.rand(90, device=dev())
    c = Case(G, [(1, 3000)], 4, 2, 64, 16, 8)
    cfg = G.QuantizeConfig(bits=4, group_size=128)
    S = torch.eye(256, device=dev()) * 100
    U, perm, _ = G.gptq_prepare_hinv(S.clone(), 100, cfg)
    W = torch.randn(64, 256, device=dev())
    solved = G.gptq_quantize_layer(W, U, perm, cfg)
    layer = (G.gptq_pack(solved["codes"], 4), solved["scales"], solved["zeros"], solved["g_idx"])
    q_sorted, g_sorted, order = G.gptq_dequant_order(layer[0], layer[3], 4)
    calls = [
        (G.gptq_integer_workspace_size(40, torch.bfloat16, 256, 90), lambda ws: G.gptq_integer_matmul(x, w, s, ws=ws)),
        (G.gptq_attention_workspace_size(c.cache, 1, 4, 1, c.args[0].shape[1]),
         lambda ws: G.gptq_cache_attention(c.q, c.cache, *c.args, ws=ws)),
        (G.gptq_hessian_workspace_size(256, 40, torch.bfloat16),
         lambda ws: G.gptq_hessian_accumulate(torch.zeros(256, 256, device=dev()), x, ws=ws)),
        (G.gptq_prepare_workspace_size(256), lambda ws: G.gptq_prepare_hinv(S.clone(), 100, cfg, ws=ws)[0]),
        (G.gptq_workspace_size(64, 256, cfg), lambda ws: G.gptq_quantize_layer(W, U, perm, cfg, ws=ws)["codes"]),
        (G.gptq_dequant_workspace_size(40, 256, 64), lambda ws: G.gptq_dequant_matmul(x, *layer, 4, ws=ws)),
        (G.gptq_dequant_ordered_workspace_size(40, 256, 64),
         lambda ws: G.gptq_dequant_matmul_ordered(x, q_sorted, layer[1], layer[2], g_sorted, order, 4, ws=ws)),
    ]
    for need, call in calls:
        want = call(None)
        whole, *views = whole_and_views(max(need, 256))
        assert torch.equal(call(whole), want)
        for view in views:
            with pytest.raises(ValueError, match="contiguous"):
                call(view)
