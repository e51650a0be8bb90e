"""A layer's bias on its way through a checkpoint: kept in the file, in the form that the integer products read, and in
what integer_apply, the gated product and a served block make of it."""
import numpy as np
import pytest
import torch


def _layer(d_out, d_in, seed, bias=True):
    """A layer of 8 bits with one group per output channel, as a solve returns it (codes by themselves)."""
    r = np.random.default_rng(seed)
    words = r.integers(-2 ** 31, 2 ** 31, (d_in // 4, d_out)).astype(np.int32)
    out = {"qweight": torch.from_numpy(words), "scales": torch.from_numpy(np.exp(r.standard_normal((1, d_out))).astype(np.float32) / 50),
           "zeros": torch.full((1, d_out), 128, dtype=torch.int32), "g_idx": torch.zeros(d_in, dtype=torch.int32)}
    if bias:
        out["bias"] = torch.from_numpy(r.standard_normal(d_out).astype(np.float32))
    return out


def _config():
    from post_weight_quantization_07_amd import QuantizeConfig
    return QuantizeConfig(bits=8, group_size=-1, desc_act=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_bias_round_trip(tmp_path, dtype):
    from post_weight_quantization_07_amd.checkpoint import load_quantized, save_quantized
    layers = {"a": _layer(40, 64, 1), "b": _layer(24, 64, 2, bias=False)}
    layers["a"]["bias"] = layers["a"]["bias"].to(dtype)
    save_quantized(str(tmp_path), layers, _config())
    _, got = load_quantized(str(tmp_path))
    assert got["a"]["bias"].dtype == dtype and torch.equal(got["a"]["bias"], layers["a"]["bias"])
    assert "bias" not in got["b"]


def test_bias_of_another_shape_is_refused(tmp_path):
    from post_weight_quantization_07_amd.checkpoint import save_quantized
    for bad in (torch.zeros(41), torch.zeros(1, 40), torch.zeros(40, dtype=torch.int32)):
        layer = _layer(40, 64, 1)
        layer["bias"] = bad
        with pytest.raises(ValueError, match="bias"):
            save_quantized(str(tmp_path), {"a": layer}, _config())


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 7, 100])
def test_bias_is_applied(tmp_path, m):
    import post_weight_quantization_07_amd as G
    from gpu_helpers import banner, dev
    from post_weight_quantization_07_amd.checkpoint import integer_apply, integer_layer, load_quantized, save_quantized
    banner(f"checkpoint with a bias, {m} tokens")
    save_quantized(str(tmp_path), {"a": _layer(72, 64, 1), "b": _layer(72, 64, 2, bias=False)}, _config())
    _, got = load_quantized(str(tmp_path))
    a, b = (integer_layer(got[n], 8, dev()) for n in ("a", "b"))
    assert a["bias"].dtype == torch.float32 and "bias" not in b
    x = torch.randn(m, 64, device=dev()).to(torch.bfloat16)
    call = lambda t, **kw: G.gptq_integer_matmul(x, t["w"], t["scales"], t.get("offsets"), **kw)  # noqa: E731
    assert torch.equal(integer_apply(x, a), call(a, bias=a["bias"])) and not torch.equal(integer_apply(x, a), call(a))
    assert torch.equal(integer_apply(x, b), call(b))
    assert torch.equal(integer_apply(x, a, bias=None), call(a))                      # what the call says goes first
    kw = dict(activation="silu", out_dtype=torch.bfloat16)
    assert torch.equal(integer_apply(x, a, **kw), call(a, bias=a["bias"], **kw))
    # one dict, one meaning.  Both take z + b, whose terms they may round apart (2^-22 of each), through a slope of at most
    # 1.1 and silu's own error on each side, (|z + b| + 4) 2^-23 of it; the products and stores add three roundings.
    gated = G.gptq_integer_gated(x, a, b).double()
    z, bias, up = call(a).double(), a["bias"].double(), integer_apply(x, b).double()
    act = integer_apply(x, a, activation="silu").double()
    off = 1.1 * 2.0 ** -22 * (z.abs() + bias.abs()) + ((z + bias).abs() + 4) * 2.0 ** -22 * act.abs()
    assert ((gated - act * up).abs() <= off * up.abs() + 2.0 ** -22 * (act * up).abs()).all()


@pytest.mark.gpu
def test_bias_of_another_shape_is_no_layer():
    from gpu_helpers import banner, dev
    from post_weight_quantization_07_amd.checkpoint import integer_layer
    banner("integer layer with a wrong bias")
    layer = _layer(40, 64, 1)
    layer["bias"] = torch.zeros(64)
    with pytest.raises(ValueError, match="bias"):
        integer_layer(layer, 8, dev())
