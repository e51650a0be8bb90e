"""The product in 8-bit integers against its plain form (oracle.serving_oracle).

Codes, scales and sums have to be equal: the code is the exact quotient's, and
the scale one correctly rounded division.  The product's sums are exact
integers, so y differs from the fp64 value only by the rounding of the sum to
fp32, of the two scales' products, and to y's type: relative
(1 + 2^-24)^3 - 1, and (1 + 2^-24)^3 (1 + 2^-8) - 1 for bf16."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import banner, dev, host, to_dev
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu
REL = {torch.float32: (1 + 2.0 ** -24) ** 3 - 1, torch.bfloat16: (1 + 2.0 ** -24) ** 3 * (1 + 2.0 ** -8) - 1}


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def _x(m, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = (r.standard_normal((m, d)) * np.exp(r.standard_normal(d))).astype(np.float32)
    if m > 2:
        x[1] = 0.0                                        # a padded token
        x[2] = np.round(x[2] * 4) / 4                     # many exact ties
    return to_dev(x, dtype)


def _layer(d_out, d_in, seed, asym):
    r = np.random.default_rng(seed)
    w = r.integers(-128 if asym else -127, 128, (d_out, d_in)).astype(np.int8)
    s = (0.001 * np.exp(r.standard_normal(d_out))).astype(np.float32)
    off = r.integers(-128, 129, d_out).astype(np.int32) if asym else np.zeros(d_out, np.int32)
    return w, s, off


def _d(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(1, 1), (3, 7), (5, 64), (4, 129), (3, 2048), (2, 2056), (3, 4096), (2, 8192), (2, 8200),
                                 (2, 28672), (1, 40000)])
def test_codes(G, m, d, dtype):
    banner(f"token codes {m}x{d} {dtype}")
    x = _x(m, d, dtype, m * 7 + d)
    codes, scales, sums = G.gptq_quantize_tokens(x)
    ref, sref = S.row_codes(host(x), 127)
    np.testing.assert_array_equal(codes.cpu().numpy(), ref)
    np.testing.assert_array_equal(scales.cpu().numpy(), sref)
    np.testing.assert_array_equal(sums.cpu().numpy(), ref.sum(axis=1))


def test_codes_extremes_and_strides(G):
    banner("token codes: subnormal, huge, NaN and infinite rows; strided rows")
    r = np.random.default_rng(3)
    x = r.standard_normal((8, 96)).astype(np.float32)
    x[0] *= np.float32(2.0 ** -140)
    x[1] *= np.float32(2.0 ** -120)
    x[2] *= np.float32(2.0 ** 124)
    x[3, 5] = np.nan
    x[4, 95] = np.inf
    x[5, 0] = -np.inf
    x[6] *= np.float32(2.0 ** -61)
    for dtype in ("f32", "bf16"):
        t = to_dev(x, dtype) if dtype == "f32" else to_dev(x, "f32").to(torch.bfloat16)
        codes, scales, _ = G.gptq_quantize_tokens(t)
        ref, sref = S.row_codes(t.float().cpu().numpy(), 127)
        np.testing.assert_array_equal(codes.cpu().numpy(), ref)
        np.testing.assert_array_equal(scales.cpu().numpy(), sref)
    wide = torch.randn(6, 200, device=dev())
    for view in (wide[:, :96], wide[:, 8:72], wide[:, 3:100]):     # aligned, aligned, odd start
        codes, _, _ = G.gptq_quantize_tokens(view)
        np.testing.assert_array_equal(codes.cpu().numpy(), S.row_codes(view.cpu().numpy(), 127)[0])
    codes, scales, sums = G.gptq_quantize_tokens(wide[:0])
    assert codes.shape == (0, 200) and scales.shape == (0,) and sums.shape == (0,)


@pytest.mark.parametrize("bits,sym", [(8, True), (8, False), (4, False), (3, True), (2, False)])
def test_layer_layout(G, bits, sym):
    banner(f"integer weight, {bits} bits")
    d_out, d_in = 77, 224
    t = synth.quantized_layer(d_out, d_in, bits, -1, False, seed=bits)
    zeros = np.full((1, d_out), 2 ** (bits - 1), np.int32) if sym else t["zeros"]
    w, off = G.gptq_integer_weight(_d(t["qweight"]), _d(zeros), bits)
    import oracle as O
    codes = O.unpack(t["qweight"], bits, d_in)
    np.testing.assert_array_equal(w.cpu().numpy(), codes - 2 ** (bits - 1))
    np.testing.assert_array_equal(off.cpu().numpy(), zeros[0] - 2 ** (bits - 1))


SHAPES = [(1, 32, 1), (1, 96, 17), (1, 4096, 300), (2, 160, 33), (15, 4096, 64), (16, 224, 48), (17, 1024, 100),
          (31, 352, 257), (33, 2048, 130), (64, 4096, 272), (65, 32, 500), (100, 4128, 260), (128, 768, 768),
          (129, 288, 511), (200, 11008, 70), (257, 1056, 300), (300, 96, 1030), (513, 4096, 520), (4100, 96, 4200),
          (2049, 352, 8300)]


@pytest.mark.parametrize("m,d_in,d_out", SHAPES)
@pytest.mark.parametrize("asym,xt,yt", [(False, "bf16", torch.bfloat16), (True, "f32", torch.float32)])
def test_product(G, m, d_in, d_out, asym, xt, yt):
    banner(f"integer product {m}x{d_in}->{d_out} asym={asym} x={xt}")
    x = _x(m, d_in, xt, m + d_in)
    w, s, off = _layer(d_out, d_in, d_out + d_in, asym)
    codes, scales = S.row_codes(host(x), 127)
    ref = S.integer_matmul(codes, scales, w, s, off)
    dw, ds, doff = _d(w), _d(s), _d(off) if asym else None
    y = G.gptq_integer_matmul(x, dw, ds, doff, out_dtype=yt)
    two = G.gptq_integer_matmul(G.gptq_quantize_tokens(x), dw, ds, doff, out_dtype=yt)
    assert y.dtype == yt and torch.equal(y, two)          # quantized inside or before: the same
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= REL[yt] * np.abs(ref) + 2.0 ** -149).all(), float((err / (np.abs(ref) + 1e-30)).max())


def test_largest_sums(G):
    """d_in at its limit with every product at its largest: sums near 2^30, the offset term as large."""
    banner("integer product at d_in 65536, extreme codes")
    d = 65536
    x = torch.ones(20, d, device=dev())
    x[1::2] = -1.0
    w = torch.full((40, d), -128, dtype=torch.int8, device=dev())
    w[1::2] = 127
    off = torch.full((40,), 128, dtype=torch.int32, device=dev())
    off[2::4] = -128
    s = torch.ones(40, device=dev())
    y = G.gptq_integer_matmul(x, w, s, off).double().cpu().numpy()
    sign = np.where(np.arange(20) % 2, -1.0, 1.0)
    wv, ov = w[:, 0].double().cpu().numpy(), off.double().cpu().numpy()
    ref = sign[:, None] * (127.0 * d * (wv - ov))[None, :] * np.float64(np.float32(1 / 127))
    assert (np.abs(y - ref) <= REL[torch.float32] * np.abs(ref)).all()
    with pytest.raises(G.GptqError):
        G.gptq_integer_matmul(torch.ones(1, d + 32, device=dev()), torch.zeros((8, d + 32), dtype=torch.int8, device=dev()),
                              torch.ones(8, device=dev()))


def test_nan_rows_and_strides(G):
    banner("integer product: a NaN row, strided x, no tokens, a given y and workspace")
    x = torch.randn(40, 320, device=dev()).to(torch.bfloat16)
    x[7, 3] = float("nan")
    w, s, _ = _layer(90, 256, 1, False)
    dw, ds = _d(w), _d(s)
    view = x[:, 32:288]
    assert not torch.isnan(G.gptq_integer_matmul(view, dw, ds)).any()       # column 3 lies before the view
    x[7, 40] = float("nan")
    y = G.gptq_integer_matmul(view, dw, ds)
    assert torch.isnan(y[7]).all() and not torch.isnan(y[torch.arange(40) != 7]).any()
    assert torch.equal(y[:7], G.gptq_integer_matmul(view[:7].contiguous(), dw, ds))
    assert G.gptq_integer_matmul(view[:0], dw, ds).shape == (0, 90)
    out = torch.full((40, 90), 7.0, device=dev())
    ws = torch.empty(G.gptq_integer_workspace_size(40, torch.bfloat16, 256, 90), dtype=torch.uint8, device=dev())
    G.gptq_integer_matmul(view, dw, ds, y=out, ws=ws)
    torch.testing.assert_close(out, y, rtol=0, atol=0, equal_nan=True)
    for bad in (lambda: G.gptq_integer_matmul(view, dw[:, :128], ds), lambda: G.gptq_integer_matmul(view.double(), dw, ds),
                lambda: G.gptq_integer_matmul(view, dw, ds.cpu()), lambda: G.gptq_integer_matmul(view, dw, ds[:5]),
                lambda: G.gptq_integer_matmul(view, dw, ds, out_dtype=torch.float16),
                lambda: G.gptq_quantize_tokens(x.t())):
        with pytest.raises(ValueError):
            bad()


def test_stream_and_graph(G):
    banner("integer product on another stream and in a graph, replayed with new inputs")
    w, s, off = _layer(300, 512, 5, True)
    dw, ds, doff = _d(w), _d(s), _d(off)
    for m in (1, 24, 150):
        xs = [torch.randn(m, 512, device=dev()).to(torch.bfloat16) for _ in range(3)]
        want = [G.gptq_integer_matmul(x, dw, ds, doff) for x in xs]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = G.gptq_integer_matmul(xs[0], dw, ds, doff, stream=side)
        side.synchronize()
        assert torch.equal(got, want[0])
        hold = xs[0].clone()
        y = torch.empty(m, 300, device=dev())
        ws = torch.empty(G.gptq_integer_workspace_size(m, torch.bfloat16, 512, 300), dtype=torch.uint8, device=dev())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            G.gptq_integer_matmul(hold, dw, ds, doff, y=y, ws=ws)
        for i in (1, 2, 0, 1):
            hold.copy_(xs[i])
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
            G.gptq_integer_matmul(xs[i], dw, ds, doff)      # eager work between the replays


@pytest.mark.parametrize("m,d_in,d_out,asym", [(5, 4096, 16401, True), (16, 8192, 16384, False), (16, 288, 20000, True),
                                               (1, 32, 65536, False), (13, 11008, 16400, True)])
def test_many_channels(G, m, d_in, d_out, asym):
    """Few tokens, codes given, through more row blocks than the card has CUs."""
    banner(f"integer product {m}x{d_in}->{d_out}")
    w, s, off = _layer(d_out, d_in, d_in, asym)
    x = _x(m, d_in, "bf16", m)
    xq = G.gptq_quantize_tokens(x)
    codes, sx = S.row_codes(host(x), 127)
    ref = S.integer_matmul(codes, sx, w, s, off)
    for dtype in (torch.float32, torch.bfloat16):
        y = host(G.gptq_integer_matmul(xq, _d(w), _d(s), _d(off) if asym else None, out_dtype=dtype)).astype(np.float64)
        assert np.all(np.abs(y - ref) <= REL[dtype] * np.abs(ref))


def test_more_rows_than_one_launch(G):
    banner("token codes of 2^21 + 5 rows")
    r = np.random.default_rng(3)
    x = to_dev(r.standard_normal((2 ** 21 + 5, 8)).astype(np.float32), "bf16")
    codes, scales, sums = G.gptq_quantize_tokens(x)
    rows = np.r_[0:40, 2 ** 20:2 ** 20 + 40, 2 ** 21 - 40:2 ** 21 + 5]
    ref, sref = S.row_codes(host(x[rows]), 127)
    np.testing.assert_array_equal(codes[rows].cpu().numpy(), ref)
    np.testing.assert_array_equal(scales[rows].cpu().numpy(), sref)
    np.testing.assert_array_equal(sums[rows].cpu().numpy(), ref.sum(axis=1))


def test_expanded_rows_are_refused(G):
    """Rows that overlap have no row stride the kernels can use."""
    banner("integer product: expanded rows")
    x = torch.randn(1, 64, device=dev()).to(torch.bfloat16)
    w, s = torch.ones(8, 64, dtype=torch.int8, device=dev()), torch.ones(8, device=dev())
    for m in (3, 80):
        with pytest.raises(G.GptqError):
            G.gptq_quantize_tokens(x.expand(m, 64))
        with pytest.raises(G.GptqError):
            G.gptq_integer_matmul(x.expand(m, 64), w, s)
    wide = torch.randn(1, 200, device=dev()).to(torch.bfloat16)[:, 8:72]        # one row of a wider matrix is fine
    assert torch.equal(G.gptq_integer_matmul(wide, w, s), G.gptq_integer_matmul(wide.contiguous(), w, s))


@pytest.mark.parametrize("m,d_in,d_out", [(515, 1056, 2049), (1030, 8224, 1800), (1030, 16384, 1800), (140, 4096, 1000),
                                        (70, 32768, 50)])
@pytest.mark.parametrize("asym,xt,yt", [(True, "bf16", torch.float32), (False, "f32", torch.bfloat16)])
def test_tiles(G, m, d_in, d_out, asym, xt, yt):
    """Tiles of both sizes, with K slices and without, at sizes that end inside a tile."""
    test_product(G, m, d_in, d_out, asym, xt, yt)


def test_graph_with_slices(G):
    banner("integer product in K slices, replayed with new inputs")
    w, s, off = _layer(300, 4128, 6, True)
    dw, ds, doff = _d(w), _d(s), _d(off)
    xs = [torch.randn(150, 4128, device=dev()).to(torch.bfloat16) for _ in range(3)]
    want = [G.gptq_integer_matmul(x, dw, ds, doff) for x in xs]
    hold, graph = xs[0].clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = G.gptq_integer_matmul(hold, dw, ds, doff)
    for i in (1, 2, 0, 1):
        hold.copy_(xs[i])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        G.gptq_integer_matmul(xs[i], dw, ds, doff)          # eager work between the replays
