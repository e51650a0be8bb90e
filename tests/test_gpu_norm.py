"""The norm of tokens against its 64-bit form (oracle.layer_oracle).

h = x + residual and u = h weight are one fp32 rounding each, in the definition
too: total and codes have to be equal.  The factor s is rounded to fp32 once
(the squares are summed in 64 bits, whose roundings 2^-40 covers), s max|u| and its
division once each: a scale is off by (1 + 2^-24)^3 (1 + 2^-40) - 1 relative; so is y =
u s, u's own rounding the third, and by 2^-8 (1 + 2^-8) more in bf16."""
import numpy as np
import pytest
import torch

from gpu_helpers import banner, dev, host, to_dev
from oracle import layer_oracle as L

pytestmark = pytest.mark.gpu
R32 = (1 + 2.0 ** -24) ** 3 * (1 + 2.0 ** -40) - 1
REL = {torch.float32: R32, torch.bfloat16: (1 + R32) * (1 + 2.0 ** -8) - 1}
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def _rows(m, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = (r.standard_normal((m, d)) * np.exp(r.standard_normal(d))).astype(np.float32)
    if m > 3:
        x[1] = 0.0                        # a padded token
        x[2] = np.round(x[2] * 4) / 4     # many exact ties
    return to_dev(x, dtype)


def check_codes(rows, h, w, eps):
    codes, scales, sums = rows
    ref, sref = L.norm_codes(h, w, eps)
    np.testing.assert_array_equal(codes.cpu().numpy(), ref)
    np.testing.assert_array_equal(sums.cpu().numpy(), ref.sum(axis=1))
    got = scales.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(sref))
    fine = ~np.isnan(sref)
    assert (np.abs(got - sref)[fine] <= R32 * sref[fine]).all()


def check_y(y, h, w, eps):
    ref = L.norm(h, w, eps)
    assert (np.abs(y.double().cpu().numpy() - ref) <= REL[y.dtype] * np.abs(ref) + 2.0 ** -126).all()


def check_total(total, h, res):
    if res is not None:
        assert total.dtype == res.dtype
        assert torch.equal(total, torch.from_numpy(h).to(dev()).to(res.dtype))


SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (4, 129), (9, 2048), (2, 2056), (3, 4096), (5, 5120), (2, 8192), (2, 8200), (1, 16385),
         (2, 28672), (2, 32776), (1, 40000)]


@pytest.mark.parametrize("xt,rt,wt", [("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f32", "f32", "f32"),
                                      ("f32", "bf16", "bf16"), ("bf16", None, None), ("f32", None, "f32")])
@pytest.mark.parametrize("m,d", SIZES)
def test_norm(G, m, d, xt, rt, wt):
    banner(f"norm {m}x{d} x={xt} residual={rt} weight={wt}")
    x = _rows(m, d, xt, 7 * m + d)
    res = None if rt is None else _rows(m, d, rt, 5 * m + d)
    wh = (1 + 0.3 * np.random.default_rng(d).standard_normal(d)).astype(np.float32)
    w = None if wt is None else to_dev(wh, wt)
    h = L.added(host(x), None if res is None else host(res))
    whost = None if w is None else host(w)
    eps = 1e-5
    rows, total = G.gptq_norm_tokens(x, w, res, eps)
    check_codes(rows, h, whost, eps)
    check_total(total, h, res)
    if res is None:
        assert total is x
    for dtype in (torch.float32, torch.bfloat16):
        y, total = G.gptq_norm_tokens(x, w, res, eps, dtype=dtype)
        assert y.dtype == dtype
        check_y(y, h, whost, eps)
        check_total(total, h, res)


@pytest.mark.parametrize("d", [96, 5120, 40000])
def test_in_place_and_beside(G, d):
    """The total over the residual and over x, y beside the codes, for rows held and read twice."""
    banner(f"norm in place, d {d}")
    x, res, w = _rows(6, d, "f32", 1), _rows(6, d, "f32", 2), _rows(1, d, "f32", 3)[0]
    h = L.added(host(x), host(res))
    want, total = G.gptq_norm_tokens(x, w, res)
    for over in ("residual", "x"):
        a, b = x.clone(), res.clone()
        y = torch.empty(6, d, dtype=torch.bfloat16, device=dev())
        rows, t = G.gptq_norm_tokens(a, w, b, total=b if over == "residual" else a, y=y)
        assert t is (b if over == "residual" else a)
        assert torch.equal(t, total) and all(torch.equal(p, q) for p, q in zip(rows, want))
        check_y(y, h, host(w), 1e-6)


def test_strides_and_rows_around(G):
    banner("norm: strided x, residual and total; what lies around stays")
    wide = torch.randn(9, 400, device=dev())
    hold = torch.full((11, 300), 7.0, device=dev())
    res = torch.randn(9, 96, device=dev())
    for at in (0, 96, 131):                     # aligned, aligned, not aligned
        x = wide[:, at:at + 96]
        hold.fill_(7.0)
        rows, total = G.gptq_norm_tokens(x, None, res, total=hold[1:10, 100:196])
        h = L.added(host(x), host(res))
        check_codes(rows, h, None, 1e-6)
        assert torch.equal(hold[1:10, 100:196], torch.from_numpy(h).to(dev()))
        hold[1:10, 100:196] = 7.0
        assert (hold == 7.0).all()
    # one buffer for both: columns side by side do not touch
    both = torch.randn(9, 192, device=dev())
    h = L.added(host(both[:, :96]), host(res))
    _, total = G.gptq_norm_tokens(both[:, :96], None, res, total=both[:, 96:])
    assert torch.equal(both[:, 96:], torch.from_numpy(h).to(dev()))


@pytest.mark.parametrize("d", [96, 40000])
def test_extremes(G, d):
    banner(f"norm: tiny, huge, zero and not finite rows, d {d}")
    r = np.random.default_rng(3)
    x = r.standard_normal((9, d)).astype(np.float32)
    x[0] *= np.float32(2.0 ** -100)
    x[1] *= np.float32(2.0 ** -70)
    x[2] *= np.float32(2.0 ** 100)              # whose squares fp32 does not hold
    x[3] = 0.0
    x[4, 5] = np.nan
    x[5, d - 1] = np.inf
    x[6, 0] = -np.inf
    x[7] *= np.float32(2.0 ** 64)
    t = to_dev(x)
    for eps in (1e-6, 1e-30):
        rows, _ = G.gptq_norm_tokens(t, None, None, eps)
        check_codes(rows, x, None, eps)
        y, _ = G.gptq_norm_tokens(t, None, None, eps, dtype=torch.float32)
        keep = [0, 1, 2, 3, 7, 8]
        check_y(y[keep], x[keep], None, eps)
        assert torch.isnan(y[4]).all() and torch.isnan(y[5, d - 1]) and torch.isnan(y[6, 0])
    big = to_dev(np.full((1, d), 3e38, np.float32))
    rows, total = G.gptq_norm_tokens(big, None, big.clone())      # the sum leaves fp32
    assert torch.isinf(total).all() and torch.isnan(rows[1]).all() and not rows[0].any()


def test_products_take_the_codes(G):
    """What the norm returns is what a product in integers takes as x."""
    banner("norm into a product")
    x, w = _rows(20, 256, "bf16", 4), torch.randint(-127, 128, (70, 256), dtype=torch.int8, device=dev())
    s, off = torch.rand(70, device=dev()), torch.randint(-100, 100, (70,), dtype=torch.int32, device=dev())
    rows, _ = G.gptq_norm_tokens(x)
    y = G.gptq_integer_matmul(rows, w, s, off)
    n = rows[0].double() @ (w.double() - off.double()[:, None]).t()
    ref = n * rows[1].double()[:, None] * s.double()
    assert ((y.double() - ref).abs() <= ((1 + 2.0 ** -24) ** 3 - 1) * ref.abs()).all()


def test_stream_graph_and_empty(G):
    banner("norm: another stream, a graph, no tokens")
    x, res, w = _rows(33, 4096, "bf16", 5), _rows(33, 4096, "bf16", 6), _rows(1, 4096, "f32", 7)[0]
    want, total = G.gptq_norm_tokens(x, w, res)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, t = G.gptq_norm_tokens(x, w, res, stream=side)
    side.synchronize()
    assert torch.equal(t, total) and all(torch.equal(a, b) for a, b in zip(got, want))
    xs, rs = x.clone(), res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows, t = G.gptq_norm_tokens(xs, w, rs, total=rs)        # the hidden state in place
    for i in range(4):
        xs.copy_(_rows(33, 4096, "bf16", 50 + i))
        rs.copy_(_rows(33, 4096, "bf16", 60 + i))
        eager, et = G.gptq_norm_tokens(xs, w, rs)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rs, et) and all(torch.equal(a, b) for a, b in zip(rows, eager))
    rows, t = G.gptq_norm_tokens(x[:0], w, res[:0])
    assert rows[0].shape == (0, 4096) and rows[1].shape == (0,) and t.shape == (0, 4096)


def test_refusals(G):
    banner("norm: refusals")
    x, res, w = torch.randn(4, 64, device=dev()), torch.randn(4, 64, device=dev()), torch.randn(64, device=dev())
    call = G.gptq_norm_tokens
    for bad in (lambda: call(x.half()), lambda: call(x.t()), lambda: call(x[0]), lambda: call(x, w[:32]), lambda: call(x, w.cpu()),
                lambda: call(x, w, res[:3]), lambda: call(x, w, res.double()), lambda: call(x, w, None, total=res),
                lambda: call(x, w, res, total=res.to(torch.bfloat16)), lambda: call(x, w, res, dtype=torch.float16),
                lambda: call(x, w, res, y=torch.empty(4, 32, device=dev())),
                lambda: call(x, w, res, dtype=torch.bfloat16, y=torch.empty(4, 64, device=dev()))):
        with pytest.raises(ValueError):
            bad()
    wide = torch.randn(4, 100, device=dev())
    for bad in (lambda: call(x, w, eps=0.0), lambda: call(x, w, eps=float("nan")), lambda: call(x, w, y=x),
                lambda: call(wide[:, :64], w, res, total=wide[:, 32:96]),        # over half of x
                lambda: call(x[:3], w, x[1:], total=x[1:])):                     # the residual's rows are x's, moved by one
        with pytest.raises(G.GptqError):
            bad()
    rows, total = call(x[:3], w, x[1:])                                          # read only: they may share rows
    check_total(total, L.added(host(x[:3]), host(x[1:])), x)
