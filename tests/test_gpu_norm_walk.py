"""The norm where a workgroup walks over several rows: the next row's values are on their way while one is
reduced, two LDS buffers are used by turns, and a row's code sum is stored with the next row.  Rows are dense and all
different, and every row's codes, scale, sum and total are compared: with the 64-bit form, and bit for bit with the same
rows normed a few at a time, which no workgroup walks over (bounds: test_gpu_norm)."""
import pytest
import torch

from gpu_helpers import banner, dev, host
from oracle import layer_oracle as L
from test_gpu_norm import REL, R32, check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def _walks(d):
    """Rows of a call that gives workgroups three of them, and some two: of one wave for each row up to 1024 values (four
    rows a workgroup), of a whole workgroup past that."""
    room = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * (4 if d <= 1024 else 1) * room + 5


def _rows(m, d, dtype, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(m, d, generator=g, device=dev()) * torch.exp(torch.randn(d, generator=g, device=dev()))
    return (x * torch.linspace(0.5, 3.0, m, device=dev())[:, None]).to(dtype)     # rows of different scales


# (rows past 8192 values go without the next one ahead)
DIMS = [40, 512, 600, 1000, 1001, 2000, 2044, 4096, 5004, 5120, 8192, 12000, 12004]
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("xt,rt", [(BF, BF), (F32, F32), (BF, F32), (BF, None), (F32, None)])
def test_walk(G, d, xt, rt):
    m = _walks(d)
    banner(f"norm walk {m}x{d} x={xt} residual={rt}")
    x, w = _rows(m, d, xt, d), _rows(1, d, F32, 3)[0]
    res = None if rt is None else _rows(m, d, rt, d + 1)
    y = torch.empty(m, d, dtype=BF, device=dev())
    (codes, scales, sums), total = G.gptq_norm_tokens(x, w, res, 1e-5, y=y)
    # the same rows, a few in each call
    part = 512
    for a in range(0, m, part):
        b = min(a + part, m)
        ys = torch.empty(b - a, d, dtype=BF, device=dev())
        one, t = G.gptq_norm_tokens(x[a:b], w, None if res is None else res[a:b], 1e-5, y=ys)
        for got, want in zip((codes, scales, sums, total, y), (*one, t, ys)):
            assert torch.equal(got[a:b], want), (a, b)
    # and all of them against the definition
    h = x.float() if res is None else x.float() + res.float()
    if res is not None:
        assert torch.equal(total, h.to(rt))
    h64, u64 = h.double(), (h * w).double()
    factor = torch.rsqrt((h64 ** 2).mean(dim=1) + float(torch.tensor(1e-5, dtype=F32)))
    ref = factor * u64.abs().amax(dim=1) / 127
    assert ((scales.double() - ref).abs() <= R32 * ref).all()
    assert torch.equal(sums, codes.sum(dim=1, dtype=torch.int32))
    off = (127 * u64 / u64.abs().amax(dim=1, keepdim=True) - codes).abs()         # no further than the nearest integer
    assert off.max() <= 0.5 * (1 + 2.0 ** -40)
    ref = factor[:, None] * h64 * w.double()
    assert ((y.double() - ref).abs() <= REL[BF] * ref.abs() + 2.0 ** -126).all()
    for rows in (slice(0, 3), slice(m - 9, m)):                                    # ties to even too
        check_codes((codes[rows], scales[rows], sums[rows]), host(h[rows]), host(w), 1e-5)


@pytest.mark.parametrize("d", [512, 1001, 4096, 5120, 8192, 12004])
@pytest.mark.parametrize("over", ["residual", "x"])
def test_walk_in_place(G, d, over):
    """The total over what the next rows are read from."""
    m = _walks(d)
    banner(f"norm walk in place {m}x{d} over {over}")
    x, res, w = _rows(m, d, BF, d), _rows(m, d, BF, d + 1), _rows(1, d, BF, 3)[0]
    want, total = G.gptq_norm_tokens(x, w, res)
    assert torch.equal(total, (x.float() + res.float()).to(BF))
    for _ in range(2):
        a, b = x.clone(), res.clone()
        rows, t = G.gptq_norm_tokens(a, w, b, total=b if over == "residual" else a)
        assert torch.equal(t, total) and all(torch.equal(p, q) for p, q in zip(rows, want))
        assert torch.equal(a, total if over == "x" else x) and torch.equal(b, total if over == "residual" else res)


def test_walk_from_strided_rows(G):
    """x, the residual and the total as columns of wider matrices, several rows a workgroup."""
    d, m = 1000, _walks(1000)
    banner(f"norm walk {m}x{d}, strided")
    wide, keep = _rows(m, 2300, BF, 1), _rows(m, 1100, F32, 2)
    x, res = wide[:, 3:3 + d], wide[:, 1201:1201 + d]
    whole, total = G.gptq_norm_tokens(x.contiguous(), None, res.contiguous())
    around = wide.clone()
    rows, t = G.gptq_norm_tokens(x, None, res, total=x)
    assert all(torch.equal(p, q) for p, q in zip(rows, whole)) and torch.equal(t, total)
    around[:, 3:3 + d] = total
    assert torch.equal(wide, around)
    h = keep[:, 50:50 + d]
    rows, _ = G.gptq_norm_tokens(h)
    assert all(torch.equal(p, q) for p, q in zip(rows, G.gptq_norm_tokens(h.contiguous())[0]))
