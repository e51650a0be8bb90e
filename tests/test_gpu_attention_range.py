"""Attention over the quantized cache where scores or value scales lie far apart.

The bound, per output element, in the terms of test_gpu_attention.py (u = 2^-24,
h = 2^-11, L keys seen, c the largest code, A = sum p |v|, B = sum p sv,
W the scores' magnitude), with X = max over seen keys of p sv:
  scores  2 (hd + 7) u W
  fp16    weight (numerator and, where it is of the rounded weights, denominator),
          value factor and value: h relative each, 4 h (1 + 2^-9) A.  What fp16
          loses below its normal range is under 2^-24 c X a key
  sums    (L + 64) 4 u of A; at 4 bits the values enter as 24 + code: another
          (L + 64) 2 u of 32 B
  output  bf16: 2^-8 of the value, and half its least subnormal
"""
import numpy as np
import pytest
import torch

from gpu_helpers import banner, dev
from oracle import serving_oracle as S
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def bound(ref, A, B, W, X, seen, hd, bits):
    top = 127 if bits == 8 else 7
    return (A * (4 * 2.0 ** -11 * (1 + 2.0 ** -9) + 2 * (hd + 7) * U * W + (seen + 64) * 4 * U)
            + (32 * B * (seen + 64) * 2 * U if bits == 4 else 0) + seen * top * U * X
            + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(ref) + 2.0 ** -134)


def largest_product(q, k, v, scale):
    s = scale * (k[0] @ q) * k[1]
    p = np.exp(s - s.max())
    return (p / p.sum() * v[1]).max()


def upload(G, c):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    c.cache = G.QuantizedCache(*[d(x) for x in c.codes], *[d(x) for x in c.scales], c.bits)


def check(c, out, same_scores=False, last=0):
    """same_scores: the caller made all scores equal, so that q counts as zero.  The `last` tokens of a sequence
    are not looked at."""
    scale = c.hd ** -0.5
    got = out.double().cpu().numpy()
    for i, (n, length) in enumerate(c.lens):
        pages, a = c.table[i, :-(-length // c.page)], int(c.starts[i])
        for h in range(c.heads):
            k, v = (S.cache_rows(x, s, c.bits, pages, h // (c.heads // c.kv), length) for x, s in zip(c.codes, c.scales))
            if same_scores:
                k = (k[0], np.ones_like(k[1]))
            for t in (np.arange(n) if n <= 24 else np.unique(np.r_[0:4, 30:34, n // 2:n // 2 + 3, n - 4:n])):
                if t >= n - last:
                    continue
                seen = length - n + t + 1
                q = c.q_host[a + t, h] * (0.0 if same_scores else 1.0)
                k1, v1 = (k[0][:seen], k[1][:seen]), (v[0][:seen], v[1][:seen])
                ref, A, B, W, _ = S.attention(q[None], k1, v1, scale)
                tol = bound(ref, A, B, W[0], largest_product(q, k1, v1, scale), seen, c.hd, c.bits)
                err = np.abs(got[a + t, h] - ref[0])
                assert (err <= tol[0]).all(), (i, h, int(t), float((err / tol[0]).max()), float(np.abs(ref).max()))


# one kernel each: keys split over waves with one and two row blocks, its parts joined,
# wide heads, rows split over waves, its parts joined, wide heads
SHAPES = [([(1, 300)], 4, 2, 64, 16), ([(20, 300)], 2, 1, 64, 16), ([(1, 3000)], 2, 1, 128, 32), ([(9, 200)], 2, 1, 144, 16),
          ([(130, 500)], 2, 1, 128, 64), ([(70, 3000)], 2, 1, 64, 16), ([(96, 300)], 1, 1, 256, 16)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens,heads,kv,hd,page", SHAPES)
def test_scores_far_below_zero(G, lens, heads, kv, hd, page, bits):
    """Scores near -10^32, all the same: the mean of the values seen."""
    banner(f"attention: scores near -1e32, {lens} {heads}/{kv}x{hd} int{bits}")
    c = Case(G, lens, heads, kv, hd, page, bits, seed=21)
    top = 127 if bits == 8 else 7
    c.codes[0] = S.pack_rows(np.full((*c.scales[0].shape, hd), -top), bits)
    c.scales[0] = np.where(np.isnan(c.scales[0]), np.nan, 1e32 * hd ** 0.5 / (2.0 * top * hd)).astype(np.float32)
    upload(G, c)
    c.q.fill_(2.0)
    c.q_host[:] = 2.0
    check(c, G.gptq_cache_attention(c.q, c.cache, *c.args), same_scores=True)


def plant(c, key, score, ratio):
    """Key `key` of every sequence scores `score` for every query, and its value scale is `ratio` times what it was."""
    top = 127 if c.bits == 8 else 7
    c.q[..., 0] = 8.0
    c.q_host[..., 0] = 8.0
    row = np.zeros(c.hd, np.int64)
    row[0] = top if score > 0 else -top
    for i, (_, length) in enumerate(c.lens):
        page, at = c.table[i, key % length // c.page], key % length % c.page
        c.codes[0][page, :, at] = S.pack_rows(row, c.bits)
        c.scales[0][page, :, at] = abs(score) / (c.hd ** -0.5 * 8.0 * top)
        c.scales[1][page, :, at] *= ratio


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens,heads,kv,hd,page", SHAPES)
def test_large_values_of_little_weight(G, lens, heads, kv, hd, page, bits):
    """One key of weight near e^-60 whose value scale is 2^r times the others': nothing of it shows up to r near 80."""
    for r in (9, 13, 17, 20, 27, 45, 100):
        for key in (0, 150, -1):
            banner(f"attention: value scale 2^{r} at key {key}, {lens} {heads}/{kv}x{hd} int{bits}")
            c = Case(G, lens, heads, kv, hd, page, bits, seed=22)
            plant(c, key, -60.0, 2.0 ** r)
            upload(G, c)
            check(c, G.gptq_cache_attention(c.q, c.cache, *c.args))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens,heads,kv,hd,page", SHAPES)
def test_small_values_of_all_weight(G, lens, heads, kv, hd, page, bits):
    """One key that takes all the weight and has a small value, or none: the others' share shows."""
    for ratio in (0.0, 2.0 ** -10, 2.0 ** -30, 2.0 ** -60):
        for key in (0, 150):
            banner(f"attention: value scale x {ratio} at key {key}, {lens} {heads}/{kv}x{hd} int{bits}")
            c = Case(G, lens, heads, kv, hd, page, bits, seed=23)
            plant(c, key, 40.0, ratio)
            upload(G, c)
            check(c, G.gptq_cache_attention(c.q, c.cache, *c.args))


@pytest.mark.parametrize("bits", [8, 4])
def test_values_of_every_size(G, bits):
    """Value scales over forty powers of two, in falling and rising order and mixed; some of them zero."""
    for lens, heads, kv, hd, page in SHAPES:
        for how in ("fall", "rise", "mix"):
            banner(f"attention: value scales that {how}, {lens} {heads}/{kv}x{hd} int{bits}")
            c = Case(G, lens, heads, kv, hd, page, bits, seed=24)
            r = np.random.default_rng(5)
            length = lens[0][1]
            power = {"fall": np.linspace(20, -20, length), "rise": np.linspace(-20, 20, length),
                     "mix": r.uniform(-20, 20, length)}[how]
            for j in range(length):
                c.scales[1][c.table[0, j // page], :, j % page] *= 0.0 if j % 7 == 3 else np.float32(2.0 ** power[j])
            upload(G, c)
            check(c, G.gptq_cache_attention(c.q, c.cache, *c.args))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens,heads,kv,hd,page", SHAPES)
def test_values_near_the_largest(G, lens, heads, kv, hd, page, bits):
    """Values up to 1.5e38: their mean is finite, their sum is not."""
    banner(f"attention: values near the largest, {lens} {heads}/{kv}x{hd} int{bits}")
    c = Case(G, lens, heads, kv, hd, page, bits, seed=25)
    top = 127 if bits == 8 else 7
    c.codes[1] = S.pack_rows(np.full((*c.scales[1].shape, hd), top), bits)
    c.scales[1] = np.where(np.isnan(c.scales[1]), np.nan, 2.0 ** (120 if bits == 8 else 124)).astype(np.float32)
    upload(G, c)
    out = G.gptq_cache_attention(c.q, c.cache, *c.args)
    assert torch.isfinite(out).all()
    check(c, out)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("lens,heads,kv,hd,page", [x for x in SHAPES if x[0][0][0] > 2])
def test_scales_that_are_not_finite(G, lens, heads, kv, hd, page, zeros, bits):
    """A key or value scale of NaN makes the tokens that see it NaN, and no others; also among values some of which
    are zero.  An infinite value scale holds infinities, and NaN for codes of 0, so what sees it is not finite; an
    infinite key scale gives NaN or the value of a key with all the weight."""
    n, length = lens[0]
    for which in (0, 1):
        for bad in (np.nan, np.inf):
            banner(f"attention: {'kv'[which]} scale {bad}, zeros {zeros}, {lens} {heads}/{kv}x{hd} int{bits}")
            c = Case(G, lens, heads, kv, hd, page, bits, seed=26)
            if zeros:
                for j in range(0, length, 5):
                    c.scales[1][c.table[0, j // page], :, j % page] = 0.0
            key = length - 2                              # the last two tokens see it
            c.scales[which][c.table[0, key // page], :, key % page] = bad
            upload(G, c)
            out = G.gptq_cache_attention(c.q, c.cache, *c.args)
            if np.isnan(bad):
                assert torch.isnan(out[-2:]).all()
            elif which == 1:
                assert not torch.isfinite(out[-2:]).any()
            assert torch.isfinite(out[:-2]).all()
            c.scales[which][c.table[0, key // page], :, key % page] = 1.0      # hidden from the tokens that are checked
            check(c, out, last=2)
