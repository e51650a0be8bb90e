"""Attention with capped scores, a bias by distance and a prefix, against its 64-bit form.

The bound is that of test_gpu_attention with the scores' part taken key by key: with
u = 2^-24 and key j's reach W_j = scale sk_j sum_d |q_d| (|ck_d| + 24), a score is off by
  products, two scales      (hd + 7) u W_j     (a cap's slope is at most 1)
  cap                       3 u |z_j| for its constants; then cap (1 - 2 r), r = 1 / (1 + e) <= 1, where e = 2^y,
                            1 + e and r are off by 2^-23, 2^-24 and 2^-23 relative:
                            2 r (r e 2^-23 + 3 2^-24) + u, r e <= 1 / 4 where r counts, in all
                            under 5 2^-23 cap <= 2^-20 cap; past caps of 2^8 the same relative
                            to tanh's value >= 0.29 where it is used, and 2^-22 below: 2^-19 |capped_j|
  bias                      the slope times log2 e and the multiply-add: 3 u slope |a - j| and u |s_j|
  s_j - max and its exp2    3 u (|s_j| + |max s|)
err_j their sum; p_j is off by err_j of itself (and second order, 1.01), numerator and
denominator: 1.01 (sum p_j err_j |v_j| + sum p_j err_j A).  The other terms, and their
derivation, are test_gpu_attention's."""
import numpy as np
import pytest
import torch

from gpu_helpers import banner, dev
from oracle import layer_oracle as L
from oracle import serving_oracle as S
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def G():
    import post_weight_quantization_07_amd as G
    assert torch.cuda.is_available()
    return G


def tolerance(one, cap, slope, hd, bits, top_scale):
    top = 127 if bits == 8 else 7
    p, s, vs = one["p"], one["s"], one["vs"]
    absv = np.abs(one["vc"]) * np.abs(vs)[:, None]
    A, B, seen = p @ absv, (p * vs).sum(), len(p)
    capping = 0.0 if cap is None else 3 * U * np.abs(one["z"]) + (2.0 ** -20 * cap if cap <= 256 else 2.0 ** -19 * np.abs(one["capped"]))
    err = ((hd + 7) * U * one["reach"] + capping + 3 * U * abs(slope) * one["away"]
           + U * np.abs(s) + 3 * U * (np.abs(s) + abs(s.max())))
    return (1.01 * ((p * err) @ absv + (p * err).sum() * A) + A * (3 * 2.0 ** -11 * (1 + 2.0 ** -9) + (seen + 64) * 4 * U)
            + (32 * B * (seen + 64) * 2 * U if bits == 4 else 0) + 2.0 ** -23 * top_scale * (1 + top * seen * p.max())
            + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(one["out"]))


def check(c, out, cap=None, slopes=None, prefixes=None, hidden=None):
    got = out.double().cpu().numpy()
    for i, (n, length) in enumerate(c.lens):
        pages = c.table[i, :-(-length // c.page)]
        a = int(c.starts[i])
        prefix = 0 if prefixes is None else min(max(int(prefixes[i]), 0), length)
        for h in range(c.heads):
            if length == 0:
                assert (got[a:a + n] == 0).all()
                continue
            k, v = (S.cache_rows(x, s, c.bits, pages, h // (c.heads // c.kv), length) for x, s in zip(c.codes, c.scales))
            slope = 0.0 if slopes is None else float(slopes[h])
            pick = np.arange(n) if n <= 24 else np.unique(np.r_[0:6, n // 2 - 3:n // 2 + 3, n - 6:n])
            for t in pick:
                one = L.attention(c.q_host[a + t, h], length - n + t, k, v, c.hd ** -0.5, cap, slope, prefix,
                                  None if hidden is None else hidden[i])
                if one is None:
                    assert (got[a + t, h] == 0).all(), (i, h, t)
                    continue
                tol = tolerance(one, cap, slope, c.hd, c.bits, v[1].max())
                off = np.abs(got[a + t, h] - one["out"])
                assert (off <= tol + 1e-30).all(), (i, h, t, float((off / (tol + 1e-30)).max()))


def _slopes(heads):
    s = np.exp2(-8.0 * np.arange(1, heads + 1) / heads).astype(np.float32)
    if heads > 2:
        s[1] = -0.01                                       # grows with the distance
    return s


def _prefixes(lens, seed):
    r = np.random.default_rng(seed)
    p = np.array([int(r.integers(0, length + 1)) for _, length in lens], np.int32)
    if len(p) > 1:
        p[0], p[-1] = 1 << 30, -5                          # clamped to the length and to none
    return p


def _call(G, c, cap, slopes, prefixes, **kw):
    d = lambda a: None if a is None else torch.from_numpy(a).to(dev())  # noqa: E731
    return G.gptq_cache_attention(c.q, c.cache, *c.args, cap=cap, slopes=d(slopes), prefix_lens=d(prefixes), **kw)


# lens: (new tokens, keys); heads, key heads, head_dim, page
CASES = [
    ([(1, 1)], 1, 1, 16, 16),
    ([(1, 2), (1, 15), (1, 17), (1, 33), (1, 64), (1, 65)], 4, 2, 64, 16),
    ([(1, 5000), (1, 3), (1, 700)], 8, 1, 128, 32),
    ([(1, 9000)], 16, 2, 128, 64),
    ([(1, 2100), (1, 0), (2, 1), (3, 3)], 6, 2, 96, 16),
    ([(5, 5), (1, 40), (17, 33), (0, 9), (40, 100)], 6, 3, 80, 32),
    ([(3, 515)], 12, 4, 256, 128),
    ([(17, 17), (20, 900)], 3, 1, 64, 16),
    ([(33, 2500), (31, 31), (2, 1)], 2, 1, 80, 16),
    ([(130, 130)], 2, 2, 128, 64),
    ([(200, 712), (65, 65), (128, 3000)], 8, 2, 64, 32),
    ([(257, 900), (3, 500)], 14, 2, 112, 128),
    ([(96, 96)], 3, 1, 256, 16),
    ([(200, 50), (150, 0), (130, 1), (129, 64)], 2, 1, 64, 16),
]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["cap", "slopes", "prefix", "cap slopes", "cap slopes prefix"])
@pytest.mark.parametrize("lens,heads,kv,hd,page", CASES)
def test_scores(G, lens, heads, kv, hd, page, kind, bits):
    banner(f"attention {kind} {lens} {heads}/{kv}x{hd} page {page} int{bits}")
    c = Case(G, lens, heads, kv, hd, page, bits, seed=21)
    cap = 5.0 if "cap" in kind else None
    slopes = _slopes(heads) if "slopes" in kind else None
    prefixes = _prefixes(lens, hd) if "prefix" in kind else None
    out = _call(G, c, cap, slopes, prefixes)
    check(c, out, cap, slopes, prefixes)
    assert torch.equal(out, _call(G, c, cap, slopes, prefixes))     # deterministic


@pytest.mark.parametrize("lens", [[(1, 700), (1, 90)], [(20, 400)], [(150, 500)]])
def test_caps_large_and_small(G, lens):
    """A cap that no score reaches, one that all reach, and scores next to 0 against a large cap."""
    banner(f"attention: caps at their limits {lens}")
    c = Case(G, lens, 4, 2, 64, 16, 8, seed=22)
    for cap in (2.0 ** 20, 1e4, 257.0, 256.0, 0.3, 2.0 ** -20):
        check(c, _call(G, c, cap, None, None), cap)


def test_nothing_set_is_the_plain_call(G):
    banner("attention: slopes of zero, prefixes of zero, no cap")
    for lens in ([(1, 700), (1, 90)], [(20, 400)], [(150, 500)]):
        c = Case(G, lens, 4, 2, 64, 16, 8, seed=23)
        plain = G.gptq_cache_attention(c.q, c.cache, *c.args)
        zero = _call(G, c, None, np.zeros(4, np.float32), np.zeros(len(lens), np.int32))
        c.check(zero)
        assert torch.equal(plain, G.gptq_cache_attention(c.q, c.cache, *c.args, cap=None))


@pytest.mark.parametrize("lens", [[(1, 700), (1, 90)], [(20, 400), (3, 50)], [(150, 500), (130, 130)]])
def test_bad_pages_in_the_prefix(G, lens):
    """A page entry outside the cache hides its keys, in the prefix too; a prefix that is all hidden leaves zeros."""
    banner(f"attention: bad pages under a prefix {lens}")
    c = Case(G, lens, 4, 2, 64, 16, 8, seed=24)
    table, starts, klen = c.args
    bad = table.clone()
    bad[0, 1], bad[1, 2] = -1, c.cache.n_pages
    prefixes = np.array([length - 1 for _, length in lens], np.int32)
    d = torch.from_numpy(prefixes).to(dev())
    out = G.gptq_cache_attention(c.q, c.cache, bad, starts, klen, cap=20.0, prefix_lens=d)
    hidden = [np.arange(length) // 16 == page for (_, length), page in zip(lens, (1, 2))]
    check(c, out, 20.0, None, prefixes, hidden)
    all_bad = torch.full_like(table, -1)
    assert not G.gptq_cache_attention(c.q, c.cache, all_bad, starts, klen, prefix_lens=d).any()


@pytest.mark.parametrize("lens", [[(6, 60), (1, 30)], [(80, 200)]])
def test_nan_scale_reaches_only_who_sees_it(G, lens):
    banner(f"attention: a key with a NaN scale behind a prefix {lens}")
    c = Case(G, lens, 2, 1, 64, 16, 8, seed=25)
    n, length = lens[0]
    key = length - 3
    c.cache.k_scales[int(c.table[0, key // 16]), 0, key % 16] = float("nan")
    for prefix in (length - 4, length):
        out = _call(G, c, 10.0, _slopes(2), np.array([prefix] + [0] * (len(lens) - 1), np.int32))
        nan = torch.isnan(out[:n]).flatten(1)
        if prefix == length:
            assert nan.all()
        else:
            assert nan[n - 3:].all() and not nan[:n - 3].any()
        assert not torch.isnan(out[n:]).any()


def test_rows_outside_are_left(G):
    banner("attention scores: rows outside the sequences, strided q and out")
    c = Case(G, [(3, 90), (1, 2000), (6, 6)], 4, 2, 64, 16, 8, seed=26)
    slopes, prefixes = _slopes(4), np.array([50, 7, 6], np.int32)
    want = _call(G, c, 30.0, slopes, prefixes)
    check(c, want, 30.0, slopes, prefixes)
    hold = torch.full((c.total + 4, 512), 7.0, dtype=torch.bfloat16, device=dev())
    out = hold[:, 256:].unflatten(1, (4, 64))
    q = torch.randn(c.total + 4, 4, 64, device=dev()).to(torch.bfloat16)
    q[2:-2] = c.q
    table, starts, klen = c.args
    d = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    G.gptq_cache_attention(q, c.cache, table, starts + 2, klen, out=out, cap=30.0, slopes=d(slopes), prefix_lens=d(prefixes))
    assert torch.equal(out[2:-2], want)
    assert (hold[:2] == 7).all() and (hold[-2:] == 7).all() and (hold[:, :256] == 7).all()


@pytest.mark.parametrize("lens", [[(1, 2500), (1, 90)], [(70, 70), (130, 600)]])
def test_stream_and_graph(G, lens):
    """Captured once, replayed with other queries, slopes and prefixes, eager work between."""
    banner(f"attention scores: another stream, a graph, {lens}")
    c = Case(G, lens, 8, 2, 128, 16, 8, seed=27)
    want = _call(G, c, 30.0, _slopes(8), _prefixes(lens, 1))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    d = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    sl, pr = d(_slopes(8)), d(_prefixes(lens, 1))
    torch.cuda.synchronize()
    got = G.gptq_cache_attention(c.q, c.cache, *c.args, cap=30.0, slopes=sl, prefix_lens=pr, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    q = c.q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gptq_cache_attention(q, c.cache, *c.args, out=out, cap=30.0, slopes=sl, prefix_lens=pr)
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=dev()))
        sl.copy_(d(_slopes(8) * (i + 1)))
        pr.copy_(d(_prefixes(lens, i)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, G.gptq_cache_attention(q, c.cache, *c.args, cap=30.0, slopes=sl, prefix_lens=pr))


def test_refusals(G):
    banner("attention scores: refusals")
    c = Case(G, [(2, 20)], 4, 2, 64, 16, 8)
    call = lambda **kw: G.gptq_cache_attention(c.q, c.cache, *c.args, **kw)  # noqa: E731
    slopes, prefixes = torch.zeros(4, device=dev()), torch.zeros(1, dtype=torch.int32, device=dev())
    for bad in (dict(cap=0.0), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=2.0 ** 21),
                dict(slopes=slopes[:2]), dict(slopes=slopes.double()), dict(slopes=slopes.cpu()), dict(prefix_lens=prefixes.long()),
                dict(prefix_lens=prefixes.expand(2)), dict(prefix_lens=prefixes.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    assert call(cap=1.0, slopes=slopes, prefix_lens=prefixes).shape == c.q.shape
