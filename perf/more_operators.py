"""Cases and plain forms of the operators between a served layer's products:
the root-mean-square norm with the residual's addition and an output in 8-bit
codes, the 8-bit integer product with bias, activation and residual, the gated
feed-forward product (both projections, activation and product), and attention
over the quantized cache with capped scores, a bias by distance and a prefix
that every token sees.

A row x of values is held as the integers nearest to top * x / max|x| (ties to
the even one; top = 127 for 8 bits, 7 for 4) and the scale max|x| / top.
Cache layout (the one of include/gptq.h): codes [n_pages, n_kv_heads,
page_size, head_dim * bits / 8] bytes, scales [n_pages, n_kv_heads, page_size]
fp32; 4 bits: code + 8 in a nibble, the lower dimension in the low one.
"""
import math
import random

import torch

own = False  # True: run() calls this repository's kernels; False: the plain forms below

BF16, F32, I8 = "bf16", "f32", "i8"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4, I8: 1}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases --

def _norm(name, m, d, x=BF16, res=BF16, y=I8):
    """x: type of the sublayer's output; res: of the hidden state it is added to ("": nothing is added); y: of the normed row."""
    return {"name": name, "op": "norm", "m": m, "d": d, "x": x, "res": res, "y": y}


def _linear(name, m, d_in, d_out, x=BF16, y=BF16, asym=False, bias=False, act="", res=""):
    return {"name": name, "op": "linear", "m": m, "d_in": d_in, "d_out": d_out, "x": x, "y": y, "asym": asym,
            "bias": bias, "act": act, "res": res}


def _gated(name, m, d_in, d_out, x=BF16, y=BF16, asym=False, bias=False, act="silu"):
    return {"name": name, "op": "gated", "m": m, "d_in": d_in, "d_out": d_out, "x": x, "y": y, "asym": asym,
            "bias": bias, "act": act}


def _attention(name, n_seq, new, ctx, heads, kv_heads, head_dim, page, bits, cap=0.0, slopes=False, prefix=False, pick=0):
    return {"name": name, "op": "attention", "n_seq": n_seq, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "bits": bits,
            "cap": cap, "slopes": slopes, "prefix": prefix, "pick": pick}


def listed():
    return [
        # one sequence being decoded: the norm between two layers of a 4096-wide model, latency
        _norm("norm 1 x 4096 int8", 1, 4096),
        # an odd number of tokens with the hidden state in fp32, as the block driver keeps it; a layer that takes fp32
        _norm("norm 777 x 5120 fp32", 777, 5120, x=F32, res=F32, y=F32),
        # the tokens of eight prompts of 2048
        _norm("norm 16384 x 4096 int8", 16384, 4096),
        # one sequence through the output projection of a 4096-wide model, added to the hidden state: latency
        _linear("linear 1 x 4096 -> 4096 residual", 1, 4096, 4096, res=BF16),
        # an odd number of prompt tokens, fp32 around them, a layer with everything
        _linear("linear 509 x 11008 -> 4096 all fp32", 509, 11008, 4096, x=F32, y=F32, asym=True, bias=True, act="gelu", res=F32),
        # a prompt through the down projection of an 8192-wide model, added to the hidden state
        _linear("linear 2048 x 28672 -> 8192 res", 2048, 28672, 8192, res=BF16),
        # one sequence through gate and up of a 4096-wide model: both weights are read once
        _gated("gated 1 x 4096 -> 11008", 1, 4096, 11008),
        # an odd number of sequences decoded together; asymmetric layers, codes from the norm before
        _gated("gated 61 x 4096 -> 11008 asym", 61, 4096, 11008, x=I8, asym=True),
        # a prompt through gate and up of an 8192-wide model
        _gated("gated 2048 x 8192 -> 28672", 2048, 8192, 28672, x=I8),
        # a serving batch of a model with distance biases: 48 sequences of very different lengths, one token each
        _attention("decode 48 ragged 32/8x128 slopes", 48, (1, 1), (200, 8000), 32, 8, 128, 16, 8, slopes=True, pick=1),
        # whole prompts of a model with capped scores
        _attention("prompts 2 x 2048 32/16x128 cap", 2, (2048, 2048), (0, 0), 32, 16, 128, 64, 8, cap=50.0),
        # chunks whose context is a prefix that all tokens see, capped scores, the cache in 4 bits
        _attention("chunks 3 x 300..700 16/4x64 prefix", 3, (300, 700), (1000, 4000), 16, 4, 64, 32, 4, cap=30.0, prefix=True, pick=2),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "gated", "attention", "attention"))
    if op == "norm":
        d = _log(rng, 16, 28672)
        if rng.random() < 0.5:
            d = 64 * max(1, d // 64)
        m = _log(rng, 1, max(1, min(16384, 16384 * 4096 // (3 * d))))
        c = _norm("", m, d, rng.choice((BF16, BF16, F32)), rng.choice((BF16, BF16, F32, "")), rng.choice((I8, I8, BF16, F32)))
    elif op in ("linear", "gated"):
        d_in = 32 * _log(rng, 2, 896)
        d_out = _log(rng, 16, 28672)
        m = _log(rng, 1, max(1, min(2048, 2048 * 28672 * 8192 // (4 * d_in * d_out))))
        x, y, asym, bias = rng.choice((BF16, F32, I8)), rng.choice((BF16, F32)), rng.random() < 0.5, rng.random() < 0.5
        if op == "linear":
            act, res = rng.choice(("", "", "relu", "gelu", "gelu_tanh", "silu")), rng.choice(("", BF16, F32))
            if not bias and not act and not res:
                res = BF16
            c = _linear("", m, d_in, d_out, x, y, asym, bias, act, res)
        else:
            c = _gated("", m, d_in, d_out, x, y, asym, bias, rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu")))
    else:
        kv_heads, group, head_dim = _log(rng, 1, 32), rng.choice((1, 1, 2, 3, 4, 7, 8)), rng.choice((32, 64, 80, 96, 128, 128, 256))
        n_seq = _log(rng, 1, 64)
        heads = kv_heads * group
        new = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 16, 1024)))
        new = max(1, min(new, int(math.sqrt(2.5e8 / (n_seq * heads)))))
        ctx = int(min(60000, 2e8 / (n_seq * kv_heads * head_dim), 2.5e8 / (n_seq * heads * new)))
        ctx = _log(rng, 1, max(2, ctx))
        kind = rng.choice(("cap", "slopes", "prefix", "cap prefix", "cap slopes", "slopes prefix", "cap slopes prefix"))
        c = _attention("", n_seq, (max(1, new // 2) if new > 1 else 1, new), (ctx // 5, ctx), heads, kv_heads, head_dim,
                       rng.choice((16, 32, 64, 128, 256)), rng.choice((8, 8, 4)),
                       rng.choice((5.0, 20.0, 30.0, 50.0)) if "cap" in kind else 0.0, "slopes" in kind, "prefix" in kind,
                       rng.randrange(1000))
    del c["name"]
    return c


def _lengths(case):
    """Per sequence: (new tokens, keys with the new ones, keys that every token sees), drawn from the case alone."""
    r = random.Random(case["pick"])
    got = []
    for _ in range(case["n_seq"]):
        new = r.randint(case["new_lo"], case["new_hi"])
        ctx = case["ctx_lo"] if case["ctx_lo"] == case["ctx_hi"] else _log(r, max(1, case["ctx_lo"]), case["ctx_hi"])
        got.append((new, ctx + new, r.randint(0, ctx + new) if case["prefix"] else 0))
    return got


def _seen(new, length, prefix):
    """Pairs of a new token and a key that it sees."""
    return sum(max(length - new + t + 1, prefix) for t in range(new))


def work(case):
    if case["op"] == "norm":
        n, res = case["m"] * case["d"], SIZE.get(case["res"], 0)
        row = 4 * case["m"] if case["y"] == I8 else 0
        return {"bytes": n * (SIZE[case["x"]] + 2 * res + SIZE[case["y"]]) + 4 * case["d"] + row, "flops": 8 * n}
    if case["op"] in ("linear", "gated"):
        m, k, n = case["m"], case["d_in"], case["d_out"]
        layers = 2 if case["op"] == "gated" else 1
        one = n * k + 4 * n * (1 + case["asym"] + case["bias"])
        x = m * k * SIZE[case["x"]] + (4 * m * (1 + case["asym"]) if case["x"] == I8 else 0)
        return {"bytes": x + layers * one + m * n * (SIZE[case["y"]] + SIZE.get(case.get("res", ""), 0)),
                "flops": layers * 2 * m * n * k}
    d, h, kv = case["head_dim"], case["heads"], case["kv_heads"]
    lens = _lengths(case)
    return {"bytes": sum(n for n, _, _ in lens) * 4 * h * d + sum(length for _, length, _ in lens) * 2 * kv * (d * case["bits"] // 8 + 4),
            "flops": 4 * sum(_seen(*one) for one in lens) * h * d}


# ------------------------------------------------------------------ inputs --

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _activations(gen, rows, d, dtype, spread=1.0, hot=50.0):
    """Log-normal channel scales and a few channels `hot` times as large, as activations have them."""
    sigma = torch.exp(spread * _normal(gen, d))
    is_hot = torch.rand(d, generator=gen, device=DEV) < 0.01
    return (_normal(gen, rows, d) * torch.where(is_hot, hot * sigma, sigma)).to(dtype)


def _pages(case, lens, gen):
    """Every sequence's pages, spread over the cache in a random order."""
    page = case["page"]
    need = [-(-one[1] // page) for one in lens]
    order = torch.randperm(sum(need) + 3, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 3


def _random_cache(gen, n_pages, case):
    """A cache in use: rows of normal values and their scales, already quantized."""
    shape = (n_pages, case["kv_heads"], case["page"])
    codes, scales = [], []
    for _ in range(2):
        q = torch.empty(*shape, case["head_dim"] * case["bits"] // 8, dtype=torch.int8 if case["bits"] == 8 else torch.uint8, device=DEV)
        s = torch.empty(shape, dtype=torch.float32, device=DEV)
        for a in range(0, n_pages, 4096):
            b = min(n_pages, a + 4096)
            c, s[a:b] = _quantized(_normal(gen, b - a, *shape[1:], case["head_dim"]), case["bits"], torch.float32)
            q[a:b] = _packed(c, case["bits"])
        codes.append(q)
        scales.append(s)
    return codes, scales


def _layer(gen, case):
    """A layer in 8-bit integers, as a checkpoint's is laid out once: codes, scales, offsets and the bias."""
    d_out, d_in = case["d_out"], case["d_in"]
    w = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV)
    scale = torch.empty(d_out, device=DEV)
    for a in range(0, d_out, 4096):
        b = min(d_out, a + 4096)
        c, scale[a:b] = _quantized(d_in ** -0.5 * _normal(gen, b - a, d_in), 8, torch.float32)
        w[a:b] = c.to(torch.int8)
    layer = {"w": w, "scales": scale}
    if case["asym"]:
        layer["offsets"] = torch.randint(-20, 21, (d_out,), generator=gen, device=DEV, dtype=torch.int32)
    if case["bias"]:
        layer["bias"] = _normal(gen, d_out)
    return layer


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "norm":
        m, d = case["m"], case["d"]
        st["input"] = _activations(gen, m, d, DTYPE[case["x"]], 0.5, 8.0)
        st["hidden"] = 4.0 * _activations(gen, m, d, DTYPE[case["res"]], 0.5, 8.0) if case["res"] else None
        st["weight"] = 1.0 + 0.2 * _normal(gen, d)
        return st
    if case["op"] in ("linear", "gated"):
        m, d_in = case["m"], case["d_in"]
        if case["x"] == I8:  # what the norm before gave
            code, scale = _quantized(_activations(gen, m, d_in, torch.float32, 0.5, 8.0), 8)
            st["input"] = (code.to(torch.int8), scale, code.sum(dim=1).to(torch.int32))
        else:
            st["input"] = _activations(gen, m, d_in, DTYPE[case["x"]], 0.5, 8.0)
        st["layers"] = [_layer(gen, case) for _ in range(2 if case["op"] == "gated" else 1)]
        if case.get("res"):
            st["hidden"] = (4.0 * _normal(gen, m, case["d_out"])).to(DTYPE[case["res"]])
        return st
    lens = _lengths(case)
    st["table"], n_pages = _pages(case, lens, gen)
    st["codes"], st["scales"] = _random_cache(gen, n_pages, case)
    starts = [0]
    for new, _, _ in lens:
        starts.append(starts[-1] + new)
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st["q"] = (3.0 * _normal(gen, starts[-1], case["heads"], case["head_dim"])).to(torch.bfloat16)
    st["starts"], st["lens"] = whole(starts), whole([one[1] for one in lens])
    st["prefixes"] = whole([one[2] for one in lens]) if case["prefix"] else None
    st["slope"] = torch.exp2(-8.0 * torch.arange(1, case["heads"] + 1, device=DEV) / case["heads"]) if case["slopes"] else None
    st["max_new"], st["max_len"] = max(one[0] for one in lens), max(one[1] for one in lens)
    return st


# -------------------------------------------------------------- plain forms --

def _quantized(x, bits, calc=torch.float64):
    """Codes (as whole numbers in `calc`) and fp32 scales of the rows of x.  The nearest integer is
    decided in 64 bits: ties (max/2 -> 63.5) are common among bf16 values."""
    top = 127 if bits == 8 else 7
    xc = x.to(calc)
    most = xc.abs().amax(dim=-1)
    code = torch.round(xc * top / torch.where(most > 0, most, torch.ones_like(most))[..., None])
    return code, (most / top).float()


def _packed(code, bits):
    if bits == 8:
        return code.to(torch.int8)
    n = (code + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpacked(held, bits):
    """The codes as fp32."""
    if bits == 8:
        return held.float()
    return torch.stack((held & 15, held >> 4), dim=-1).flatten(-2).float() - 8


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_norm(st):
    h = st["input"].float()
    got = {}
    if st["hidden"] is not None:
        h = h + st["hidden"].float()
        got["hidden"] = h.to(DTYPE[st["res"]])
    rstd = torch.rsqrt((h * h).mean(dim=-1, keepdim=True) + EPS)
    u = h * st["weight"]
    if st["y"] != I8:
        got["y"] = (u * rstd).to(DTYPE[st["y"]])
        return got
    code, scale = _quantized(u, 8)  # the codes of a row are those of any multiple of it
    scale = scale * rstd.squeeze(-1)
    got["scales"] = scale
    got["values"] = (code.float() * scale[:, None]).to(torch.bfloat16)
    return got


def _plain_product(x, layer):
    code, scale = x
    w = layer["w"].float()
    if "offsets" in layer:
        w = w - layer["offsets"].float()[:, None]
    z = ((code @ w.t()) * scale[:, None]) * layer["scales"]
    return z + layer["bias"] if "bias" in layer else z


def _plain_layers(st):
    if st["x"] == I8:
        code, scale, _ = st["input"]
    else:
        code, scale = _quantized(st["input"], 8)
    x = (code.float(), scale)
    y = _act(_plain_product(x, st["layers"][0]), st["act"])
    if st["op"] == "gated":
        y = y * _plain_product(x, st["layers"][1])
    elif st["res"]:
        y = y + st["hidden"].float()
    return {"y": y.to(DTYPE[st["y"]])}


def _plain_attention(st):
    kv, d, page, bits = st["kv_heads"], st["head_dim"], st["page"], st["bits"]
    group, most, longest = st["heads"] // kv, st["max_new"], st["max_len"]
    n_seq = st["n_seq"]
    new = (st["starts"][1:] - st["starts"][:-1]).long()
    tok = torch.arange(most, device=DEV)
    row = torch.clamp(st["starts"][:-1].long()[:, None] + tok, max=st["q"].shape[0] - 1)     # [seq, token]
    q = st["q"].float()[row].view(n_seq, most, kv, group, d).permute(0, 2, 1, 3, 4).reshape(n_seq, kv, most * group, d)
    both = []
    for held, scales in zip(st["codes"], st["scales"]):
        x = _unpacked(held[st["table"].long()], bits) * scales[st["table"].long()][..., None]  # [seq, page, kv, token, d]
        both.append(x.transpose(1, 2).reshape(n_seq, kv, -1, d)[:, :, :longest])
        del x
    k, v = both
    score = ((q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))).view(n_seq, kv, most, group, longest)
    if st["cap"]:
        score.mul_(1.0 / st["cap"]).tanh_().mul_(st["cap"])
    at = st["lens"].long()[:, None] - new[:, None] + tok                                     # place of each token
    key = torch.arange(longest, device=DEV)
    if st["slopes"]:
        away = (at[:, :, None] - key).abs().float()                                          # [seq, token, key]
        score -= away[:, None, :, None, :] * st["slope"].view(1, kv, 1, group, 1)
        del away
    last = torch.maximum(at, st["prefixes"].long()[:, None] - 1) if st["prefix"] else at     # last key each token sees
    score.masked_fill_((key > last[:, :, None])[:, None, :, None, :], -math.inf)
    score -= torch.clamp(score.amax(dim=-1, keepdim=True), min=-1e30)
    score.exp_()
    score = score.view(n_seq, kv, most * group, longest)
    total = score.sum(dim=-1, keepdim=True)
    out = (score @ v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(n_seq, kv, most, group, d).permute(0, 2, 1, 3, 4).reshape(n_seq, most, kv * group, d)
    return {"out": out[tok < new[:, None]].to(torch.bfloat16)}


def run(state):
    if not own:
        return {"norm": _plain_norm, "linear": _plain_layers, "gated": _plain_layers, "attention": _plain_attention}[state["op"]](state)
    import post_weight_quantization_07_amd as G
    if state["op"] == "norm":
        y = state["y"]
        rows, hidden = G.gptq_norm_tokens(state["input"], state["weight"], state["hidden"], EPS, dtype=torch.int8 if y == I8 else DTYPE[y])
        got = {"hidden": hidden} if state["hidden"] is not None else {}
        if y != I8:
            return {**got, "y": rows}
        codes, scales, _ = rows
        values = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
        return {**got, "scales": scales, "values": torch.mul(codes, scales[:, None], out=values)}
    if state["op"] == "linear":
        layer = state["layers"][0]
        return {"y": G.gptq_integer_matmul(state["input"], layer["w"], layer["scales"], layer.get("offsets"), out_dtype=DTYPE[state["y"]],
                                           bias=layer.get("bias"), activation=state["act"] or None, residual=state.get("hidden"))}
    if state["op"] == "gated":
        return {"y": G.gptq_integer_gated(state["input"], *state["layers"], activation=state["act"], out_dtype=DTYPE[state["y"]])}
    cache = G.QuantizedCache(state["codes"][0], state["codes"][1], state["scales"][0], state["scales"][1], state["bits"])
    return {"out": G.gptq_cache_attention(state["q"], cache, state["table"], state["starts"], state["lens"], cap=state["cap"] or None,
                                          slopes=state["slope"], prefix_lens=state["prefixes"])}


# ------------------------------------------------------------ in 64 bits --

def _exact_codes(x, top):
    """Nearest integers to top x / max|x|, ties to even, by comparing products that 64 bits hold exactly."""
    a = x.double().abs()
    most = a.amax(dim=-1, keepdim=True)
    safe = torch.where(most > 0, most, torch.ones_like(most))
    up = torch.floor((2 * top * a + safe) / (2 * safe))
    tie = 2 * top * a + safe == 2 * safe * up
    near = torch.where(tie & (up.remainder(2) == 1), up - 1, up)
    return torch.sign(x.double()) * near, most / top


def _exact_values(held, scales, bits):
    n = held.to(torch.int16)
    c = n if bits == 8 else torch.stack((n % 16, n // 16), dim=-1).reshape(*n.shape[:-1], -1) - 8
    return c.double() * scales.double().unsqueeze(-1)


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        got = {"hidden": [], "y": [], "scales": [], "values": []}
        for a in range(0, case["m"], 2048):
            h = st["input"][a:a + 2048].double()
            if st["hidden"] is not None:
                h = h + st["hidden"][a:a + 2048].double()
                got["hidden"].append(h)
            y = st["weight"].double() * h / (h.pow(2).sum(dim=-1, keepdim=True) / case["d"] + EPS).sqrt()
            if case["y"] == I8:
                code, scale = _exact_codes(y, 127)
                got["scales"].append(scale.squeeze(-1))
                got["values"].append(code * scale)
            else:
                got["y"].append(y)
        return {k: torch.cat(v) for k, v in got.items() if v}
    if case["op"] in ("linear", "gated"):
        if case["x"] == I8:
            code, scale = st["input"][0].double(), st["input"][1].double().unsqueeze(1)
        else:
            code, scale = _exact_codes(st["input"], 127)
        x = code * scale
        y = torch.empty(case["m"], case["d_out"], dtype=torch.float64, device=DEV)
        for a in range(0, case["d_out"], 2048):
            z = []
            for layer in st["layers"]:
                w = layer["w"][a:a + 2048].double()
                if case["asym"]:
                    w -= layer["offsets"][a:a + 2048].double().unsqueeze(1)
                one = torch.mm(x, (w * layer["scales"][a:a + 2048].double().unsqueeze(1)).t().contiguous())
                z.append(one + layer["bias"][a:a + 2048].double() if case["bias"] else one)
            z[0] = _exact_act(z[0], case["act"])
            if case["op"] == "gated":
                y[:, a:a + 2048] = z[0] * z[1]
            else:
                y[:, a:a + 2048] = z[0] + st["hidden"][:, a:a + 2048].double() if case["res"] else z[0]
        return {"y": y}
    kv, d = case["kv_heads"], case["head_dim"]
    group = case["heads"] // kv
    outs = []
    for i, (new, length, prefix) in enumerate(_lengths(case)):
        pages = st["table"][i, :-(-length // case["page"])].long()
        a = int(st["starts"][i])
        q = st["q"][a:a + new].double().view(new, kv, group, d)
        one = torch.empty(new, kv, group, d, dtype=torch.float64, device=DEV)
        j = torch.arange(length, device=DEV)
        place = (length - new + torch.arange(new, device=DEV)).unsqueeze(1)
        hidden = (j > place) & (j >= prefix)
        for h in range(kv):
            k, v = (_exact_values(c[pages, h], s[pages, h], case["bits"]).view(-1, d)[:length] for c, s in zip(st["codes"], st["scales"]))
            p = torch.mm(q[:, h].reshape(-1, d), k.t().contiguous()).view(new, group, length) / math.sqrt(d)
            if case["cap"]:
                p = case["cap"] * torch.tanh(p / case["cap"])
            if case["slopes"]:
                slope = st["slope"][h * group:(h + 1) * group].double()
                p = p - slope.view(1, group, 1) * (place - j).abs().double().unsqueeze(1)
            p = torch.softmax(p.masked_fill(hidden.unsqueeze(1), -math.inf), dim=-1)
            one[:, h] = torch.mm(p.view(-1, length), v).view(new, group, d)
        outs.append(one.view(new, case["heads"], d))
    return {"out": torch.cat(outs)}
