"""Layer-sequential quantization of one transformer block.

AutoGPTQ examples walkthrough (true_sequential; the layer groups of a
decoder block, inside_layer_modules) and the GPTQ 实战 chapter's layer loop:
calibration activations run through the block, the inputs of the layers about
to be quantized are collected, H is accumulated from them, the layers are
solved, and the following layers see the outputs of the already-quantized
ones.  The groups, in order:

    k_proj, v_proj, q_proj    (one input: the normalized hidden states)
    o_proj                    (the attention output)
    up_proj, gate_proj        (the normalized hidden states after attention)
    down_proj                 (silu(gate) * up)

Each group shares one input, so it is solved against one H and one U
(solve_layers_shared).  The block is Llama-shaped: RMSNorm, causal multi-head
attention without position encoding, a gated MLP; unit norm weights, plain
scores and SiLU unless the caller says what the model has.
The block's own arithmetic (norms, attention, activation) is the driver's
plumbing and runs in torch (fp32); the layer solves run in libgptq.so.  For a
model that will be served with a quantized key/value cache, cache_bits runs
the attention over such a cache, so that o_proj and the layers after it are
calibrated on the outputs they will see.

serve_block is the block as it is served once quantized: its layers in 8-bit
integers (checkpoint.integer_layer), its keys and values in a QuantizedCache,
and everything between them in libgptq.so's kernels.
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import Dict, List, Mapping, Optional

import torch
import torch.nn.functional as F

from . import solve_layers_shared
from ._lib import (ACTIVATIONS, QuantizeConfig, QuantizedCache, gptq_cache_attention, gptq_cache_write, gptq_integer_gated,
                   gptq_integer_matmul, gptq_norm_tokens)

QUANT_ORDER: List[List[str]] = [["k_proj", "v_proj", "q_proj"], ["o_proj"], ["up_proj", "gate_proj"],
                                ["down_proj"]]


@dataclass
class Block:
    d_model: int
    n_heads: int
    d_ff: int
    weights: Dict[str, torch.Tensor]  # name -> [d_out, d_in] fp32 on the device
    eps: float = 1e-6


_ACTIVATE = {None: lambda z: z, "relu": F.relu, "gelu": F.gelu, "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
             "silu": F.silu}


def rms_norm(x: torch.Tensor, eps: float) -> torch.Tensor:
    return x * torch.rsqrt(x.pow(2).mean(dim=-1, keepdim=True) + eps)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_seq: int, seq_len: int, n_heads: int,
              seqs_per_call: int = 8, cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
              prefix_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal multi-head attention over n_seq sequences of seq_len tokens
    (rows of q, k, v are tokens, sequence-major), fp32, a few sequences per call;
    cap, slopes and prefix_lens as for gptq_cache_attention."""
    d = q.shape[1]
    hd = d // n_heads
    out = torch.empty_like(q)
    plain = cap is None and slopes is None and prefix_lens is None
    if not plain:
        place = torch.arange(seq_len, device=q.device)
        away = (place[:, None] - place).abs().to(torch.float32)

    def changed(qh, kh, vh, s0, s1):
        s = torch.matmul(qh, kh.transpose(-1, -2).contiguous()) * hd ** -0.5
        if cap is not None:
            s = cap * torch.tanh(s / cap)
        if slopes is not None:
            s = s - slopes.view(1, n_heads, 1, 1) * away
        seen = (place <= place[:, None]).expand(s1 - s0, 1, seq_len, seq_len)
        if prefix_lens is not None:
            seen = seen | (place < prefix_lens[s0:s1].view(-1, 1, 1, 1))
        return torch.matmul(torch.softmax(s.masked_fill(~seen, float("-inf")), dim=-1), vh)
    for s0 in range(0, n_seq, seqs_per_call):
        s1 = min(n_seq, s0 + seqs_per_call)
        r0, r1 = s0 * seq_len, s1 * seq_len

        def heads(t):
            return t[r0:r1].reshape(s1 - s0, seq_len, n_heads, hd).transpose(1, 2).contiguous()
        if plain:
            o = F.scaled_dot_product_attention(heads(q), heads(k), heads(v), is_causal=True)
        else:
            o = changed(heads(q), heads(k), heads(v), s0, s1)
        out[r0:r1] = o.transpose(1, 2).reshape((s1 - s0) * seq_len, d)
    return out


def cached_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_seq: int, seq_len: int, n_heads: int,
                     bits: int, page_size: int = 64, cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
                     prefix_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """attention() with the keys and values held as `bits`-bit codes in a
    QuantizedCache, queries in bf16, out in q's dtype.  A head's dimension is a
    multiple of 16 up to 256."""
    hd = q.shape[1] // n_heads
    pages = -(-seq_len // page_size)
    cache = QuantizedCache.empty(n_seq * pages, page_size, n_heads, hd, bits, q.device)
    table = torch.arange(n_seq * pages, dtype=torch.int32, device=q.device).view(n_seq, pages)
    starts = torch.arange(0, n_seq * seq_len + 1, seq_len, dtype=torch.int32, device=q.device)
    lens = torch.full((n_seq,), seq_len, dtype=torch.int32, device=q.device)
    tok = torch.arange(n_seq * seq_len, device=q.device)
    slots = torch.div(tok, seq_len, rounding_mode="floor") * (pages * page_size) + tok % seq_len

    def heads(t):
        return t.reshape(n_seq * seq_len, n_heads, hd).contiguous()
    gptq_cache_write(cache, heads(k), heads(v), slots)
    o = gptq_cache_attention(heads(q).to(torch.bfloat16), cache, table, starts, lens, cap=cap, slopes=slopes,
                             prefix_lens=prefix_lens)
    return o.reshape(q.shape).to(q.dtype)


@dataclass
class BlockResult:
    layers: Dict[str, dict] = field(default_factory=dict)   # per layer: solve outputs
    inputs: Dict[str, torch.Tensor] = field(default_factory=dict)  # per group (first member): bf16 input
    output: Optional[torch.Tensor] = None                   # block output with the quantized weights
    ms: Dict[str, float] = field(default_factory=dict)      # forward / solve time per group


def quantize_block(block: Block, x0: torch.Tensor, n_seq: int, seq_len: int, cfg: QuantizeConfig,
                   keep_inputs: bool = False, timed: bool = False, cache_bits: Optional[int] = None,
                   norms: Optional[Mapping[str, torch.Tensor]] = None, activation: Optional[str] = "silu",
                   cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
                   prefix_lens: Optional[torch.Tensor] = None) -> BlockResult:
    """Quantize the block's seven layers group by group (true-sequential).
    x0: hidden states entering the block, [n_seq * seq_len, d_model] fp32.
    Each quantized layer's weights are replaced by its dequantized Q before the
    next group's input is computed.  Returns the solve outputs per layer, the
    block output computed with the quantized weights, optionally each group's
    input (bf16, as accumulated into H) and, with `timed`, per-stage times.
    cache_bits (8 or 4): attention reads its keys and values from a cache of
    that many bits (cached_attention); None: fp32.  norms, activation, cap, slopes
    and prefix_lens: of the model, as serve_block takes them, so that each group is
    calibrated on what it will see there (layers with a bias are not solved here)."""
    res = BlockResult()
    W = block.weights
    norms = norms or {}
    if activation not in ACTIVATIONS:
        raise ValueError(f"quantize_block: unknown activation {activation!r}")
    scores = dict(cap=cap, slopes=slopes, prefix_lens=prefix_lens)

    def norm(x, name):
        y = rms_norm(x, block.eps)
        return y if norms.get(name) is None else y * norms[name].to(torch.float32)
    ev = {}

    def mark(tag):
        if timed:
            e = torch.cuda.Event(enable_timing=True)
            e.record()
            ev[tag] = e

    def solve(group: List[str], inp: torch.Tensor):
        xb = inp.to(torch.bfloat16)
        if keep_inputs:
            res.inputs[group[0]] = xb
        mark(f"solve {'+'.join(group)} start")
        outs = solve_layers_shared([W[n].to(torch.bfloat16) for n in group], [xb], cfg)
        mark(f"solve {'+'.join(group)} end")
        for n, o in zip(group, outs):
            res.layers[n] = o
            W[n] = o["Q"].contiguous()

    mark("forward 1 start")
    xn1 = norm(x0, "input")
    mark("forward 1 end")
    solve(QUANT_ORDER[0], xn1)
    mark("forward 2 start")
    qkv = [F.linear(xn1, W[n]) for n in ("q_proj", "k_proj", "v_proj")]
    if cache_bits is None:
        att = attention(*qkv, n_seq, seq_len, block.n_heads, **scores)
    else:
        att = cached_attention(*qkv, n_seq, seq_len, block.n_heads, cache_bits, **scores)
    del qkv
    mark("forward 2 end")
    solve(QUANT_ORDER[1], att)
    mark("forward 3 start")
    h = x0 + F.linear(att, W["o_proj"])
    xn2 = norm(h, "post_attention")
    mark("forward 3 end")
    solve(QUANT_ORDER[2], xn2)
    mark("forward 4 start")
    m = _ACTIVATE[activation](F.linear(xn2, W["gate_proj"])) * F.linear(xn2, W["up_proj"])
    mark("forward 4 end")
    solve(QUANT_ORDER[3], m)
    mark("forward 5 start")
    res.output = h + F.linear(m, W["down_proj"])
    mark("forward 5 end")
    if timed:
        torch.cuda.synchronize()
        tags = sorted({t.rsplit(" ", 1)[0] for t in ev})
        res.ms = {t: ev[t + " start"].elapsed_time(ev[t + " end"]) for t in tags}
    return res


def serve_block(layers: Mapping[str, Mapping[str, torch.Tensor]], x: torch.Tensor, cache: QuantizedCache,
                slots: torch.Tensor, page_table: torch.Tensor, q_starts: torch.Tensor, kv_lens: torch.Tensor,
                n_heads: int, norms: Optional[Mapping[str, torch.Tensor]] = None, eps: float = 1e-6,
                activation: Optional[str] = "silu",
                cap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
                prefix_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The block's output for the hidden states x [n_tokens, d_model] (bf16 or
    fp32) of new tokens, prompts and single tokens alike, in x's dtype.

    layers: the seven layers of QUANT_ORDER as checkpoint.integer_layer gives
    them, each optionally with a "bias" (fp32 [d_out]).  norms: the weights of
    the norms before the attention ("input") and after it ("post_attention"),
    ones where absent.  The new tokens' keys and values are written to `slots`
    of the cache; page_table, q_starts, kv_lens, cap, slopes and prefix_lens as
    for gptq_cache_attention, activation as for gptq_integer_gated.  Rows of x
    outside the sequences (a padded batch; their slots -1) come back undefined
    and touch no others.  Between the layers values are bf16 or 8-bit codes; sums, norms and softmax are fp32."""
    n = x.shape[0]
    hd = cache.head_dim
    norms = norms or {}

    def apply(inp, name, dtype=torch.bfloat16, residual=None):
        t = layers[name]
        return gptq_integer_matmul(inp, t["w"], t["scales"], t.get("offsets"), out_dtype=dtype, bias=t.get("bias"),
                                   residual=residual)
    rows, _ = gptq_norm_tokens(x, norms.get("input"), eps=eps)
    q, k, v = (apply(rows, name) for name in ("q_proj", "k_proj", "v_proj"))
    gptq_cache_write(cache, k.view(n, cache.n_kv_heads, hd), v.view(n, cache.n_kv_heads, hd), slots)
    att = gptq_cache_attention(q.view(n, n_heads, hd), cache, page_table, q_starts, kv_lens, cap=cap, slopes=slopes,
                               prefix_lens=prefix_lens)
    rows, h = gptq_norm_tokens(apply(att.view(n, n_heads * hd), "o_proj"), norms.get("post_attention"), residual=x, eps=eps)
    m = gptq_integer_gated(rows, layers["gate_proj"], layers["up_proj"], activation, out_dtype=torch.bfloat16)
    return apply(m, "down_proj", x.dtype, residual=h)
