"""The cache-side operators of one attention layer: what is measured, and their plain forms.

Four operators stand between a layer's QKV projection and its attention output:

* ``qk``      norms of queries and keys for each head, with the position rotation in the same pass;
* ``append``  keys normed and rotated on the way into the bf16 paged cache, values copied, and the
  same into the FP8 cache (e4m3 codes, one power-of-two scale per 16 tokens and head);
* ``attn``    attention of query segments straight over the FP8 cache, one token to whole wavefronts.

``run`` computes them in plain torch operations in 32 bits, or, with ``own`` set, through this
repository's package.  ``exact`` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 16            # tokens per scale of the FP8 cache
E4M3_MAX = 448.0      # largest e4m3 magnitude
EXP_MIN, EXP_MAX = -100, 119   # exponents of a scale
EPS = 1e-6
FRAME = (30, 52)      # patches of one latent frame, rows and columns


def listed():
    return [
        # one new token of a language-model head layout (queries share K/V heads), q and k as
        # slices of one fused projection, at a far position
        {"name": "qk_token", "op": "qk", "tokens": 1, "start": 37439, "q_heads": 32, "k_heads": 8,
         "head_dim": 128, "axes": 1, "pairs": 64, "interleaved": False, "packed": True},
        # part of one latent frame, small heads, half of the channels rotated, an odd row count
        {"name": "qk_part", "op": "qk", "tokens": 1001, "start": 0, "q_heads": 16, "k_heads": 4,
         "head_dim": 64, "axes": 1, "pairs": 16, "interleaved": False, "packed": False},
        # the five chunks in flight of the 1.3B wavefront, frame / row / column rotation
        {"name": "qk_wavefront", "op": "qk", "tokens": 23400, "start": 9360, "q_heads": 12,
         "k_heads": 12, "head_dim": 128, "axes": 3, "pairs": 64, "interleaved": True,
         "packed": True},
        # one token into the bf16 cache
        {"name": "append_token", "op": "append", "cache": "bf16", "tokens": 1, "start": 32760,
         "heads": 8, "head_dim": 128, "page": 64, "axes": 1, "pairs": 64, "interleaved": False,
         "packed": True},
        # the five chunks in flight into the bf16 cache
        {"name": "append_wavefront", "op": "append", "cache": "bf16", "tokens": 23400,
         "start": 9360, "heads": 12, "head_dim": 128, "page": 64, "axes": 3, "pairs": 64,
         "interleaved": True, "packed": True},
        # one token into the middle of a block of the FP8 cache, whose earlier rows stay
        {"name": "append8_token", "op": "append", "cache": "fp8", "tokens": 1, "start": 37445,
         "heads": 8, "head_dim": 128, "page": 64, "axes": 1, "pairs": 64, "interleaved": False,
         "packed": True},
        # the five chunks in flight into the FP8 cache
        {"name": "append8_wavefront", "op": "append", "cache": "fp8", "tokens": 23400,
         "start": 9360, "heads": 12, "head_dim": 128, "page": 64, "axes": 3, "pairs": 64,
         "interleaved": True, "packed": True},
        # one query token against eight chunks, eight K/V heads shared by 32 query heads
        {"name": "attn_token", "op": "attn", "rows": 1, "keys": 37441, "chunks": 1, "blank": 0,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64},
        # one query token against the eleven chunks of the 14B-shaped wavefront
        {"name": "attn_token_40h", "op": "attn", "rows": 1, "keys": 51480, "chunks": 1, "blank": 0,
         "q_heads": 40, "kv_heads": 40, "head_dim": 128, "page": 128},
        # a few odd rows in two segments, some of which see no key yet, small heads and pages
        {"name": "attn_ragged", "op": "attn", "rows": 77, "keys": 8191, "chunks": 2, "blank": 3,
         "q_heads": 16, "kv_heads": 4, "head_dim": 64, "page": 16},
        # one rank's chunk against the eight it sees
        {"name": "attn_rank", "op": "attn", "rows": 4680, "keys": 37440, "chunks": 1, "blank": 0,
         "q_heads": 12, "kv_heads": 12, "head_dim": 128, "page": 64},
        # the whole 1.3B 5-step wavefront: two context chunks, five in flight
        {"name": "attn_wavefront", "op": "attn", "rows": 23400, "keys": 32760, "chunks": 5,
         "blank": 0, "q_heads": 12, "kv_heads": 12, "head_dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("qk", "append", "append", "attn", "attn", "attn"))
    d = rng.choice((64, 128, 128))
    page = 16 * _log(rng, 1, 16)
    if op == "attn":
        kv = rng.choice((1, 2, 4, 8, 12, 40))
        q = kv * rng.choice((1, 1, 2, 4)) if kv <= 12 else kv
        rows, keys = _log(rng, 1, 23400), _log(rng, 16, 51480)
        rows = min(rows, max(1, int(7e12 / (4.0 * d * q * keys))))
        chunks = rng.randint(1, min(5, rows))
        return {"op": op, "rows": rows, "keys": max(keys, rows), "chunks": chunks,
                "blank": rng.choice((0, 0, min(2, rows - 1))), "q_heads": q, "kv_heads": kv,
                "head_dim": d, "page": page}
    axes = rng.choice((1, 3))
    half = d // 2
    pairs = half if axes == 3 else rng.choice((half, half, half // 2))
    case = {"op": op, "tokens": _log(rng, 1, 23400), "start": _log(rng, 1, 30000),
            "head_dim": d, "axes": axes, "pairs": pairs,
            "interleaved": axes == 3 or rng.random() < 0.3, "packed": rng.random() < 0.5}
    heads = rng.choice((1, 2, 4, 8, 12))
    if op == "qk":
        return {**case, "k_heads": heads, "q_heads": heads * rng.choice((1, 1, 2, 4))
                if heads <= 4 else heads}
    return {**case, "cache": rng.choice(("bf16", "fp8", "fp8")), "heads": heads, "page": page}


# ------------------------------------------------------------------------------------- inputs
def _axis_pairs(case):
    """Pairs that turn with each axis of the position: all, or frame / row / column."""
    p = case["pairs"]
    return [p] if case["axes"] == 1 else [p - 2 * (p // 3), p // 3, p // 3]


def _positions(case):
    tok = torch.arange(case["start"], case["start"] + case["tokens"])
    if case["axes"] == 1:
        return tok.view(-1, 1)
    h, w = FRAME
    return torch.stack((tok // (h * w), tok // w % h, tok % w), 1)


def _angles(case, rows):
    """[rows, pairs] angles in 64 bits: position times 10000^(-i / pairs of the axis)."""
    freq = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
                      for n in _axis_pairs(case)])
    return torch.arange(rows, dtype=torch.float64).view(-1, 1) * freq


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rule(s, case):
    """The rotation table, the positions and which axis each pair turns with."""
    pos = _positions(case)
    ang = _angles(case, int(pos.max()) + 1)
    s["table"] = torch.stack((ang.cos(), ang.sin()), -1).float().cuda()
    s["positions"] = pos.to(torch.int32).cuda().contiguous()
    s["axis"] = torch.cat([torch.full((n,), a) for a, n in enumerate(_axis_pairs(case))]).cuda()
    if own:
        from block_causal_streaming_b200 import NormRope
        s["rule"] = NormRope(s["table"], axis_pairs=_axis_pairs(case),
                             interleaved=case["interleaved"], norm=True, eps=EPS)


def _projection(g, case, head_counts):
    """[T, H, D] tensors as a projection leaves them: apart, or slices of one fused output."""
    t, d = case["tokens"], case["head_dim"]
    x = _randn(g, t, sum(head_counts), d).mul_(1.7).add_(0.6 * _randn(g, 1, sum(head_counts), d))
    parts = x.to(torch.bfloat16).split(list(head_counts), dim=1)
    return list(parts) if case["packed"] else [p.contiguous() for p in parts]


def _weight(g, d):
    return (1 + 0.2 * _randn(g, d)).to(torch.bfloat16)


def _page_table(g, tokens, page):
    pages = -(-tokens // page)
    return torch.randperm(pages, generator=g, device="cuda").to(torch.int32), pages


def _slots(table, page, lo, hi):
    """Pool rows of logical tokens lo..hi-1."""
    tok = torch.arange(lo, hi, device="cuda")
    return table.long()[tok // page] * page + tok % page


def _encode(x):
    """x [blocks, 16, H, D] in 32 bits -> e4m3 codes and the scale exponents [blocks, H]: the
    smallest power of two that brings the block's largest finite magnitude to 448 or less."""
    x = torch.where(x.isfinite(), x, float("nan"))
    top = x.abs().nan_to_num(0.0).amax((1, 3))
    m, e = torch.frexp(top)                                   # top = m 2^e, m in [0.5, 1)
    e = torch.where(top > 0, e - 9 + (m > 0.875), EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    y = torch.ldexp(x, -e.float()[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), e


def _fill(g, s, case, tokens, heads):
    """An FP8 cache that holds `tokens` tokens; every other row holds anything, NaN codes here."""
    page, d = case["page"], case["head_dim"]
    table, pages = s["page_row"], s["pages"]
    for t in "kv":
        x = _randn(g, -(-tokens // BLOCK) * BLOCK, heads, d)
        if t == "k":
            x.mul_(1.2).add_(_randn(g, 1, heads, d))
        x.mul_(torch.exp(0.5 * _randn(g, x.shape[0], 1, 1)))
        codes, exp = _encode(x.view(-1, BLOCK, heads, d))
        pool = torch.full((pages * page, heads, d), 0x7F, dtype=torch.uint8, device="cuda")
        rows = _slots(table, page, 0, tokens)
        pool[rows] = codes.view(torch.uint8).view(-1, heads, d)[:tokens]
        scale = torch.full((pages * page // BLOCK, heads), 255, dtype=torch.uint8, device="cuda")
        scale[rows[::BLOCK] // BLOCK] = (exp + 127).to(torch.uint8)
        s[t + "_codes"] = pool.view(pages, page, heads, d)
        s[t + "_scale"] = scale.view(pages, page // BLOCK, heads)


def _limits(case):
    """Query segments: ([end row], [visible keys]).  Each chunk of rows is the end of the keys up
    to it, as in a wavefront; the first `blank` rows see no key."""
    r, n, b = case["rows"], case["keys"], case["blank"]
    ends = [r * (i + 1) // case["chunks"] for i in range(case["chunks"])]
    seen = [n - r + e for e in ends]
    return ([b] if b else []) + ends, ([0] if b else []) + seen


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    d = case["head_dim"]
    if case["op"] == "qk":
        _rule(s, case)
        s["q"], s["k"], _ = _projection(g, case, (case["q_heads"], case["k_heads"],
                                                  case["k_heads"]))
        s["q_weight"], s["k_weight"] = _weight(g, d), _weight(g, d)
        s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "append":
        _rule(s, case)
        h, end = case["heads"], case["start"] + case["tokens"]
        _, s["k"], s["v"] = _projection(g, case, (h, h, h))
        s["k_weight"] = _weight(g, d)
        s["page_row"], s["pages"] = _page_table(g, end, case["page"])
        if case["cache"] == "fp8":
            _fill(g, s, case, case["start"], h)
            for name in ("k_codes", "v_codes"):   # what is returned: no NaN in rows never written
                s[name].masked_fill_(s[name] == 0x7F, 0)
            for name in ("k_scale", "v_scale"):
                s[name].masked_fill_(s[name] == 255, 127)
        else:
            shape = (s["pages"], case["page"], h, d)
            s["k_pool"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            s["v_pool"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        if own:
            from block_causal_streaming_b200 import WavefrontDesc
            s["page_table"] = s["page_row"].view(1, -1)
            s["wf"] = WavefrontDesc([0, case["start"], end], [0, 0], 1, s["pages"])
    else:
        hq, hk = case["q_heads"], case["kv_heads"]
        s["page_row"], s["pages"] = _page_table(g, case["keys"], case["page"])
        _fill(g, s, case, case["keys"], hk)
        s["q"] = _randn(g, case["rows"], hq, d).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(hq, case["rows"], device="cuda")
        s["rows_end"], s["kv_end"] = _limits(case)
        if own:
            from block_causal_streaming_b200 import Segments, attn_fp8_block_workspace_size
            # a segment that ends before one in front of it takes that one's rows over
            ends = [min(s["rows_end"][i:]) for i in range(len(s["rows_end"]))]
            s["seg"] = Segments(ends, s["kv_end"], case["keys"], s["pages"])
            need = attn_fp8_block_workspace_size(s["seg"], hq, hk, d)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return s


# --------------------------------------------------------------------------------- plain forms
def _norm_rope(s, x, weight):
    """RMS norm of each head's row in 32 bits, then the rotation; not rounded."""
    case = s["case"]
    p = case["pairs"]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    cs = s["table"][s["positions"].long()[:, s["axis"]], torch.arange(p, device="cuda")]
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (y[..., 0:2 * p:2], y[..., 1:2 * p:2]) if case["interleaved"] else \
        (y[..., :p], y[..., p:2 * p])
    a, b = a * c - b * n, a * n + b * c
    turned = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., 2 * p:]), -1)


def _append_fp8(s, which, rows):
    """Rows (32 bits) of the new tokens into the cache: every block they touch is coded anew from
    its live rows, the new ones and those that stay."""
    case = s["case"]
    lo, hi = case["start"], case["start"] + case["tokens"]
    b0, b1 = lo // BLOCK, -(-hi // BLOCK)
    h, d = rows.shape[1:]
    codes, scale = s[which + "_codes"].view(-1, h, d), s[which + "_scale"].view(-1, h)
    x = torch.zeros((b1 - b0) * BLOCK, h, d, device="cuda")
    if lo % BLOCK:
        at = _slots(s["page_row"], case["page"], b0 * BLOCK, lo)
        old = codes[at].view(torch.float8_e4m3fn).float()
        x[:lo % BLOCK] = torch.ldexp(old, scale[at[0] // BLOCK].float()[None, :, None] - 127)
    x[lo - b0 * BLOCK:hi - b0 * BLOCK] = rows
    new, exp = _encode(x.view(-1, BLOCK, h, d))
    at = _slots(s["page_row"], case["page"], b0 * BLOCK, hi)
    codes[at] = new.view(torch.uint8).view(-1, h, d)[:hi - b0 * BLOCK]
    scale[at[::BLOCK] // BLOCK] = (exp + 127).to(torch.uint8)


def _dequantized(s, which, dtype):
    """The cache's live rows in logical order, [keys, H, D]."""
    case = s["case"]
    at = _slots(s["page_row"], case["page"], 0, case["keys"])
    c = s[which + "_codes"].flatten(0, 1)[at].view(torch.float8_e4m3fn).to(dtype)
    e = s[which + "_scale"].flatten(0, 1)[at // BLOCK].to(dtype) - 127
    return torch.ldexp(c, e[:, :, None])


def _attention(s):
    """Every segment: all heads' logits at once (query heads of one K/V head side by side)."""
    case = s["case"]
    hk, group, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["head_dim"]
    k, v = (_dequantized(s, t, torch.float32).transpose(0, 1) for t in "kv")
    q = (s["q"].float() * s["scale"]).view(-1, hk, group, d).permute(1, 2, 0, 3)
    out = torch.zeros(hk, group, case["rows"], d, device="cuda")
    lse = torch.full((hk, group, case["rows"]), -math.inf, device="cuda")
    for lo, hi, n in zip([0] + s["rows_end"], s["rows_end"], s["kv_end"]):
        if n:
            t = q[:, :, lo:hi].flatten(1, 2) @ k[:, :n].transpose(1, 2)
            top = t.amax(2, keepdim=True)
            p = t.sub_(top).exp_()
            total = p.sum(2, keepdim=True)
            out[:, :, lo:hi] = (p @ v[:, :n] / total).view(hk, group, hi - lo, d)
            lse[:, :, lo:hi] = (top + total.log()).view(hk, group, hi - lo)
    out = out.permute(2, 0, 1, 3).reshape(case["rows"], -1, d)
    return out.to(torch.bfloat16), lse.flatten(0, 1)


def _cache8(s):
    """The FP8 cache's buffers as the values that they hold."""
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"k_codes": s["k_codes"].view(f8), "k_scale": s["k_scale"].view(e8),
            "v_codes": s["v_codes"].view(f8), "v_scale": s["v_scale"].view(e8)}


def run(s):
    case = s["case"]
    if own:
        import block_causal_streaming_b200 as wf
    if case["op"] == "qk":
        if own:
            wf.qk_norm_rope(s["q"], s["q_out"], s["k"], s["k_out"], s["rule"], s["positions"],
                            s["q_weight"], s["k_weight"])
            return s["q_out"], s["k_out"]
        return (_norm_rope(s, s["q"], s["q_weight"]).to(torch.bfloat16),
                _norm_rope(s, s["k"], s["k_weight"]).to(torch.bfloat16))
    if case["op"] == "append" and case["cache"] == "bf16":
        if own:
            wf.kv_append_rope(s["k_pool"], s["v_pool"], 0, 1, 2, s["k"], s["v"], s["page_table"],
                              s["wf"], s["rule"], s["positions"], s["k_weight"])
        else:
            at = _slots(s["page_row"], case["page"], case["start"],
                        case["start"] + case["tokens"])
            s["k_pool"].flatten(0, 1)[at] = _norm_rope(s, s["k"], s["k_weight"]).to(torch.bfloat16)
            s["v_pool"].flatten(0, 1)[at] = s["v"]
        return s["k_pool"], s["v_pool"]
    if case["op"] == "append":
        if own:
            wf.kv_append_fp8_block(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], 0, 1, 2,
                                   s["k"], s["v"], s["page_table"], s["wf"], s["rule"],
                                   s["positions"], s["k_weight"])
        else:
            _append_fp8(s, "k", _norm_rope(s, s["k"], s["k_weight"]))
            _append_fp8(s, "v", s["v"].float())
        return _cache8(s)
    if own:
        wf.attn_forward_fp8_block(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                                  s["page_row"], s["seg"], s["scale"], s["out"], s["lse"],
                                  workspace=s["workspace"])
        return s["out"], s["lse"]
    return _attention(s)


def work(case):
    d = case["head_dim"]
    if case["op"] == "attn":
        hq, hk, r = case["q_heads"], case["kv_heads"], case["rows"]
        ends, seen = _limits(case)
        visible = sum((e - b) * n for b, e, n in zip([0] + ends, ends, seen))
        read = max(seen)
        return {"bytes": 4 * r * hq * d + 4 * r * hq + 2 * read * hk * d
                + 2 * -(-read // BLOCK) * hk, "flops": 4.0 * d * hq * visible}
    t = case["tokens"]
    table = 8 * case["pairs"] * min(t, 1024) + 4 * t * case["axes"]
    if case["op"] == "qk":
        h = case["q_heads"] + case["k_heads"]
        return {"bytes": 4 * t * h * d + table, "flops": 10.0 * t * h * d}
    h = case["heads"]
    written = 4 * t * h * d if case["cache"] == "bf16" else \
        2 * t * h * d + 2 * -(-t // BLOCK) * h
    return {"bytes": 4 * t * h * d + written + table, "flops": 12.0 * t * h * d}


# ------------------------------------------------------------------------------- definitions
def _exact_norm_rope(s, x, weight):
    """The definition in 64 bits, channel by channel: channel j of pair i is turned by its angle."""
    case = s["case"]
    p, d = case["pairs"], case["head_dim"]
    x = x.double()
    norm = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    y = x / norm * weight.double()
    first = torch.arange(p, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else p)
    z = torch.complex(y[..., first], y[..., second])
    cs = s["table"].double()                        # the table is an input: fp32 values
    pos = s["positions"].long()
    turn = torch.stack([torch.complex(cs[pos[:, a], i, 0], cs[pos[:, a], i, 1])
                        for i, a in enumerate(s["axis"].tolist())], 1)
    z = z * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _e4m3(y):
    """The nearest e4m3 value, ties to even: steps of 2^-9 up to 2^-6, then 3 bits after the first."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_append_fp8(s, which, rows):
    case = s["case"]
    lo, hi = case["start"], case["start"] + case["tokens"]
    h, d = rows.shape[1:]
    codes = s[which + "_codes"].view(torch.float8_e4m3fn).double().view(-1, h, d)
    scale = torch.exp2(s[which + "_scale"].double() - 127).view(-1, h)
    b0, b1 = lo // BLOCK, -(-hi // BLOCK)
    live = _slots(s["page_row"], case["page"], b0 * BLOCK, hi)
    value = torch.cat((codes[live[:lo - b0 * BLOCK]] * scale[live[:lo - b0 * BLOCK] // BLOCK, :, None],
                       rows.double()))
    pad = torch.cat((value, value.new_zeros(b1 * BLOCK - hi, h, d)))
    top = pad.view(b1 - b0, BLOCK, h, d).abs().amax((1, 3))
    # a largest magnitude of exactly 448 2^n has the exponent n, whatever log2 makes of its last bit
    exp = torch.ceil(torch.log2(top / E4M3_MAX) - 1e-12).clamp(EXP_MIN, EXP_MAX)
    size = torch.exp2(exp)
    new = _e4m3(value / size.repeat_interleave(BLOCK, 0)[:hi - b0 * BLOCK, :, None])
    codes[live] = new
    scale[live[::BLOCK] // BLOCK] = size
    return codes.view(s[which + "_codes"].shape), scale.view(s[which + "_scale"].shape)


def _exact_attention(s):
    case = s["case"]
    group = case["q_heads"] // case["kv_heads"]
    k, v = (_dequantized(s, t, torch.float64) for t in "kv")
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full((case["q_heads"], case["rows"]), -math.inf, dtype=torch.float64,
                     device="cuda")
    step = max(1, int(3e8) // case["keys"])
    start = [0] + s["rows_end"][:-1]
    for lo, hi, n in zip(start, s["rows_end"], s["kv_end"]):
        for a in range(lo, hi if n else lo, step):
            b = min(hi, a + step)
            for h in range(case["q_heads"]):
                logit = torch.matmul(q[a:b, h], k[:n, h // group].t()) * s["scale"]
                lse[h, a:b] = torch.logsumexp(logit, 1)
                out[a:b, h] = torch.exp(logit - lse[h, a:b, None]) @ v[:n, h // group]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return (_exact_norm_rope(s, s["q"], s["q_weight"]),
                _exact_norm_rope(s, s["k"], s["k_weight"]))
    if case["op"] == "attn":
        return _exact_attention(s)
    k = _exact_norm_rope(s, s["k"], s["k_weight"])
    if case["cache"] == "bf16":
        at = _slots(s["page_row"], case["page"], case["start"], case["start"] + case["tokens"])
        pools = []
        for x in (k, s["v"].double()):
            pool = torch.zeros(s["k_pool"].shape, dtype=torch.float64, device="cuda")
            pool.flatten(0, 1)[at] = x
            pools.append(pool)
        return tuple(pools)
    k_codes, k_scale = _exact_append_fp8(s, "k", k)
    v_codes, v_scale = _exact_append_fp8(s, "v", s["v"])
    return {"k_codes": k_codes, "k_scale": k_scale, "v_codes": v_codes, "v_scale": v_scale}
