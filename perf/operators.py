"""Cases of the operators around the latent cache, with their plain forms.

Three operators:

* ``mla_norm_rope``: every query head's row and the token's latent row (576
  values each) get an RMS norm over the first 512 values and the position
  rotation over the last 64, and the latent row goes into its slot of a bf16,
  FP8 or 4-bit cache.
* ``mla_norm_rope_bwd``: its gradients, from the fp32 dq and dkv that the
  attention's backward writes.
* ``sparse_mla_decode_fp4``: paged sparse decode over the 4-bit cache.

A 4-bit cache slot is 416 bytes: 256 bytes of e2m1 codes (code 2i in the low
half of byte i), 32 e4m3 scales (one for each 16 codes) and 64 bf16 values
(the rotated part).  The row is code * scale * kv_scale, then the 64 values.
"""
import math

import torch

own = False

D, DV, DR = 576, 512, 64
FP4_SLOT, FP8_SLOT = 416, 656
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _norm(name, tokens, heads, q_norm, cache, pairs, pad=0, far=0, kv_scale=1.0):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "q_norm": q_norm, "cache": cache,
            "pairs": pairs, "pad": pad, "far": far, "kv_scale": kv_scale}


def _grad(name, tokens, heads, q_norm, pairs, pad=0):
    return {"name": name, "op": "norm_rope_bwd", "tokens": tokens, "heads": heads, "q_norm": q_norm,
            "pairs": pairs, "pad": pad, "far": 0}


def _decode(name, batch, s_next, heads, topk, lo, hi, page, kv_scale=1.0):
    return {"name": name, "op": "decode_fp4", "batch": batch, "s_next": s_next, "heads": heads, "topk": topk,
            "lo": lo, "hi": hi, "page": page, "kv_scale": kv_scale}


def listed():
    return [
        # one new token of one request, far into its context: latency alone counts
        _norm("norm one token, 4-bit", 1, 8, False, "fp4", True, far=131071),
        # the decode workload's step: 16 requests of 6 speculative tokens, each at a position of its own
        _norm("norm decode step, bf16", 96, 8, False, "bf16", True, far=32768),
        # the mid prefill, 8 tensor-parallel heads with a query norm, padded behind its last token
        _norm("norm prefill 2119, FP8", 2128, 8, True, "fp8", False, pad=9),
        # the wide-head prefill: 8192 tokens of 64 heads
        _norm("norm prefill 8192, 4-bit", 8192, 64, True, "fp4", True),
        # a small training batch at the 8-head shape, the norm on the latent row alone
        _grad("grad 257 tokens", 257, 8, False, True),
        # the mid prefill's backward, query norm as well
        _grad("grad 2119 tokens", 2128, 8, True, False, pad=9),
        # packed training tokens at 64 heads
        _grad("grad 8192 tokens", 8192, 64, True, True),
        # one token of one long request: a single list over the whole card
        _decode("decode one token", 1, 1, 8, 2048, 32768, 32768, 64),
        # the paged decode workload: 16 requests, 6 speculative tokens each, 8 heads
        _decode("decode 16 x 6, 8 heads", 16, 6, 8, 2048, 4096, 32768, 64),
        # ragged: 24 heads, a list that ends inside a block, contexts shorter than the list, small pages
        _decode("decode ragged, 24 heads", 7, 3, 24, 1000, 3, 2500, 16, kv_scale=0.3),
        # many requests at 64 heads (heads not split over cards)
        _decode("decode 128 x 1, 64 heads", 128, 1, 64, 2048, 2048, 16384, 64),
        # a chunk of prompt tokens read against a cached prefix
        _decode("decode chunk of 512, 16 heads", 1, 512, 16, 2048, 24000, 24000, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope_bwd", "decode_fp4"))
    if op == "decode_fp4":
        heads = rng.choice((1, 2, 5, 8, 8, 16, 16, 24, 32, 48, 64, 64, 100, 128))
        topk = _log(rng, 17, 2048)
        s_next = rng.choice((1, 1, 2, 3, 6, 6, 6, _log(rng, 7, 300)))
        batch = max(1, min(_log(rng, 1, 160), 768 * 16 // (s_next * max(heads, 16))))
        lo = _log(rng, 1, 16384)
        hi = max(lo, _log(rng, 256, 32768))
        return {"op": op, "batch": batch, "s_next": s_next, "heads": heads, "topk": topk, "lo": lo, "hi": hi,
                "page": rng.choice((16, 32, 64, 64)), "kv_scale": rng.choice((1.0, 1.0, 0.5, 0.3))}
    heads = rng.choice((1, 3, 8, 8, 16, 20, 32, 64, 128))
    tokens = _log(rng, 1, 8192 * 64 // max(heads, 64))
    case = {"op": op, "tokens": tokens, "heads": heads, "q_norm": rng.random() < 0.5, "pairs": rng.random() < 0.5,
            "pad": rng.randrange(0, 1 + tokens // 8), "far": rng.choice((0, 0, 32768, 131071))}
    if op == "norm_rope":
        case["cache"] = rng.choice(("bf16", "fp8", "fp4", "fp4"))
        case["kv_scale"] = rng.choice((1.0, 1.0, 0.5, 0.3)) if case["cache"] == "fp4" else 1.0
    return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _table(n):
    """cos and sin of every position, [n, 64] fp32: 32 cosines, then 32 sines."""
    f = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _prepare_norm(case, seed):
    g = _gen(seed)
    t, h, pad, far = case["tokens"], case["heads"], case["pad"], case["far"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    # latent channels of unequal size, and rows too, as projections give them
    size = torch.exp(0.5 * randn(D))
    s = {"op": case["op"], "pairs": case["pairs"], "eps": 1e-6}
    s["q"] = (randn(t, h, D) * size * torch.exp(randn(t, h, 1))).bfloat16()
    s["kv"] = (randn(t, D) * size * torch.exp(randn(t, 1))).bfloat16()
    s["q_weight"] = (1 + 0.2 * randn(DV)).bfloat16() if case["q_norm"] else None
    s["kv_weight"] = (1 + 0.2 * randn(DV)).bfloat16()
    n_pos = max(far, t) + 1
    if far:   # decode: every token at a position of its own
        pos = torch.randint(max(0, far - 32768), far + 1, (t,), generator=g, device="cuda")
    else:
        pos = torch.arange(t, device="cuda")
    if pad:   # rows behind the last sequence belong to no token
        pos[t - pad:] = -1
    s["positions"] = pos.int()
    s["cos_sin"] = _table(n_pos)
    if case["op"] == "norm_rope_bwd":
        s["dq"], s["dkv"] = randn(t, h, D) * 0.01, randn(t, D) * 0.1
        return s
    page = 64
    blocks = t // page + 9
    slots = torch.randperm(blocks * page, generator=g, device="cuda")[:t]
    if pad:
        slots[t - pad:] = -1
    s["slots"] = slots.int()
    s["kv_scale"] = case["kv_scale"]
    s["format"] = case["cache"]
    if case["cache"] == "bf16":
        s["kv_cache"] = torch.zeros(blocks, page, D, dtype=torch.bfloat16, device="cuda")
    else:
        slot = FP4_SLOT if case["cache"] == "fp4" else FP8_SLOT
        s["kv_cache"] = torch.zeros(blocks, page, slot, dtype=torch.uint8, device="cuda")
    s["q_out"], s["kv_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["kv"])
    return s


def _codes(x):
    """Nearest e2m1 code (0..7) of magnitudes x; halfway goes to the even code."""
    b = torch.tensor([(E2M1[i] + E2M1[i + 1]) / 2 for i in range(7)], dtype=x.dtype, device=x.device)
    up = torch.bucketize(x, b)                 # halfway points go down
    even = (x[..., None] == b[1::2]).any(-1)   # halfway between an odd code and the even one above it: up
    return up + even


def _over(x, number):
    """x / number with one rounding: torch multiplies by the reciprocal of a Python number on the GPU, which
    moves quotients that lie halfway between two codes."""
    return x / torch.full((), number, dtype=x.dtype, device=x.device)


def _pack_fp4(rows, kv_scale):
    """Latent rows [n, 576] as 4-bit slots [n, 416]."""
    v = rows[:, :DV].float().view(-1, DV // 16, 16)
    scale = _over(v.abs().amax(-1), 6 * kv_scale).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    x = v / (scale.float() * kv_scale)[..., None]
    code = (_codes(x.abs()) | (torch.signbit(x).long() << 3)).view(-1, DV // 2, 2).to(torch.uint8)
    rope = rows[:, DV:].contiguous().view(torch.uint8)
    return torch.cat([code[..., 0] | (code[..., 1] << 4), scale.view(torch.uint8), rope], dim=1)


def _prepare_decode(case, seed):
    g = _gen(seed)
    b, sn, h, topk, page = case["batch"], case["s_next"], case["heads"], case["topk"], case["page"]
    randint = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")  # noqa: E731
    lens = randint(case["lo"], case["hi"], b)
    most = case["hi"]
    width = (most + page - 1) // page
    blocks = b * width + 3
    cache = torch.empty(blocks * page, FP4_SLOT, dtype=torch.uint8, device="cuda")
    for part in cache.split(1 << 18):
        rows = torch.randn(part.shape[0], D, generator=g, device="cuda")
        part.copy_(_pack_fp4((rows * (1 + 0.3 * torch.randn(D, generator=g, device="cuda"))).bfloat16(),
                             case["kv_scale"]))
    table = torch.randperm(blocks, generator=g, device="cuda")[:b * width].view(b, width).int()
    # each token's list: distinct positions that it can see, in rising order, -1 behind them
    n = b * sn
    sees = (lens[:, None] - sn + 1 + torch.arange(sn, device="cuda")).clamp(min=0).view(n)   # visible positions
    lists = torch.empty(n, topk, dtype=torch.int32, device="cuda")
    k = min(topk, most)
    for at in range(0, n, 256):
        part = sees[at:at + 256]
        key = torch.rand(part.numel(), most, generator=g, device="cuda")
        key.masked_fill_(torch.arange(most, device="cuda") >= part[:, None], -1.0)
        best, pos = key.topk(k, dim=1)
        pos = pos.masked_fill(best < 0, most).sort(dim=1).values
        lists[at:at + 256] = -1
        lists[at:at + 256, :k] = torch.where(pos < most, pos, -1).int()
    q = torch.randn(b, sn, h, D, generator=g, device="cuda").bfloat16()
    return {"op": "decode_fp4", "q": q, "kv_cache": cache.view(blocks, page, FP4_SLOT), "block_table": table,
            "cache_seqlens": lens.int(), "indices": lists.view(b, sn, topk), "sm_scale": D ** -0.5,
            "kv_scale": case["kv_scale"]}


def prepare(case, seed):
    return _prepare_decode(case, seed) if case["op"] == "decode_fp4" else _prepare_norm(case, seed)


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, pairs, back=False):
    """The rotation of x [..., 64] by cos, sin [..., 32]: neighbouring values
    turn together (`pairs`) or values 32 apart do."""
    if back:
        sin = -sin
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)


def _pow2(e):
    """2^e in float64 from its bits (torch's own powers of two are not all exact on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_bf16(y):
    """float64 rounded once to bf16 values (8 significant bits, ties to even)."""
    m, e = torch.frexp(y)
    return (torch.round(m * 256) * _pow2(e - 8)).float()


def _stored_fp4(y, kv_scale):
    """bf16 values [n, 512] as the 4-bit cache holds them."""
    v = y.view(-1, DV // 16, 16)
    scale = _over(v.abs().amax(-1), 6 * kv_scale).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn).float()
    step = (scale * kv_scale)[..., None]
    x = v / step
    value = torch.tensor(E2M1, device=y.device)[_codes(x.abs())]
    return (torch.copysign(value, x) * step).reshape(y.shape)


def _stored_fp8(y):
    """bf16 values [n, 512] as the FP8 cache holds them: tiles of 128, each
    with the smallest power of two that brings its values to at most 448."""
    v = y.view(-1, DV // 128, 128)
    m, e = torch.frexp(v.abs().amax(-1))                       # largest = m * 2^e, 0.5 <= m < 1
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 31)   # 448 = 0.875 * 2^9
    scale = torch.where(m > 0, _pow2(k), 1.0).float()[..., None]
    return ((v / scale).to(torch.float8_e4m3fn).float() * scale).reshape(y.shape)


def _plain_norm_rope(s):
    pos = s["positions"].long()
    live = pos >= 0
    table = s["cos_sin"][pos.clamp(min=0)]
    cos, sin = table[:, :32], table[:, 32:]
    q, kv = s["q"].float(), s["kv"].double()
    top = q[..., :DV]
    if s["q_weight"] is not None:
        top = top * torch.rsqrt((top * top).mean(-1, keepdim=True) + s["eps"]) * s["q_weight"].float()
    q_out = torch.cat([top, _rotate(q[..., DV:], cos[:, None], sin[:, None], s["pairs"])], -1).bfloat16()
    # the latent row's values meet the borders of the cache's codes: in 64 bits up to their rounding to bf16
    top = kv[:, :DV]
    y = _to_bf16(top * torch.rsqrt((top * top).mean(-1, keepdim=True) + s["eps"]) * s["kv_weight"].double())
    if s["format"] == "fp4":
        y = _stored_fp4(y, s["kv_scale"])
    elif s["format"] == "fp8":
        y = _stored_fp8(y)
    kv_out = torch.cat([y, _rotate(kv[:, DV:].float(), cos, sin, s["pairs"])], -1).bfloat16()
    return torch.where(live[:, None, None], q_out, s["q_out"]), torch.where(live[:, None], kv_out, s["kv_out"])


def _plain_grad(x, dy, w, eps, cos, sin, live, pairs):
    """dx and dw of one operand: x [..., 576], dy fp32, w [512] or None."""
    x, dy = x.float(), dy * live
    top, g = x[..., :DV], dy[..., :DV]
    dw = None
    if w is not None:
        r = torch.rsqrt((top * top).mean(-1, keepdim=True) + eps)
        xhat = top * r
        dw = (g * xhat).flatten(0, -2).sum(0, dtype=torch.float64).float()
        g = g * w.float()
        g = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return torch.cat([g, _rotate(dy[..., DV:], cos, sin, pairs, back=True)], -1).bfloat16(), dw


def _plain_norm_rope_bwd(s):
    pos = s["positions"].long()
    table = s["cos_sin"][pos.clamp(min=0)]
    cos, sin = table[:, :32], table[:, 32:]
    live = (pos >= 0).float()[:, None]
    dq, dwq = _plain_grad(s["q"], s["dq"], s["q_weight"], s["eps"], cos[:, None], sin[:, None], live[:, None],
                          s["pairs"])
    dkv, dwkv = _plain_grad(s["kv"], s["dkv"], s["kv_weight"], s["eps"], cos, sin, live, s["pairs"])
    return [x for x in (dq, dkv, dwq, dwkv) if x is not None]


def _plain_decode(s):
    b, sn, h, _ = s["q"].shape
    page = s["kv_cache"].shape[1]
    idx = s["indices"].long()
    keep = (idx >= 0) & (idx < s["cache_seqlens"].long()[:, None, None])
    idx = torch.where(keep, idx, 0)
    blk = torch.gather(s["block_table"].long(), 1, (idx // page).view(b, -1)).view(idx.shape)
    slot = s["kv_cache"].view(-1, FP4_SLOT)[blk * page + idx % page]     # [b, sn, topk, 416]
    codes = torch.stack([slot[..., :256] & 15, slot[..., :256] >> 4], -1).flatten(-2)
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")[codes.int()]
    scale = slot[..., 256:288].contiguous().view(torch.float8_e4m3fn).float() * s["kv_scale"]
    lat = (value.unflatten(-1, (32, 16)) * scale[..., None]).flatten(-2)
    row = torch.cat([lat, slot[..., 288:].contiguous().view(torch.bfloat16).float()], -1)
    score = torch.matmul(s["q"].float(), row.transpose(-1, -2)) * s["sm_scale"]
    score = score.masked_fill(~keep[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, row[..., :DV]) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))
    return out.bfloat16(), lse[..., 0]


def run(state):
    s = state
    if own:
        import serving_sparse_mla_gb300 as smla
        if s["op"] == "norm_rope":
            return smla.mla_norm_rope(s["q"], s["kv"], s["positions"], s["cos_sin"], q_weight=s["q_weight"],
                                      kv_weight=s["kv_weight"], eps=s["eps"], interleaved=s["pairs"],
                                      kv_cache=s["kv_cache"], slots=s["slots"], kv_scale=s["kv_scale"],
                                      q_out=s["q_out"], kv_out=s["kv_out"])
        if s["op"] == "norm_rope_bwd":
            got = smla.mla_norm_rope_bwd(s["q"], s["kv"], s["positions"], s["cos_sin"], s["dq"], s["dkv"],
                                         q_weight=s["q_weight"], kv_weight=s["kv_weight"], eps=s["eps"],
                                         interleaved=s["pairs"])
            return [x for x in got if x is not None]
        return smla.sparse_mla_decode_fp4(s["q"], s["kv_cache"], s["block_table"], s["cache_seqlens"], s["indices"],
                                          s["sm_scale"], kv_scale=s["kv_scale"])
    if s["op"] == "norm_rope":
        return _plain_norm_rope(s)
    if s["op"] == "norm_rope_bwd":
        return _plain_norm_rope_bwd(s)
    return _plain_decode(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "decode_fp4":
        n, h = case["batch"] * case["s_next"], case["heads"]
        seen = rows = 0.0
        for i in range(16):   # contexts are uniform in [lo, hi]
            length = case["lo"] + (case["hi"] - case["lo"]) * (i + 0.5) / 16
            used = min(case["topk"], length)
            seen += used / 16
            # slots that at least one of the request's lists names
            rows += length * (1 - (1 - used / length) ** case["s_next"]) / 16
        return {"bytes": case["batch"] * rows * FP4_SLOT + n * (4 * case["topk"] + h * (2 * D + 2 * DV + 4)),
                "flops": 2.0 * n * h * seen * (D + DV)}
    t, h = case["tokens"], case["heads"]
    live = t - case["pad"]
    if case["op"] == "norm_rope":
        slot = {"bf16": 2 * D, "fp8": FP8_SLOT, "fp4": FP4_SLOT}[case["cache"]]
        return {"bytes": live * ((h + 1) * 4 * D + slot + 4 * DR) + 8 * t, "flops": live * (h + 1) * 6.0 * D}
    # x where a norm needs it, dy, dx
    read = live * ((h if case["q_norm"] else 0) + 1) * 2 * D + live * (h + 1) * 4 * D
    return {"bytes": read + t * (h + 1) * 2 * D + live * 4 * DR + 4 * t, "flops": live * (h + 1) * 12.0 * D}


# ------------------------------------------------------------------ the definition in 64 bits

def _turned(x, cs, pairs, sign):
    """One rotation, complex: value a + ib of a pair times cos + i sign sin."""
    lo, hi = (slice(0, DR, 2), slice(1, DR, 2)) if pairs else (slice(0, 32), slice(32, DR))
    z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(cs[..., :32], sign * cs[..., 32:])
    out = torch.empty_like(x)
    out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _exact_quantized(y, form, g):
    """Nearest representable values, by trying every code's value."""
    if form == "bf16":
        return y
    if form == "fp8":
        grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        t = y.reshape(-1, 128)
        powers = torch.tensor([2.0 ** k for k in range(-64, 32)], dtype=torch.float64, device="cuda")
        k = torch.searchsorted(powers * 448, t.abs().amax(1)).clamp(max=95)
        step = torch.where(t.abs().amax(1) > 0, powers[k], 1.0)[:, None]
    else:
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        t = y.reshape(-1, 16)
        scales = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        step = _nearest(_over(t.abs().amax(1), 6 * g).clamp(2.0 ** -9, 448), scales)[:, None] * g
    return (torch.sign(t) * _nearest(t.abs() / step, grid) * step).reshape(y.shape)


def _nearest(x, grid):
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    below, above = grid[hi - 1], grid[hi]
    down = (x - below < above - x) | ((x - below == above - x) & (hi % 2 == 1))
    return torch.where(down, below, above)


def _eight_bits(y):
    """The nearest number of 8 significant bits (bf16), ties to even, on the bits of a float64."""
    bits = y.view(torch.int64)
    return ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) >> 45 << 45).view(torch.float64)


def _exact_norm(case, s):
    live = (s["positions"] >= 0)
    cs = s["cos_sin"].double()[s["positions"].clamp(min=0).long()]

    def rows(x, w, c, form):
        x = x.double()
        lat = x[..., :DV]
        if w is not None:
            lat = lat / torch.sqrt(lat.square().sum(-1, keepdim=True) / DV + s["eps"]) * w.double()
        if form is not None:
            lat = _exact_quantized(_eight_bits(lat), form, case["kv_scale"])
        return torch.cat([lat, _turned(x[..., DV:].contiguous(), c, case["pairs"], 1.0)], -1)

    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for at in range(0, case["tokens"], 512):
        q[at:at + 512] = rows(s["q"][at:at + 512], s["q_weight"], cs[at:at + 512, None], None)
    kv = rows(s["kv"], s["kv_weight"], cs, case["cache"])
    return q * live[:, None, None], kv * live[:, None]


def _exact_grad(case, s):
    """The vector-Jacobian product, row by row blocks, from d(x / |x|)."""
    live = (s["positions"] >= 0)
    cs = s["cos_sin"].double()[s["positions"].clamp(min=0).long()]

    def back(x, dy, w, c):
        x, dy = x.double(), dy.double()
        if w is None:
            return torch.cat([dy[..., :DV], _turned(dy[..., DV:].contiguous(), c, case["pairs"], -1.0)], -1), None
        lat, g = x[..., :DV], dy[..., :DV]
        size = torch.sqrt(lat.square().sum(-1, keepdim=True) / DV + s["eps"])
        gw = g * w.double()
        d = gw / size - lat * (gw * lat).sum(-1, keepdim=True) / (DV * size ** 3)
        return (torch.cat([d, _turned(dy[..., DV:].contiguous(), c, case["pairs"], -1.0)], -1),
                (g * lat / size).reshape(-1, DV).sum(0))

    dq = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    dwq = None if s["q_weight"] is None else torch.zeros(DV, dtype=torch.float64, device="cuda")
    for at in range(0, case["tokens"], 512):
        part = slice(at, at + 512)
        d, w = back(s["q"][part], s["dq"][part] * live[part, None, None], s["q_weight"], cs[part, None])
        dq[part] = d
        if w is not None:
            dwq += w
    dkv, dwkv = back(s["kv"], s["dkv"] * live[:, None], s["kv_weight"], cs)
    return [x for x in (dq, dkv, dwq, dwkv) if x is not None]


def _exact_decode(case, s):
    q = s["q"].double()
    b, sn, h, _ = q.shape
    page = case["page"]
    signed = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    out = torch.zeros(b, sn, h, DV, dtype=torch.float64, device="cuda")
    lse = torch.full((b, sn, h), -math.inf, dtype=torch.float64, device="cuda")
    lens, lists = s["cache_seqlens"].tolist(), s["indices"].long()
    slots = s["kv_cache"].view(-1, FP4_SLOT)
    for r in range(b):
        at = torch.arange(lens[r], device="cuda")
        mem = slots[s["block_table"][r].long()[at // page] * page + at % page]
        kv = torch.empty(lens[r], D, dtype=torch.float64, device="cuda")
        kv[:, 0:DV:2] = signed[(mem[:, :256] % 16).long()]
        kv[:, 1:DV:2] = signed[(mem[:, :256] // 16).long()]
        kv[:, :DV] *= mem[:, 256:288].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        kv[:, :DV] *= case["kv_scale"]
        kv[:, DV:] = mem[:, 288:].contiguous().view(torch.bfloat16).double()
        for j in range(sn):
            n = lists[r, j]
            n = n[(n >= 0) & (n < lens[r])]
            if n.numel():
                z = kv[n] @ q[r, j].T * s["sm_scale"]
                lse[r, j] = torch.logsumexp(z, 0)
                out[r, j] = torch.softmax(z, 0).T @ kv[n, :DV]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm, "norm_rope_bwd": _exact_grad, "decode_fp4": _exact_decode}[case["op"]](case, s)
