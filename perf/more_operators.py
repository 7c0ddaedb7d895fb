"""Cases of the operators around a layer's dense attention, with their plain forms.

Four operators:

* ``mla_add_norm``: the residual's addition, the RMS norm of the sum and, where
  asked for, its output as e4m3 codes with a power-of-two scale for each 128
  values or each row.
* ``mla_add_norm_bwd``: its gradients.
* ``dense_mha_fwd``: causal attention over whole prompts in the heads' own
  space (query and key heads of 192 or 128 values, value heads of 128), packed
  sequences of different lengths, query heads in groups that share a key and
  value head.  The queries of a sequence are its last positions.
* ``dense_mha_bwd``: its gradients.
"""
import math
import random

import torch

own = False

GROUP = 128          # values under one scale
LARGEST = 448.0      # of e4m3


# ------------------------------------------------------------------ cases

def _norm(name, rows, width, form, residual=True):
    return {"name": name, "op": "add_norm", "rows": rows, "width": width, "form": form, "residual": residual}


def _norm_grad(name, rows, width, residual=True):
    return {"name": name, "op": "add_norm_bwd", "rows": rows, "width": width, "residual": residual}


def _attn(name, op, d_qk, heads, kv_heads, batch, lo, hi, back_lo=0, back_hi=0, tail=0):
    """`batch` sequences of lo to hi queries, each behind back_lo to back_hi earlier positions (fewer than none:
    its first queries see nothing), and `tail` rows behind the last one."""
    return {"name": name, "op": op, "d_qk": d_qk, "heads": heads, "kv_heads": kv_heads, "batch": batch, "lo": lo,
            "hi": hi, "back_lo": back_lo, "back_hi": back_hi, "tail": tail}


def listed():
    return [
        # one new token of one request: latency alone counts
        _norm("norm one token, groups", 1, 7168, "group"),
        # an odd batch at an odd width, one scale a row
        _norm("norm 333 x 1544, rows", 333, 1544, "row"),
        # the mid prefill, its rows kept in 16 bits
        _norm("norm 2119 x 5120, 16 bits", 2119, 5120, "bf16"),
        # a long prefill that feeds 8-bit products
        _norm("norm 8192 x 7168, groups", 8192, 7168, "group"),
        # a small training batch, the first layer's norm (no gradient of a later sum)
        _norm_grad("norm grad 257 x 2048", 257, 2048, residual=False),
        # a training step's tokens
        _norm_grad("norm grad 8192 x 7168", 8192, 7168),
        # the last token of a prompt whose other rows are there already, 8 tensor-parallel heads
        _attn("attention one token", "dense_fwd", 192, 8, 8, 1, 1, 1, 5000, 5000),
        # packed prompts of very different lengths, some behind a cached prefix, grouped heads
        _attn("attention packed, 32 heads on 8", "dense_fwd", 128, 32, 8, 15, 3, 2000, -20, 1500, tail=9),
        # the wide-head prefill: one prompt of 8192 tokens at 64 heads
        _attn("attention 8192, 64 heads", "dense_fwd", 192, 64, 64, 1, 8192, 8192),
        # a small training batch of short texts
        _attn("attention grad short, 8 heads", "dense_bwd", 192, 8, 8, 5, 1, 130, tail=3),
        # packed training texts, grouped heads
        _attn("attention grad packed, 40 heads on 8", "dense_bwd", 128, 40, 8, 9, 40, 2119),
        # one text of 8192 tokens
        _attn("attention grad 8192, 32 heads", "dense_bwd", 192, 32, 32, 1, 8192, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("add_norm", "add_norm_bwd", "dense_fwd", "dense_fwd", "dense_bwd"))
    if op.startswith("add_norm"):
        width = 8 * _log(rng, 16, 1024)
        case = {"op": op, "rows": _log(rng, 1, 8192 * 7168 // max(width, 2048)), "width": width,
                "residual": rng.random() < 0.7}
        if op == "add_norm":
            case["form"] = rng.choice(("bf16", "group", "group", "row"))
        return case
    kv_heads = rng.choice((1, 2, 4, 8, 8, 32))
    heads = kv_heads * rng.choice((1, 1, 2, 4, 5, 8) if kv_heads < 32 else (1, 2))
    most = (64 if op == "dense_fwd" else 32) * 8192 ** 2
    hi = _log(rng, 1, 8192)
    ahead = op == "dense_fwd" and rng.random() < 0.6
    back_hi = _log(rng, 1, 8192) if ahead else 0
    batch = max(1, min(_log(rng, 1, 40), most // (heads * hi * (hi + back_hi))))
    while heads * hi * (hi + back_hi) > most:
        hi = (hi + 1) // 2
    lo = rng.choice((0, 1, hi, max(1, hi // 8)))
    return {"op": op, "d_qk": rng.choice((192, 128)), "heads": heads, "kv_heads": kv_heads, "batch": batch,
            "lo": min(lo, hi), "hi": hi, "back_lo": rng.choice((-3, 0, back_hi)) if ahead else rng.choice((0, 0, -2)),
            "back_hi": back_hi, "tail": rng.choice((0, 0, 5))}


def _lengths(case):
    """Query and key rows of each sequence of a case."""
    r = random.Random(case["batch"] * 1000003 + case["hi"] * 1009 + case["lo"] * 31 + case["back_hi"])
    q = [case["hi"] if i == 0 else min(case["hi"], max(case["lo"], _log(r, max(case["lo"], 1), max(case["hi"], 1))))
         for i in range(case["batch"])]
    r.shuffle(q)
    return q, [max(0, n + r.randint(case["back_lo"], case["back_hi"])) for n in q]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_norm(case, seed):
    g = _gen(seed)
    n, d = case["rows"], case["width"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    # channels of unequal size, a few of them large, as a residual stream has them
    size = torch.exp(0.7 * randn(d))
    s = {"op": case["op"], "eps": 1e-6, "weight": (1 + 0.2 * randn(d)).bfloat16()}
    if case["op"] == "add_norm":
        s["x"] = (randn(n, d) * 0.3).bfloat16()
        s["residual"] = (randn(n, d) * size).bfloat16() if case["residual"] else None
        s["form"] = case["form"]
    else:
        s["z"] = (randn(n, d) * size).bfloat16()
        s["dout"] = (randn(n, d) * 0.01).bfloat16()
        s["dresidual"] = (randn(n, d) * 0.01).bfloat16() if case["residual"] else None
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    h, hk, d = case["heads"], case["kv_heads"], case["d_qk"]
    lq, lk = _lengths(case)
    tq, tk = sum(lq) + case["tail"], sum(lk) + case["tail"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    offsets = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"op": case["op"], "scale": d ** -0.5, "cu_q": offsets(lq), "cu_kv": offsets(lk), "most_q": max(lq),
         "most_kv": max(lk)}
    # scores of a few units, so that rows are neither even nor one key's alone
    s["q"] = (randn(tq, h, d) * 1.5).bfloat16()
    s["k"] = (randn(tk, hk, d) * torch.exp(0.3 * randn(d))).bfloat16()
    s["v"] = randn(tk, hk, 128).bfloat16()
    if case["op"] == "dense_bwd":
        s["out"], s["lse"] = _plain_attn(s)
        s["dout"] = (randn(tq, h, 128) * 0.1).bfloat16()
    return s


def prepare(case, seed):
    return _prepare_norm(case, seed) if case["op"].startswith("add_norm") else _prepare_attn(case, seed)


# ------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in float64 from its bits (torch's own powers of two are not all exact on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_bf16(y):
    """float64 rounded once to bf16 values (8 significant bits, ties to even)."""
    m, e = torch.frexp(y)
    return (torch.round(m * 256) * _pow2(e - 8)).float()


def _quantized(y, size):
    """e4m3 codes of bf16 values [n, d] and the scale of each `size` of a row: the smallest power of two that
    brings the largest of them to at most 448."""
    n, d = y.shape
    t = torch.nn.functional.pad(y, (0, -d % size)).view(n, -1, size)
    m, e = torch.frexp(t.abs().amax(-1))                       # largest = m * 2^e, 0.5 <= m < 1
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 31)   # 448 = 0.875 * 2^9
    scale = torch.where(m > 0, _pow2(k), 1.0).float()
    return (t / scale[..., None]).view(n, -1)[:, :d].to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    z = s["x"]
    if s["residual"] is not None:
        z = (z.float() + s["residual"].float()).bfloat16()
    # where codes follow, in 64 bits up to the rounding to bf16: values meet the codes' borders
    x = z.float() if s["form"] == "bf16" else z.double()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"].to(x.dtype)
    got = [y.bfloat16()] if s["form"] == "bf16" else _quantized(_to_bf16(y), GROUP if s["form"] == "group"
                                                               else z.shape[1])
    return list(got) + ([z] if s["residual"] is not None else [])


def _plain_norm_bwd(s):
    x, dy = s["z"].float(), s["dout"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    xhat = x * r
    dw = (dy * xhat).sum(0, dtype=torch.float64).float()
    g = dy * s["weight"].float()
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return dx.bfloat16(), dw


def _rows(cu, most, total):
    """The row of position i of sequence b, [b, most], and whether there is one (else row `total`)."""
    at = torch.arange(most, device="cuda")
    live = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None].long() + at, total), live


def _spread(x, rows):
    """Rows of x [total, h, d] as [b, h, most, d] fp32, zeros where there is none."""
    x = torch.cat([x, torch.zeros_like(x[:1])])
    return x[rows].float().transpose(1, 2)


def _scores(s):
    """Queries [b, kv, g, i, d], keys and values [b, kv, 1, j, d], scores with -inf where a key is not seen."""
    h, hk = s["q"].shape[1], s["k"].shape[1]
    rq, live = _rows(s["cu_q"], s["most_q"], s["q"].shape[0])
    rk, key = _rows(s["cu_kv"], s["most_kv"], s["k"].shape[0])
    q = _spread(s["q"], rq).unflatten(1, (hk, h // hk))
    k, v = _spread(s["k"], rk)[:, :, None], _spread(s["v"], rk)[:, :, None]
    ahead = (s["cu_kv"][1:] - s["cu_kv"][:-1] - s["cu_q"][1:] + s["cu_q"][:-1])[:, None, None]
    i, j = torch.arange(s["most_q"], device="cuda")[:, None], torch.arange(s["most_kv"], device="cuda")
    hidden = ~((j <= i + ahead) & key[:, None] & live[:, :, None])
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    return q, k, v, z.masked_fill_(hidden[:, None, None], -math.inf), rq, rk


def _gather(x, rows, total, fill=0.0):
    """[b, kv, g, i, ...] back as rows [total, kv * g, ...]; `fill` in rows of no sequence."""
    x = x.flatten(1, 2).transpose(1, 2)
    out = torch.full((total + 1,) + x.shape[2:], fill, dtype=x.dtype, device="cuda")
    out[rows] = x
    return out[:total]


def _plain_attn(s):
    q, k, v, z, rq, _ = _scores(s)
    if s["most_kv"] == 0:
        top = torch.full_like(z.sum(-1, keepdim=True), -math.inf)
    else:
        top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))[..., 0]
    n = s["q"].shape[0]
    return _gather(out, rq, n).bfloat16(), _gather(lse, rq, n, -math.inf)


def _plain_attn_bwd(s):
    q, k, v, z, rq, rk = _scores(s)
    hk, g = q.shape[1:3]
    back = lambda x: _spread(x, rq).unflatten(1, (hk, g))  # noqa: E731
    do, o, lse = back(s["dout"]), back(s["out"]), back(s["lse"][..., None])
    p = z.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    n, m = s["q"].shape[0], s["k"].shape[0]
    return _gather(dq, rq, n).bfloat16(), _gather(dk, rk, m).bfloat16(), _gather(dv, rk, m).bfloat16()


def run(state):
    s = state
    if own:
        import serving_sparse_mla_gb300 as smla
        if s["op"] == "add_norm":
            group = {"bf16": None, "group": GROUP, "row": 0}[s["form"]]
            got = smla.mla_add_norm(s["x"], s["weight"], s["residual"], eps=s["eps"], group=group)
            # the rows that came out, their scales where there are any, and the sum where there was one
            return [got[0]] + ([got[1]] if group is not None else []) + ([got[2]] if s["residual"] is not None else [])
        if s["op"] == "add_norm_bwd":
            return smla.mla_add_norm_bwd(s["z"], s["weight"], s["dout"], s["dresidual"], eps=s["eps"])
        if s["op"] == "dense_fwd":
            return smla.dense_mha_fwd(s["q"], s["k"], s["v"], s["scale"], s["cu_q"], s["cu_kv"])
        return smla.dense_mha_bwd(s["q"], s["k"], s["v"], s["scale"], s["out"], s["lse"], s["dout"], s["cu_q"],
                                  s["cu_kv"])
    return {"add_norm": _plain_norm, "add_norm_bwd": _plain_norm_bwd, "dense_fwd": _plain_attn,
            "dense_bwd": _plain_attn_bwd}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"].startswith("add_norm"):
        n, d = case["rows"], case["width"]
        if case["op"] == "add_norm_bwd":   # z, dout and the later gradient read, dx written
            return {"bytes": n * d * (8 if case["residual"] else 6) + 6 * d, "flops": 12.0 * n * d}
        out = {"bf16": 2 * d, "group": d + 4 * (-(-d // GROUP)), "row": d + 4}[case["form"]]
        return {"bytes": n * (out + d * (6 if case["residual"] else 2)) + 2 * d, "flops": 6.0 * n * d}
    h, hk, d, tail = case["heads"], case["kv_heads"], case["d_qk"], case["tail"]
    lq, lk = _lengths(case)
    pairs = 0
    for a, b in zip(lq, lk):   # query i of a sees keys 0 .. i + b - a
        first = max(0, a - b)
        n = a - first
        pairs += n * (first + b - a + 1) + n * (n - 1) // 2
    q, k = sum(lq), sum(lk)
    rows_q, rows_k = (q + tail) * h, (k + tail) * hk
    if case["op"] == "dense_fwd":
        return {"bytes": 2 * q * h * d + 2 * k * hk * (d + 128) + rows_q * (2 * 128 + 4),
                "flops": 2.0 * pairs * h * (d + 128)}
    return {"bytes": q * h * (2 * d + 4 * 128 + 4) + 2 * k * hk * (d + 128) + 2 * rows_q * d + 2 * rows_k * (d + 128),
            "flops": 2.0 * pairs * h * (3 * d + 2 * 128)}


# ------------------------------------------------------------------ the definition in 64 bits

def _eight_bits(y):
    """The nearest number of 8 significant bits (bf16), ties to even, on the bits of a float64."""
    bits = y.view(torch.int64)
    return ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) >> 45 << 45).view(torch.float64)


def _nearest(x, grid):
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    below, above = grid[hi - 1], grid[hi]
    down = (x - below < above - x) | ((x - below == above - x) & (hi % 2 == 1))
    return torch.where(down, below, above)


def _exact_norm(case, s):
    z = s["x"].double()
    if case["residual"]:
        z = _eight_bits(z + s["residual"].double())
    y = z / torch.sqrt(z.square().sum(-1, keepdim=True) / case["width"] + s["eps"]) * s["weight"].double()
    tail = [z] if case["residual"] else []
    if case["form"] == "bf16":
        return [y] + tail
    y = _eight_bits(y)
    grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    powers = torch.tensor([2.0 ** k for k in range(-64, 32)], dtype=torch.float64, device="cuda")
    codes, scales = torch.empty_like(y), []
    for at in range(0, case["width"], GROUP if case["form"] == "group" else case["width"]):
        part = slice(at, at + GROUP) if case["form"] == "group" else slice(None)
        t = y[:, part]
        k = torch.searchsorted(powers * LARGEST, t.abs().amax(1)).clamp(max=95)
        scales.append(torch.where(t.abs().amax(1) > 0, powers[k], 1.0))
        codes[:, part] = torch.sign(t) * _nearest(t.abs() / scales[-1][:, None], grid)
    return [codes, torch.stack(scales, 1)] + tail


def _exact_norm_bwd(case, s):
    """The vector-Jacobian product, from d(z / |z|)."""
    z, g = s["z"].double(), s["dout"].double()
    size = torch.sqrt(z.square().sum(-1, keepdim=True) / case["width"] + s["eps"])
    gw = g * s["weight"].double()
    dx = gw / size - z * (gw * z).sum(-1, keepdim=True) / (case["width"] * size ** 3)
    if case["residual"]:
        dx += s["dresidual"].double()
    return dx, (g * z / size).sum(0)


def _exact_heads(case, s):
    """(sequence's rows, keys' rows, head, key head, weights [rows, keys]) of every head of every sequence, the rows
    that see something alone."""
    lq, lk = _lengths(case)
    share = case["heads"] // case["kv_heads"]
    at_q = at_k = 0
    for a, b in zip(lq, lk):
        first = max(0, a - b)
        rows, keys = slice(at_q + first, at_q + a), slice(at_k, at_k + b)
        at_q, at_k = at_q + a, at_k + b
        if a <= first or b == 0:
            continue
        hide = torch.ones(a - first, b, dtype=torch.bool, device="cuda").triu(b - a + first + 1)
        for h in range(case["heads"]):
            z = s["q"][rows, h].double() @ s["k"][keys, h // share].double().T * s["scale"]
            z[hide] = -math.inf
            yield rows, keys, h, h // share, z


def _exact_attn(case, s):
    out = torch.zeros(s["q"].shape[:2] + (128,), dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for rows, keys, h, kh, z in _exact_heads(case, s):
        lse[rows, h] = torch.logsumexp(z, 1)
        out[rows, h] = torch.softmax(z, 1) @ s["v"][keys, kh].double()
    return out, lse


def _exact_attn_bwd(case, s):
    """From the inputs alone: the weights and the output they give in 64 bits, not the rounded ones that a pass gets."""
    dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v"))
    for rows, keys, h, kh, z in _exact_heads(case, s):
        p, do, v = torch.softmax(z, 1), s["dout"][rows, h].double(), s["v"][keys, kh].double()
        dp = do @ v.T
        ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
        dq[rows, h] = ds @ s["k"][keys, kh].double()
        dk[keys, kh] += ds.T @ s["q"][rows, h].double()
        dv[keys, kh] += p.T @ do
    return dq, dk, dv


def exact(case, seed):
    s = prepare(case, seed)
    return {"add_norm": _exact_norm, "add_norm_bwd": _exact_norm_bwd, "dense_fwd": _exact_attn,
            "dense_bwd": _exact_attn_bwd}[case["op"]](case, s)
