"""Float64 oracle of dense causal attention over packed sequences and its
gradients, on torch tensors of any device, one head of one sequence at a
time.  Beside each result stand the sums of its terms' magnitudes, from which
the parity tests derive their bounds."""
import math

import torch


def sequences(cu, total):
    """[(first, end)] rows of each sequence; offsets cut to the tensor."""
    if cu is None:
        return [(0, total)]
    c = [min(max(int(x), 0), total) for x in cu]
    return [(a, max(a, b)) for a, b in zip(c[:-1], c[1:])]


def heads(q, k, v, scale, cu_q, cu_kv):
    """(rows, keys, head, key head, scores with -inf where hidden, sum of the
    score's terms' magnitudes) of every head of every sequence that has both."""
    share = q.shape[1] // k.shape[1]
    for (q0, q1), (k0, k1) in zip(sequences(cu_q, q.shape[0]), sequences(cu_kv, k.shape[0])):
        lq, lk = q1 - q0, k1 - k0
        if lq == 0 or lk == 0:
            continue
        i = torch.arange(lq, device=q.device)[:, None]
        hidden = torch.arange(lk, device=q.device)[None] > i + (lk - lq)
        for h in range(q.shape[1]):
            a, b = q[q0:q1, h].double(), k[k0:k1, h // share].double()
            z = (a @ b.T * scale).masked_fill(hidden, -math.inf)
            yield slice(q0, q1), slice(k0, k1), h, h // share, z, a.abs() @ b.abs().T * scale


def weights(z, lse):
    """exp(z - lse), zero in rows that see nothing."""
    return torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None]).masked_fill(z == -math.inf, 0.0)


def fwd(q, k, v, scale, cu_q=None, cu_kv=None):
    """(out, lse, sum p |v|, largest sum of a score's terms per row) in float64;
    rows that see nothing, or belong to no sequence: 0 and -inf."""
    n, h = q.shape[:2]
    out = torch.zeros(n, h, v.shape[2], dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=q.device)
    terms = torch.zeros(n, h, dtype=torch.float64, device=q.device)
    for rows, keys, j, kj, z, az in heads(q, k, v, scale, cu_q, cu_kv):
        lse[rows, j] = torch.logsumexp(z, 1)
        p = weights(z, lse[rows, j])
        w = v[keys, kj].double()
        out[rows, j], size[rows, j] = p @ w, p @ w.abs()
        terms[rows, j] = az.masked_fill(z == -math.inf, 0.0).amax(1)
    return out, lse, size, terms


def bwd(q, k, v, scale, out, lse, dout, cu_q=None, cu_kv=None, unit=2.0 ** -8, score=2.0 ** -16):
    """(dq, dk, dv) from the given out and lse, and for each the bound on what
    rounding the factors P and dS to `unit` of themselves, and sums to `score`
    of their terms' magnitudes, may change."""
    grads = [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v)]
    bounds = [torch.zeros_like(g) for g in grads]
    for rows, keys, j, kj, z, az in heads(q, k, v, scale, cu_q, cu_kv):
        a, b, w = q[rows, j].double(), k[keys, kj].double(), v[keys, kj].double()
        do, o = dout[rows, j].double(), out[rows, j].double()
        p = weights(z, lse[rows, j].double())
        dp, d = do @ w.T, (do * o).sum(1, keepdim=True)
        ds = p * (dp - d) * scale
        # a score off by `score` of its terms moves p by as much of itself; dp and d are sums of products
        ep = p * score * (az + 1.0)
        es = ep * (dp - d).abs() * scale + p * score * (do.abs() @ w.abs().T + (do * o).abs().sum(1, keepdim=True)) * scale
        grads[0][rows, j] = ds @ b
        grads[1][keys, kj] += ds.T @ a
        grads[2][keys, kj] += p.T @ do
        es = es + unit * ds.abs()
        bounds[0][rows, j] = es @ b.abs()
        bounds[1][keys, kj] += es.T @ a.abs()
        bounds[2][keys, kj] += (ep + unit * p).T @ do.abs()
    return grads, [e + unit * g.abs() for e, g in zip(bounds, grads)]
