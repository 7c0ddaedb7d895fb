"""Pins of the residual norm's and the dense attention's oracles (CPU): closed
forms, library routines and differences."""
import math

import numpy as np
import pytest
import torch

from oracle import add_norm_oracle as ano
from oracle import dense_mha_oracle as dmo


def _t(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64)


def test_norm_of_equal_values_is_the_weight():
    z = np.full((2, 24), 3.0)
    assert np.allclose(ano.norm(z, np.arange(24.0), 0.0), np.arange(24.0))


def test_codes_agree_with_torch_and_scales_are_least():
    rng = np.random.default_rng(1)
    y = torch.from_numpy(rng.standard_normal((5, 200)) * np.exp(rng.standard_normal((5, 1)) * 6)).bfloat16()
    y[2, :128] = 0
    v, s = ano.codes(y.double().numpy(), 128)
    assert s.shape == (5, 2) and s[2, 0] == 1.0
    for g in range(2):
        part = y[:, 128 * g:128 * g + 128].float() / torch.from_numpy(s[:, g:g + 1]).float()
        assert torch.equal(part.to(torch.float8_e4m3fn).double(), torch.from_numpy(v[:, 128 * g:128 * g + 128]))
        top = part.abs().amax(1)
        assert (top <= 448).all() and ((top > 224) | (top == 0)).all()


def test_norm_gradients_are_autograds():
    g = torch.Generator().manual_seed(2)
    z, w, do, dr = _t(g, 4, 24).requires_grad_(), _t(g, 24).requires_grad_(), _t(g, 4, 24), _t(g, 4, 24)
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 0.1) * w
    ((y * do).sum() + (z * dr).sum()).backward()
    dx, dw, _, _ = ano.grads(z.detach().numpy(), w.detach().numpy(), 0.1, do.numpy(), dr.numpy())
    assert np.allclose(dx, z.grad) and np.allclose(dw, w.grad)


def _packed(seed, lq, lk, h, hk, d, tail=0):
    g = torch.Generator().manual_seed(seed)
    cu = [torch.tensor([sum(x[:i]) for i in range(len(x) + 1)], dtype=torch.int32) for x in (lq, lk)]
    q, k, v = _t(g, sum(lq) + tail, h, d), _t(g, sum(lk) + tail, hk, d), _t(g, sum(lk) + tail, hk, 6)
    return q, k, v, cu[0], cu[1], _t(g, sum(lq) + tail, h, 6)


def test_one_sequence_is_the_librarys_causal_attention():
    q, k, v, *_ = _packed(3, [7], [7], 4, 2, 10)
    out, lse, _, _ = dmo.fwd(q, k, v, 0.3)
    rep = lambda x: x.repeat_interleave(2, 1).transpose(0, 1)  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), rep(k), rep(v), is_causal=True, scale=0.3)
    assert torch.allclose(out, ref.transpose(0, 1))
    assert torch.allclose(lse[0], (q[0] * rep(k)[:, 0]).sum(-1) * 0.3)   # a first row sees one key


def test_packed_sequences_are_their_parts_and_rows_without_keys_are_empty():
    q, k, v, cq, ck, _ = _packed(4, [3, 0, 5, 2], [6, 4, 2, 0], 2, 1, 8, tail=2)
    out, lse, _, _ = dmo.fwd(q, k, v, 0.2, cq, ck)
    a, b, _, _ = dmo.fwd(q[:3], k[:6], v[:6], 0.2)
    assert torch.equal(out[:3], a) and torch.equal(lse[:3], b)
    assert torch.equal(lse[0, 0], torch.logsumexp((q[0, 0] @ k[:4, 0].T) * 0.2, 0))   # 6 - 3 positions before it
    # the third has 5 queries and 2 keys: its first 3 rows see nothing; the last and the tail have no keys
    empty = [3, 4, 5, 8, 9, 10, 11]
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all() and torch.isfinite(lse[6:8]).all()


def test_gradients_are_differences():
    q, k, v, cq, ck, do = _packed(5, [3, 4], [5, 2], 4, 2, 6, tail=1)
    out, lse, _, _ = dmo.fwd(q, k, v, 0.4, cq, ck)
    grads, bounds = dmo.bwd(q, k, v, 0.4, out, lse, do, cq, ck)
    f = lambda: (dmo.fwd(q, k, v, 0.4, cq, ck)[0] * do).sum().item()  # noqa: E731
    rng = np.random.default_rng(6)
    for t, g in zip((q, k, v), grads):
        flat = t.view(-1)
        for i in rng.choice(flat.numel(), 20, replace=False):
            x = flat[i].item()
            flat[i] = x + 1e-5
            up = f()
            flat[i] = x - 1e-5
            down = f()
            flat[i] = x
            assert (up - down) / 2e-5 == pytest.approx(g.view(-1)[i].item(), abs=1e-7)
    assert all((b >= 2.0 ** -8 * g.abs()).all() for g, b in zip(grads, bounds))
    assert (grads[0][7:] == 0).all() and (grads[1][7:] == 0).all()


def test_a_dropped_key_leaves_the_bound():
    """The parity bound sees one key missing from rows of 300."""
    q, k, v, *_ = _packed(7, [300], [300], 1, 1, 64)
    out, lse, size, _ = dmo.fwd(q, k, v, 0.125)
    z = (q[:, 0] @ k[:, 0].T * 0.125).masked_fill(torch.ones(300, 300).triu(1).bool(), -math.inf)
    z[:, 17] = -math.inf
    off = torch.softmax(z[20:], 1) @ v[:, 0]
    assert (off - out[20:, 0]).norm() > 4 * 2.0 ** -8 * out[20:, 0].norm()
