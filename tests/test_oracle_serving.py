"""Pins of the fp64 forms in oracle/serving.py: finite differences, torch's fp64 attention, and the
rotation's invariants."""
import numpy as np
import pytest
import torch

from oracle import serving as O


def rng(seed=0):
    return np.random.RandomState(seed)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32])
def test_gradients_are_those_of_differences(interleaved, rot):
    r = rng(rot + interleaved)
    x, w, dy = r.randn(3, 2, 32), 1 + 0.3 * r.randn(32), r.randn(3, 2, 32)
    pos, f = np.array([0, 5, 100003]), 1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))

    def loss(x, w):
        return (O.norm_rope(x, w, pos, f, 1e-3, interleaved) * dy).sum()

    dx, dw = O.norm_rope_backward(x, w, pos, f, 1e-3, dy, interleaved)
    h = 1e-5
    for _ in range(40):
        i = tuple(r.randint(s) for s in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
        c = r.randint(32)
        e = np.zeros(32)
        e[c] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    r = rng(3)
    f = 1e4 ** (-np.arange(16) / 16)
    a, b = r.randn(1, 1, 32), r.randn(1, 1, 32)
    turn = lambda x, p: O.rotate(x, np.array([p]), f, interleaved)  # noqa: E731
    assert np.allclose((turn(a, 77) ** 2).sum(), (a ** 2).sum())
    assert np.allclose((turn(a, 1000) * turn(b, 993)).sum(), (turn(a, 7) * b).sum())
    assert np.allclose(turn(turn(a, 12345), -12345), a)


def test_paged_attention_is_causal_attention_of_the_gathered_keys():
    r = rng(5)
    page, hkv, d, G = 4, 2, 8, 3
    kp, vp = r.randn(9, hkv, page, d), r.randn(9, hkv, page, d)
    table = np.array([[4, 2, 8], [0, 7, -1], [3, -1, -1]])
    kv_len, cu = np.array([11, 7, 2]), np.array([0, 5, 6, 6])
    q = r.randn(8, hkv * G, d)
    out, lse, dots, absv = O.paged_attention(q, kp, vp, cu, kv_len, table, 0.3)
    for row, b, pos in O.new_tokens(cu, kv_len):
        at = table[b][np.arange(pos + 1) // page]
        k = torch.from_numpy(kp[at, :, np.arange(pos + 1) % page]).transpose(0, 1).repeat_interleave(G, 0)
        v = torch.from_numpy(vp[at, :, np.arange(pos + 1) % page]).transpose(0, 1).repeat_interleave(G, 0)
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[row])[:, None], k, v, scale=0.3)[:, 0]
        assert np.allclose(out[row], ref.numpy())
        z = (k @ torch.from_numpy(q[row])[:, :, None])[..., 0] * 0.3
        assert np.allclose(lse[:, row], torch.logsumexp(z, -1).numpy())
    assert (out[6:] == 0).all() and np.isneginf(lse[:, 6:]).all()
    assert (absv[:6] >= np.abs(out[:6]) - 1e-12).all() and (dots[:6] > 0).all()
