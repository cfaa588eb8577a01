"""Per-head norm with rotation on the GPU against the fp64 form, forward and gradients.

Tolerances, per element, from the arithmetic (u = 2^-24, half a step of fp32):
  a head's sum of 128 squares is off by at most 128 u of itself, its root's reciprocal by half of
  that and the special function's 2 u; two products follow: y is off by at most 70 u |y|.  The
  angle's rounding (at most pi u) and sine's and cosine's (4 u) and three operations add 12 u of
  |a| + |b|.  Together under 1e-5 (|a| + |b|), and half a step of the result's type.
  The gradients repeat this with <x, g>, a sum of 128 products: off by 128 u sum |x g| more.
  A weight's gradient sums T heads terms in chains (one thread's share, then trees): off by at most
  (chain + 150) u of the sum of |terms|, chain bounded by the number of terms."""
import numpy as np
import pytest
import torch

from oracle import serving as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def pair_size(y, r, interleaved):
    """|a| + |b| of each channel's pair (|y| alone where it is not rotated)."""
    a = np.abs(y).copy()
    i = np.arange(r)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    s = a[..., ia] + a[..., ib]
    a[..., ia], a[..., ib] = s, s
    return a


CASES = [
    # tokens, hq, hkv, d, rot, interleaved, dtype, weights, far
    (1, 4, 1, 128, 128, False, "bf16", "bf16", 10485759),
    (8, 32, 8, 128, 128, False, "bf16", "f32", 131072),
    (7, 6, 3, 64, 64, True, "bf16", "bf16", 10 ** 9),
    (13, 16, 16, 64, 32, False, "f32", "f32", 10485759),
    (5, 5, 1, 128, 16, True, "f32", "bf16", 2 ** 31 - 1),
    (300, 8, 2, 128, 64, False, "f32", "f32", 40000),
    (1111, 2, 1, 64, 48, False, "bf16", "f32", 1111),
    (3, 1, 1, 128, 0, False, "bf16", "bf16", 5),
    (6000, 9, 3, 128, 128, True, "bf16", "f32", 6000),
]


def inputs(case, dev, seed=0):
    T, hq, hkv, d, rot, inter, dt, wt, far = case
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    qkv = n(T, hq + 2 * hkv, d).to(DT[dt])
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    wq, wk = (1 + 0.5 * n(d)).to(DT[wt]), (1 + 0.5 * n(d)).to(DT[wt])
    pos = torch.randint(-3, far, (T,), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    pos[0] = far - 1
    import long_context_prefill_moba_b200 as M
    f = M.moba_rope_inv_freq(rot, 500000.0, dev)
    dq, dk = n(T, hq, d).to(DT[dt]), n(T, hkv, d).to(DT[dt])
    return q, k, wq, wk, pos, f, dq, dk


def check_forward(out, x, w, pos, f, eps, inter, dtype):
    y = O.norm(np64(x), np64(w), eps)
    want = O.rotate(y, pos.cpu().numpy(), np64(f), inter)
    tol = half_step(dtype) * np.abs(want) + 1e-5 * pair_size(y, len(f), inter) + 1e-30
    assert (np.abs(np64(out) - want) <= tol).all(), np.max(np.abs(np64(out) - want) / tol)


def check_backward(dx, dw, x, w, pos, f, eps, dy, inter, dtype, wtype):
    xn, wn, dyn = np64(x), np64(w), np64(dy)
    want, wwant = O.norm_rope_backward(xn, wn, pos.cpu().numpy(), np64(f), eps, dyn, inter)
    r = 1 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
    zsize = pair_size(dyn, len(f), inter)              # bounds |z| and its error / 12 u
    gsize = zsize * np.abs(wn)
    dots = (np.abs(xn) * gsize).mean(-1, keepdims=True)
    tol = half_step(dtype) * np.abs(want) + 2e-5 * (r * gsize + np.abs(xn) * r ** 3 * dots) + 1e-30
    err = np.abs(np64(dx) - want)
    assert (err <= tol).all(), np.max(err / tol)
    terms = (zsize * np.abs(xn) * r).sum((0, 1))
    tol = half_step(wtype) * np.abs(wwant) + (min(xn.shape[0] * xn.shape[1], 2000) + 150) * U * terms
    err = np.abs(np64(dw) - wwant)
    assert (err <= tol).all(), np.max(err / tol)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(cuda_device, case):
    import long_context_prefill_moba_b200 as M
    T, hq, hkv, d, rot, inter, dt, wt, far = case
    q, k, wq, wk, pos, f, dq, dk = inputs(case, cuda_device)
    eps = 1e-5
    with torch.no_grad():
        plain = M.moba_norm_rope(q, k, wq, wk, pos, f, eps, inter)
    check_forward(plain[0], q, wq, pos, f, eps, inter, q.dtype)
    check_forward(plain[1], k, wk, pos, f, eps, inter, q.dtype)
    leaves = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    outs = M.moba_norm_rope(*leaves, pos, f, eps, inter)
    assert torch.equal(outs[0], plain[0]) and torch.equal(outs[1], plain[1])
    grads = torch.autograd.grad(outs, leaves, (dq, dk))
    check_backward(grads[0], grads[2], q, wq, pos, f, eps, dq, inter, q.dtype, wq.dtype)
    check_backward(grads[1], grads[3], k, wk, pos, f, eps, dk, inter, q.dtype, wq.dtype)
    again = torch.autograd.grad(M.moba_norm_rope(*leaves, pos, f, eps, inter), leaves, (dq, dk))
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_gradients_are_those_of_differences(cuda_device):
    # fp32, steps large enough that the difference quotient's rounding stays below 1e-2 of the gradients' size
    import long_context_prefill_moba_b200 as M
    q, k, wq, wk, pos, f, dq, dk = inputs((4, 2, 1, 64, 64, False, "f32", "f32", 1000), cuda_device)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk)]
    grads = torch.autograd.grad(M.moba_norm_rope(*leaves, pos, f), leaves, (dq, dk))
    loss = lambda xs: sum((o.double() * d.double()).sum() for o, d in zip(M.moba_norm_rope(*xs, pos, f), (dq, dk)))  # noqa: E731
    g = torch.Generator(device=cuda_device)
    g.manual_seed(1)
    for i in range(4):
        v = torch.randn(leaves[i].shape, generator=g, device=cuda_device)
        h = 1e-2
        with torch.no_grad():
            up = [x + h * v if j == i else x for j, x in enumerate(leaves)]
            down = [x - h * v if j == i else x for j, x in enumerate(leaves)]
            diff = (loss(up) - loss(down)) / (2 * h)
        want = (grads[i].double() * v.double()).sum()
        # third-order term of a smooth function of unit-size arguments: h^2 times its size, some 1e-4 |v|^2
        assert abs(diff - want) <= 1e-2 * grads[i].double().norm() * v.double().norm(), i


def test_batched_inputs_feed_the_attention(cuda_device):
    """A layer as it is trained: norm and rotation, then MoBA attention, gradients to the projection's rows."""
    import long_context_prefill_moba_b200 as M
    b, N, hq, hkv, d = 2, 512, 4, 2, 128
    g = torch.Generator(device=cuda_device)
    g.manual_seed(3)
    qkv = torch.randn(b, N, hq + 2 * hkv, d, generator=g, device=cuda_device).to(torch.bfloat16).requires_grad_()
    w = torch.ones(d, device=cuda_device, requires_grad=True)
    pos = torch.arange(N, device=cuda_device, dtype=torch.int32).repeat(b)
    f = M.moba_rope_inv_freq(d, device=cuda_device)
    q, k = M.moba_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], w, w, pos, f)
    assert q.shape == (b, N, hq, d) and k.shape == (b, N, hkv, d)
    out = M.moba_attention(q, k, qkv[:, :, hq + hkv:], 128, 2)
    dout = torch.randn(out.shape, generator=g, device=cuda_device).to(torch.bfloat16)
    out.backward(dout)
    # the same chain by hand: the attention's own gradients through the norm's formula
    ql, kl = q.detach().requires_grad_(), k.detach().requires_grad_()
    vl = qkv.detach()[:, :, hq + hkv:].contiguous().requires_grad_()
    M.moba_attention(ql, kl, vl, 128, 2).backward(dout)
    x = qkv.detach()
    for got, x, dy in ((qkv.grad[:, :, :hq], x[:, :, :hq], ql.grad), (qkv.grad[:, :, hq:hq + hkv], x[:, :, hq:hq + hkv], kl.grad)):
        want, _ = O.norm_rope_backward(np64(x).reshape(b * N, -1, d), np64(w), pos.cpu().numpy(), np64(f), 1e-6,
                                       np64(dy).reshape(b * N, -1, d))
        err = np.abs(np64(got).reshape(want.shape) - want)
        # the attention's backward adds dq in an order that may differ between the two runs: half a bf16 step of dy more
        assert err.max() <= 2 ** -6 * np.abs(want).max()
    # dv sums over the rows of a block in the order of the gate's index, which two forwards need not share: fp32 sums
    # that differ in their last bits round to neighbouring bf16 values at most, one step (2^-7) apart
    dv = qkv.grad[:, :, hq + hkv:].double()
    assert (dv - vl.grad.double()).norm() <= 2 ** -7 * vl.grad.double().norm() and torch.isfinite(w.grad).all()


def test_zero_rows_extremes_and_in_place(cuda_device):
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    d, f, w = 64, M.moba_rope_inv_freq(64, device=dev), torch.ones(64, device=dev)
    x = torch.randn(4, 2, d, device=dev)
    x[0] = 0
    x[1] = 1e15          # squares still fit fp32
    x[2, 0, 3] = float("nan")
    x[2, 1, 5] = float("inf")
    pos = torch.arange(4, device=dev, dtype=torch.int32)
    k = x[:, :1].contiguous()
    q_out, k_out = M.moba_norm_rope(x, k, w, w, pos, f)
    assert (q_out[0] == 0).all() and torch.isfinite(q_out[1]).all() and torch.isnan(q_out[2, 0]).all()
    # an infinity's mean square is infinite: r = 0, its own pair 0 * inf = NaN, the other channels 0
    pair = torch.zeros(d, dtype=torch.bool, device=dev)
    pair[[5, 37]] = True
    assert torch.isnan(q_out[2, 1, pair]).all() and (q_out[2, 1, ~pair] == 0).all()
    assert torch.isfinite(q_out[3]).all()
    s = M.make_rope_shape(4, 2, 1, d, d, "f32")
    M.moba_qk_norm_rope(s, x, k, w, w, pos, f, x, k)
    assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(q_out)) and torch.equal(torch.nan_to_num(k), torch.nan_to_num(k_out))


def test_layouts_that_are_copied(cuda_device):
    """Heads before tokens, every second token, one token for all: as dense inputs, gradients in the inputs' layout."""
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    w, f = 1 + 0.3 * n(64), M.moba_rope_inv_freq(32, device=dev)
    pos = torch.arange(12, dtype=torch.int32, device=dev)
    for q, k in ((n(2, 4, 6, 64).transpose(1, 2), n(2, 2, 6, 64).transpose(1, 2)), (n(24, 4, 64)[::2], n(24, 2, 64)[::2]),
                 (n(1, 4, 64).expand(12, 4, 64), n(1, 2, 64).expand(12, 2, 64))):
        dense = [x.contiguous().requires_grad_() for x in (q, k)]
        want = M.moba_norm_rope(*dense, w, w, pos, f)
        leaves = [x.detach().requires_grad_() for x in (q, k)]
        got = M.moba_norm_rope(*leaves, w, w, pos, f)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        d = [n(*x.shape) for x in want]
        a, b = torch.autograd.grad(got, leaves, d), torch.autograd.grad(want, dense, d)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        one = torch.autograd.grad(M.moba_norm_rope(*leaves, w, w, pos, f)[1].sum(), leaves)   # an expanded gradient; none for q
        assert (one[0] == 0).all() and torch.isfinite(one[1]).all()


def test_second_derivatives_are_refused(cuda_device):
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    leaves = [torch.randn(3, 2, 64, device=dev).requires_grad_(), torch.randn(3, 1, 64, device=dev).requires_grad_(),
              torch.ones(64, device=dev), torch.ones(64, device=dev)]
    out = M.moba_norm_rope(*leaves, torch.arange(3, dtype=torch.int32, device=dev), M.moba_rope_inv_freq(64, device=dev))
    with pytest.raises(RuntimeError, match="not differentiable"):
        torch.autograd.grad(out[0].sum(), leaves[0], create_graph=True)
    # only some of the leaves need gradients, or one output is used
    g = torch.autograd.grad(M.moba_norm_rope(*leaves, torch.arange(3, dtype=torch.int32, device=dev),
                                             M.moba_rope_inv_freq(64, device=dev))[1].square().sum(), leaves[:2])
    assert (g[0] == 0).all() and g[1].abs().max() > 0


def test_no_tokens(cuda_device):
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    leaves = [torch.empty(0, 4, 64, device=dev), torch.empty(0, 2, 64, device=dev), torch.ones(64, device=dev),
              torch.ones(64, device=dev)]
    leaves = [x.requires_grad_() for x in leaves]
    outs = M.moba_norm_rope(*leaves, torch.empty(0, dtype=torch.int32, device=dev), M.moba_rope_inv_freq(64, device=dev))
    g = torch.autograd.grad(outs, leaves, [torch.empty_like(o) for o in outs])
    assert g[0].shape == (0, 4, 64) and (g[2] == 0).all() and (g[3] == 0).all()


def test_captured_step_and_another_stream(cuda_device):
    import long_context_prefill_moba_b200 as M
    case = (65, 8, 2, 128, 128, False, "bf16", "f32", 5000)
    q, k, wq, wk, pos, f, dq, dk = inputs(case, cuda_device)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk)]

    def step():
        # values alone: a step's autograd graph does not outlive it (a backward pass cannot be captured while an eager
        # graph of the same leaves lives)
        outs = M.moba_norm_rope(*leaves, pos, f)
        return tuple(o.detach() for o in outs) + torch.autograd.grad(outs, leaves, (dq, dk))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        for x in leaves[:2]:
            x.mul_(2).sub_(1)
    graph.replay()
    new = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, new))
    assert not torch.equal(got[0], want[0])


def test_leading_dimensions_of_one(cuda_device):
    """Dimensions of one token or sequence between others, whose strides say nothing about the rows: as dense inputs."""
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    w, f = torch.ones(64, device=dev), M.moba_rope_inv_freq(64, device=dev)
    views = [
        lambda x: x[:, None, :5],          # [2, 1, 5, h, 64]: the stride of the 1 is that of the whole sequences
        lambda x: x[:, :5, None],          # [2, 5, 1, h, 64]
        lambda x: x[:, 3:4],               # one token of each sequence
        lambda x: x[:1, 3:4],              # one token
        lambda x: x[:1, None, 2:7],
        lambda x: x[:, ::2][:, :, None],
        lambda x: x[:, :, None, None],     # every token: read where it lies
        lambda x: x[None, :, :5],
        lambda x: x[:, 4:5].expand(2, 7, *x.shape[2:]),              # one token for all of a sequence
        lambda x: x[:1, :6].expand(3, 6, *x.shape[2:])[:, None],     # one sequence for all
        lambda x: x[:, 4:5, None].expand(2, 7, 3, *x.shape[2:]),
    ]
    for view in views:
        q, k = (view(torch.randn(2, 10, h, 64, generator=g, device=dev)) for h in (4, 2))
        pos = torch.arange(q.shape[:-2].numel(), dtype=torch.int32, device=dev)
        dense = [x.contiguous().requires_grad_() for x in (q, k)]
        leaves = [x.detach().requires_grad_() for x in (q, k)]
        want, got = M.moba_norm_rope(*dense, w, w, pos, f), M.moba_norm_rope(*leaves, w, w, pos, f)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        d = [torch.randn(x.shape, generator=g, device=dev) for x in want]
        a, b = torch.autograd.grad(got, leaves, d), torch.autograd.grad(want, dense, d)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("case", [
    (9, 5, 1, 128, 128, False, "bf16", "bf16", 50), (40, 6, 3, 64, 64, True, "f32", "f32", 50),
    (300, 2, 2, 128, 64, False, "f32", "f32", 300), (17, 9, 9, 64, 0, False, "bf16", "f32", 50)], ids=str)
def test_gradients_without_eps(cuda_device, case):
    """eps = 0, head counts that leave lanes of a warp without a head."""
    import long_context_prefill_moba_b200 as M
    T, hq, hkv, d, rot, inter, dt, wt, far = case
    q, k, wq, wk, pos, f, dq, dk = inputs(case, cuda_device, 7)
    leaves = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    outs = M.moba_norm_rope(*leaves, pos, f, 0.0, inter)
    check_forward(outs[0], q, wq, pos, f, 0.0, inter, q.dtype)
    check_forward(outs[1], k, wk, pos, f, 0.0, inter, q.dtype)
    grads = torch.autograd.grad(outs, leaves, (dq, dk))
    check_backward(grads[0], grads[2], q, wq, pos, f, 0.0, dq, inter, q.dtype, wq.dtype)
    check_backward(grads[1], grads[3], k, wk, pos, f, 0.0, dk, inter, q.dtype, wq.dtype)


@pytest.mark.parametrize("size,eps", [(1e-17, 0.0), (1e-12, 0.0), (1e13, 1e-6), (1e15, 1e-6), (1e17, 1e-6), (0.0, 1e-30)])
def test_gradients_of_small_and_large_heads(cuda_device, size, eps):
    """Heads whose squares fit fp32 but whose r^3 does not: no product of the gradient leaves the normal range, so the
    bounds are those of heads of size 1."""
    import long_context_prefill_moba_b200 as M
    case = (11, 4, 2, 64, 64, False, "f32", "f32", 50)
    q, k, wq, wk, pos, f, dq, dk = inputs(case, cuda_device, 8)
    q, k = (size * x for x in (q, k))
    leaves = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    outs = M.moba_norm_rope(*leaves, pos, f, eps)
    grads = torch.autograd.grad(outs, leaves, (dq, dk))
    check_backward(grads[0], grads[2], q, wq, pos, f, eps, dq, False, q.dtype, wq.dtype)
    check_backward(grads[1], grads[3], k, wk, pos, f, eps, dk, False, q.dtype, wq.dtype)


def test_forward_mode_derivatives_are_refused(cuda_device):
    """Tangents of the inputs, and of the gradients that a backward pass is given."""
    import torch.autograd.forward_ad as fwad
    import long_context_prefill_moba_b200 as M
    q, k, wq, wk, pos, f, dq, dk = inputs((3, 4, 2, 64, 64, False, "f32", "f32", 50), cuda_device)
    args = [x.contiguous() for x in (q, k, wq, wk)]
    for at in range(4):
        for grad in (False, True):
            with fwad.dual_level():
                dual = [x.detach().clone().requires_grad_(grad) for x in args]
                dual[at] = fwad.make_dual(dual[at], torch.ones_like(args[at]))
                with pytest.raises(RuntimeError, match="forward-mode"):
                    M.moba_norm_rope(*dual, pos, f)
    leaves = [x.detach().clone().requires_grad_() for x in args]
    outs = M.moba_norm_rope(*leaves, pos, f)
    want = torch.autograd.grad(outs, leaves, (dq, dk), retain_graph=True)
    with fwad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            torch.autograd.grad(outs, leaves, (fwad.make_dual(dq, torch.ones_like(dq)), dk), retain_graph=True)
    again = torch.autograd.grad(outs, leaves, (dq, dk))
    assert all(torch.equal(a, b) for a, b in zip(want, again))
