"""Refusals of the norm/rotation and paged-cache entry points: host checks of the C ABI and of the
binding, nothing enqueued."""
import ctypes

import pytest
import torch

import long_context_prefill_moba_b200 as M
from long_context_prefill_moba_b200 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.load_library()


def rope_shape(**kw):
    base = dict(tokens=5, hq=8, hkv=2, head_dim=128, rot_dim=128)
    base.update(kw)
    return M.make_rope_shape(**base)


def paged_shape(**kw):
    base = dict(batch=2, tokens=3, hq=8, hkv=2, head_dim=128, page_size=64, num_pages=7, max_pages=4)
    base.update(kw)
    return M.make_paged_shape(**base)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(tokens=0), OK), (dict(rot_dim=0), OK), (dict(rot_dim=64), OK), (dict(rot_dim=16), OK),
    (dict(head_dim=64, rot_dim=64, dtype="f32"), OK), (dict(weight_dtype="f32"), OK),
    (dict(q_stride=1280, k_stride=1280), OK), (dict(eps=0.0), OK),
    (dict(tokens=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hkv=3), INVALID),
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(q_stride=1023), INVALID), (dict(q_stride=1028), INVALID), (dict(k_stride=255), INVALID),
    (dict(q_stride=-1024), INVALID),
    (dict(head_dim=96, rot_dim=96), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED),
    (dict(tokens=2**31 - 1), UNSUPPORTED)])
def test_rope_shapes(L, kw, want):
    s = rope_shape(**kw)
    assert M.moba_check_rope_shape(s) == want
    assert (M.moba_qk_norm_rope_bwd_workspace_size(s) > 0) == (want == OK)
    assert L.moba_check_rope_shape(None) == INVALID


def test_rope_flags_out_of_range(L):
    for name, value in (("interleaved", 2), ("weight_dtype", 2), ("weight_dtype", -1)):
        s = rope_shape()
        setattr(s.rope, name, value)
        assert M.moba_check_rope_shape(s) == INVALID
    s = rope_shape()
    s.dtype = 7
    assert M.moba_check_rope_shape(s) == INVALID


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(tokens=0), OK), (dict(page_size=16), OK), (dict(page_size=4096), OK), (dict(dtype="f32"), OK),
    (dict(k_page_stride=4 * 64 * 128, v_page_stride=4 * 64 * 128), OK), (dict(scale=0.5), OK),
    (dict(batch=65535), OK),
    (dict(batch=0), INVALID), (dict(tokens=-1), INVALID), (dict(hkv=3), INVALID), (dict(page_size=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(k_page_stride=2 * 64 * 128 - 8), INVALID), (dict(v_page_stride=2 * 64 * 128 + 4), INVALID),
    (dict(v_stride=100), INVALID), (dict(k_stride=260), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED),
    (dict(max_pages=1 << 24), OK), (dict(max_pages=(1 << 24) + 1), UNSUPPORTED), (dict(tokens=1 << 29), UNSUPPORTED)])
def test_paged_shapes(L, kw, want):
    s = paged_shape(**kw)
    assert M.moba_check_paged_shape(s) == want
    assert (M.moba_paged_attn_workspace_size(s) > 0) == (want == OK)
    assert L.moba_check_paged_shape(None) == INVALID


def test_norm_rope_pointers(L):
    s = rope_shape()
    good = [FAKE] * 8
    for i in range(8):
        for bad in (None, ODD if i < 4 or i > 5 else ctypes.c_void_p((1 << 20) + 2)):
            args = list(good)
            args[i] = bad
            args[6:] = [ctypes.c_void_p(2 << 20) if a is FAKE else a for a in args[6:]]
            assert L.moba_qk_norm_rope(ctypes.byref(s), *args, None) == INVALID, i
            assert M.moba_last_launch_count() == 0
    # results over strided inputs
    s = rope_shape(q_stride=2048, k_stride=2048)
    assert L.moba_qk_norm_rope(ctypes.byref(s), *([FAKE] * 8), None) == INVALID
    # no tokens: nothing to do, nothing enqueued
    s = rope_shape(tokens=0)
    assert L.moba_qk_norm_rope(ctypes.byref(s), *([None] * 8), None) == OK
    assert M.moba_last_launch_count() == 0


def test_norm_rope_bwd_pointers(L):
    s = rope_shape()
    need = M.moba_qk_norm_rope_bwd_workspace_size(s)
    for i in range(13):
        for bad in (None, ODD if i not in (4, 5) else ctypes.c_void_p((1 << 20) + 2)):
            args = [FAKE] * 13
            args[i] = bad
            assert L.moba_qk_norm_rope_bwd(ctypes.byref(s), *args, need, None) == INVALID, i
    assert L.moba_qk_norm_rope_bwd(ctypes.byref(s), *([FAKE] * 13), need - 1, None) == WORKSPACE
    assert M.moba_last_launch_count() == 0


def test_append_pointers(L):
    s, r = paged_shape(), M.MobaRope(128, 0, 0, 1e-6)
    names = ["q", "k", "v", "qw", "kw", "inv_freq", "cu", "kv_len", "table", "q_out", "k_pool", "v_pool", "status"]
    needed = {"k", "v", "inv_freq", "cu", "kv_len", "table", "k_pool", "v_pool"}
    for i, name in enumerate(names):
        args = [FAKE] * 13
        args[i] = ctypes.c_void_p((1 << 20) + 2)
        assert L.moba_paged_append(ctypes.byref(s), ctypes.byref(r), *args, None) == INVALID, name
        if name in needed or name in ("q", "q_out"):
            args[i] = None
            assert L.moba_paged_append(ctypes.byref(s), ctypes.byref(r), *args, None) == INVALID, name
    assert L.moba_paged_append(ctypes.byref(s), None, *([FAKE] * 13), None) == INVALID
    for bad in (M.MobaRope(8, 0, 0, 1e-6), M.MobaRope(144, 0, 0, 1e-6), M.MobaRope(128, 3, 0, 1e-6)):
        assert L.moba_paged_append(ctypes.byref(s), ctypes.byref(bad), *([FAKE] * 13), None) in (INVALID, UNSUPPORTED)
    s = paged_shape(q_stride=2048)
    assert L.moba_paged_append(ctypes.byref(s), ctypes.byref(r), *([FAKE] * 13), None) == INVALID   # q_out is q
    s = paged_shape(tokens=0)
    assert L.moba_paged_append(ctypes.byref(s), ctypes.byref(r), *([None] * 13), None) == OK
    assert M.moba_last_launch_count() == 0


def test_attention_pointers(L):
    s = paged_shape()
    need = M.moba_paged_attn_workspace_size(s)
    for i in range(10):
        args = [FAKE] * 10
        args[i] = ctypes.c_void_p((1 << 20) + 2)
        assert L.moba_paged_attn(ctypes.byref(s), *args, need, None) == INVALID, i
        if i not in (7, 8):    # lse and status may be missing
            args[i] = None
            assert L.moba_paged_attn(ctypes.byref(s), *args, need, None) == INVALID, i
    assert L.moba_paged_attn(ctypes.byref(s), *([FAKE] * 10), need - 1, None) == WORKSPACE
    s = paged_shape(tokens=0)
    assert L.moba_paged_attn(ctypes.byref(s), *([None] * 10), 0, None) == OK
    assert M.moba_last_launch_count() == 0


def test_binding_refuses_cpu_tensors(L):
    t = torch.zeros(3, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.moba_norm_rope(t, t, torch.ones(64), torch.ones(64), i, torch.zeros(0, dtype=torch.float64))
    with pytest.raises(ValueError):
        M.moba_cache_append(t, t, i, i[:1], i[None], torch.zeros(2, 4, 16, 64), torch.zeros(2, 4, 16, 64))
    with pytest.raises(ValueError):
        M.moba_cache_attention(t, torch.zeros(2, 4, 16, 64), torch.zeros(2, 4, 16, 64), i, i[:1], i[None])


def test_binding_is_built_beside_the_library(L):
    import os
    path = B.build_binding()
    assert os.path.dirname(path) == os.path.dirname(B.LIB) and os.path.exists(path)
    assert M.load_binding() is M.load_binding()
    for name in ("norm_rope", "cache_append", "cache_attention"):
        assert callable(getattr(M.load_binding(), name))


def test_inv_freq():
    f = M.moba_rope_inv_freq(64, 10000.0, "cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0 and abs(f[16] - 0.01) < 1e-15


def test_pools_whose_pages_overlap_are_refused(L):
    """A page for all (stride 0, which the C call reads as dense) and pages that overlap: no offset of a page may leave the
    pool's memory."""
    i = torch.zeros(2, dtype=torch.int32)
    x, good = torch.zeros(3, 4, 64), torch.zeros(6, 4, 16, 64)
    one = torch.zeros(1, 4, 16, 64).expand(6, 4, 16, 64)
    half = torch.zeros(6 * 4 * 16 * 64).as_strided((6, 4, 16, 64), (2 * 16 * 64, 16 * 64, 64, 1))
    for bad in (one, half):
        for pools in ((bad, good), (good, bad)):
            with pytest.raises(ValueError, match="overlap"):
                M.moba_cache_append(x, x, i, i[:1], i[None], *pools)
            with pytest.raises(ValueError, match="overlap"):
                M.moba_cache_attention(x, *pools, i, i[:1], i[None])
    # a single page has no stride that counts
    with pytest.raises(ValueError, match="CUDA"):
        M.moba_cache_attention(x, one[:1], good[:1], i, i[:1], i[None])


def test_a_row_of_heads_stays_in_32_bits(L):
    for make, check in ((rope_shape, M.moba_check_rope_shape), (paged_shape, M.moba_check_paged_shape)):
        for d, most in ((128, 2**24 - 1), (64, 2**25 - 1)):
            kw = dict(tokens=1, hkv=1, head_dim=d)
            if make is rope_shape:
                kw["rot_dim"] = d
            assert check(make(hq=most, **kw)) == OK
            assert check(make(hq=most + 1, **kw)) == UNSUPPORTED


def test_forward_mode_derivatives_are_refused(L):
    """A dual tensor needs no gradient in reverse mode; its tangent must not be lost either."""
    import torch.autograd.forward_ad as fwad
    t, w, i = torch.zeros(3, 4, 64), torch.ones(64), torch.zeros(2, dtype=torch.int32)
    f, pool = torch.zeros(0, dtype=torch.float64), torch.zeros(2, 4, 16, 64)
    norm = lambda q, k, wq, wk: M.moba_norm_rope(q, k, wq, wk, i, f)  # noqa: E731
    append = lambda k, v, q, wq, wk, kp: M.moba_cache_append(k, v, i, i[:1], i[None], kp, pool, q=q, q_weight=wq, k_weight=wk)  # noqa: E731
    attend = lambda q, kp, vp: M.moba_cache_attention(q, kp, vp, i, i[:1], i[None])  # noqa: E731
    for call, args in ((norm, (t, t, w, w)), (append, (t, t, t, w, w, pool)), (attend, (t, pool, pool))):
        for at in range(len(args)):
            with fwad.dual_level():
                dual = list(args)
                dual[at] = fwad.make_dual(args[at], torch.ones_like(args[at]))
                with pytest.raises(RuntimeError, match="forward-mode"):
                    call(*dual)
        with pytest.raises(ValueError, match="CUDA"):
            call(*args)


def test_cache_calls_refuse_gradients(L):
    """They have none: an input that asks for one is refused in grad mode, not cut off without a word."""
    t, w, i = torch.zeros(3, 4, 64), torch.ones(64), torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(2, 4, 16, 64)
    append = lambda k, v, q, wq, wk, kp, vp: M.moba_cache_append(k, v, i, i[:1], i[None], kp, vp, q=q, q_weight=wq, k_weight=wk)  # noqa: E731
    attend = lambda q, kp, vp: M.moba_cache_attention(q, kp, vp, i, i[:1], i[None])  # noqa: E731
    for call, args in ((append, (t, t, t, w, w, pool, pool)), (attend, (t, pool, pool))):
        for at in range(len(args)):
            asks = list(args)
            asks[at] = args[at].clone().requires_grad_()
            with pytest.raises(RuntimeError, match="no gradient"):
                call(*asks)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(*asks)


def test_a_single_heads_stride_does_not_count(L):
    """Pools kept as [pages, slots, 1, d] and passed with heads and slots exchanged are dense."""
    i = torch.zeros(2, dtype=torch.int32)
    x, pool = torch.zeros(3, 1, 64), torch.zeros(6, 16, 1, 64).transpose(1, 2)
    assert pool.stride(1) != 16 * 64
    with pytest.raises(ValueError, match="CUDA"):
        M.moba_cache_append(x, x, i, i[:1], i[None], pool, pool)
    with pytest.raises(ValueError, match="CUDA"):
        M.moba_cache_attention(x, pool, pool, i, i[:1], i[None])
    with pytest.raises(ValueError, match="dense"):
        M.moba_cache_attention(torch.zeros(3, 4, 64), *[torch.zeros(6, 16, 4, 64).transpose(1, 2)] * 2, i, i[:1], i[None])


def test_frequencies_have_no_gradient(L):
    t, w, i = torch.zeros(2, 4, 64), torch.ones(64), torch.zeros(2, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64, requires_grad=True)
    with pytest.raises(RuntimeError, match="inv_freq has no gradient"):
        M.moba_norm_rope(t, t, w, w, i, f)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        M.moba_norm_rope(t, t, w, w, i, f)
