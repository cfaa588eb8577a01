"""Append to a paged cache and the attention over it on the GPU, against the fp64 forms.

Attention tolerances, per element (u = 2^-24): a logit is a sum of d <= 128 products, off by at most
(d + 4) u scale sum |q_c k_c| (its products' fp32 additions, the scale and the change of base), and its
exponential by 4 u more; an output is a quotient of two sums of L terms added one after another or in
trees, off by at most (L + 64) u each.  With e the sum of these, |out - exact| <= 2 e max |v|.  bf16 adds
the rounding of the probabilities, half a step (2^-8) of each: 2^-8 sum p |v|, and of the result:
2^-8 |out|; likewise a rounded probability against the unrounded sum in its denominator is within that
term.  lse is off by at most e, and its own rounding 2 u |lse|."""
import numpy as np
import pytest
import torch

from oracle import serving as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INTERNAL = 5


def np64(t):
    return t.detach().double().cpu().numpy()


def half_step(t):
    return torch.finfo(t).eps / 2


class Cache:
    """A cache of random pages for sequences of (new tokens, length) with NaN wherever nothing may read."""

    def __init__(self, lens, page, hkv, d, dtype, dev, seed=0, spare=3, joint=False, pad=0, max_pages=None, nan=True):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.lens, self.page, self.hkv, self.d, self.dtype, self.dev = lens, page, hkv, d, DT[dtype], dev
        need = [max(0, -(-L // page)) for _, L in lens]
        self.pages = sum(need) + spare
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        cols = max_pages or max(max(need), 1) + 1
        self.table = torch.full((len(lens), cols), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, hkv, page, d)
        fill = float("nan") if nan else 0.0
        if joint:    # keys and values of a page side by side in one allocation
            both = torch.full((self.pages, 2, hkv, page, d), fill, dtype=self.dtype, device=dev)
            self.k_pool, self.v_pool = both[:, 0], both[:, 1]
        else:
            self.k_pool, self.v_pool = (torch.full(shape, fill, dtype=self.dtype, device=dev) for _ in range(2))
        for b, (n, L) in enumerate(lens):
            for j in range(need[b]):
                m = min(page, L - j * page)
                for p in (self.k_pool, self.v_pool):
                    p[int(self.table[b, j]), :, :m] = torch.randn(hkv, m, d, generator=g).to(self.dtype).to(dev)
        self.cu = torch.tensor([0] + list(np.cumsum([n for n, _ in lens])), dtype=torch.int32)
        self.kv_len = torch.tensor([L for _, L in lens], dtype=torch.int32)
        self.total = int(self.cu[-1])
        self.rows = self.total + pad
        self.index = [x.to(dev) for x in (self.cu, self.kv_len, self.table)]
        self.g = g

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(self.dtype).to(self.dev)


def check_attention(c, q, out, lse, scale=None, rows=None):
    """Every row, or the given ones."""
    d = c.d
    scale = d ** -0.5 if scale is None else scale
    kn, vn = np.nan_to_num(np64(c.k_pool)), np.nan_to_num(np64(c.v_pool))
    want, wlse, dots, absv = O.paged_attention(np64(q)[:c.total], kn, vn, c.cu.numpy(), c.kv_len.numpy(),
                                               c.table.numpy(), scale, rows and set(rows))
    L = max(max(x for _, x in c.lens), 1)
    e = (d + 8) * U * scale * dots + (L + 64) * U
    vmax = np.abs(vn).max() if vn.size else 0.0
    tol = 2 * e[..., None] * vmax + half_step(q.dtype) * np.abs(want)
    if q.dtype != torch.float32:
        tol = tol + 2 * half_step(q.dtype) * absv
    at = list(range(c.total)) if rows is None else sorted(rows)
    err = np.abs(np64(out)[:c.total] - want)
    assert not np.isnan(np64(out)[:c.total]).any()
    assert (err <= tol + 1e-30)[at].all(), float(np.max((err / (tol + 1e-30))[at]))
    if lse is not None:
        got = np64(lse)[:, at]
        wlse, e = wlse[:, at], e[at]
        assert (np.isneginf(got) == np.isneginf(wlse)).all()
        fine = np.isfinite(wlse)
        assert (np.abs(got[fine] - wlse[fine]) <= (e.T + 4 * U)[fine] + 2 * U * np.abs(wlse[fine])).all()


# (new tokens, keys) of each sequence, page, hq, hkv, d, dtype
ONE = [
    ([(1, 1)], 16, 4, 1, 128, "bf16"),
    ([(1, 1000)], 16, 4, 1, 128, "bf16"),
    ([(1, 15), (1, 16), (1, 17), (1, 31), (1, 33), (1, 64), (1, 129)], 16, 4, 4, 64, "bf16"),
    ([(1, 700), (0, 300), (1, 5), (0, 0), (1, 2049)], 64, 32, 8, 128, "bf16"),
    ([(1, 257 + 31 * i) for i in range(40)], 32, 8, 2, 128, "bf16"),
    ([(1, 9000)], 256, 16, 2, 64, "bf16"),
    ([(1, 300), (1, 77)], 16, 16, 1, 128, "bf16"),
    ([(1, 600)], 32, 24, 1, 64, "bf16"),
    ([(1, 3 * i + 1) for i in range(300)], 16, 2, 1, 64, "bf16"),
    ([(2, 500), (5, 90), (3, 3)], 64, 8, 2, 128, "bf16"),
    ([(1, 1), (1, 1000), (1, 33)], 32, 8, 2, 128, "f32"),
    ([(1, 5000), (0, 7), (2, 17)], 64, 16, 16, 64, "f32"),
    ([(4, 333)], 16, 16, 1, 128, "f32"),
]
CHUNKS = [
    ([(64, 64)], 16, 4, 1, 128, "bf16"),
    ([(37, 37), (1, 900), (0, 40), (130, 517), (16, 16)], 16, 4, 1, 128, "bf16"),
    ([(129, 129), (300, 1300)], 64, 8, 2, 128, "bf16"),
    ([(200, 333)], 256, 6, 2, 64, "bf16"),
    ([(257, 257), (255, 1111)], 128, 4, 4, 128, "bf16"),
    ([(513, 700)], 32, 16, 2, 64, "bf16"),
    ([(90, 2000)], 512, 5, 1, 128, "bf16"),
    ([(100, 130), (7, 900)], 16, 4, 2, 128, "f32"),
    ([(65, 65), (129, 400)], 64, 4, 4, 64, "f32"),
]


@pytest.mark.parametrize("case", ONE + CHUNKS, ids=lambda c: f"{c[5]}-d{c[4]}-{c[2]}x{c[3]}-p{c[1]}-{len(c[0])}seq-{c[0][0]}")
def test_attention(cuda_device, case):
    import long_context_prefill_moba_b200 as M
    lens, page, hq, hkv, d, dt = case
    c = Cache(lens, page, hkv, d, dt, cuda_device, pad=3)
    q = c.rand(c.rows, hq, d)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    keep = torch.full_like(q, 7.0)
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True, out=keep, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_attention(c, q, out, lse)
    assert (out[c.total:] == 7.0).all()          # rows behind the last sequence
    again, lse2 = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    assert torch.equal(again[:c.total], out[:c.total]) and torch.equal(lse2[:, :c.total], lse[:, :c.total])


@pytest.mark.parametrize("case", [
    ([(1500, 6000), (0, 30), (700, 700), (1, 5000)], 32, 16, 4, 64, "bf16"),
    ([(1025, 9000), (64, 20000)], 16, 8, 2, 128, "bf16"),
    ([(3, 3)] * 200 + [(4000, 4100)] + [(70, 400)] * 30, 128, 6, 2, 128, "bf16"),
    ([(300, 2000), (200, 300)], 64, 8, 8, 128, "f32"),
    ([(1, 40000), (1, 90000)], 64, 8, 2, 128, "bf16"),
    ([(1, 40000), (2, 30000)], 64, 8, 2, 64, "f32"),
    ([(20, 25 + i % 9) if i % 4 else (0, 3) for i in range(1000)], 16, 2, 2, 64, "bf16"),
    ([(20, 25 + i % 9) if i % 4 else (0, 3) for i in range(400)], 16, 2, 2, 64, "f32"),
    ([(1, 30 + i % 50) for i in range(900)], 16, 4, 1, 64, "f32"),
    ([(3, 700), (260, 900)], 32, 512, 1, 64, "bf16"),
    ([(1, 700), (1, 1500)], 32, 300, 1, 128, "bf16")],
    ids=lambda c: f"{c[5]}-d{c[4]}-{c[2]}x{c[3]}-p{c[1]}-{len(c[0])}seq-{c[0][0]}")
def test_attention_of_many_tiles(cuda_device, case):
    """Enough keys that every worker goes through many tiles and several items: rows at every border and random ones."""
    import long_context_prefill_moba_b200 as M
    lens, page, hq, hkv, d, dt = case
    c = Cache(lens, page, hkv, d, dt, cuda_device)
    q = c.rand(c.rows, hq, d)
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    again = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index)
    assert torch.equal(again, out)
    r = np.random.RandomState(0)
    cu = c.cu.numpy()
    few = cu if len(cu) < 20 else cu[::25]
    rows = {int(x) for x in list(few) + [x - 1 for x in few] + list(r.randint(0, c.total, 25)) if 0 <= x < c.total}
    check_attention(c, q, out, lse, rows=rows)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 50])
def test_sequences_that_share_pages(cuda_device, dt, new):
    """One prompt's pages in two tables, and one page twice in a table."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 64 + new), (new, 64 + new)], 16, 2, 64, dt, cuda_device)
    q = c.rand(new, 4, 64).repeat(2, 1, 1)
    cu, kv_len, table = (x.clone() for x in c.index)
    table[1] = table[0]
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, cu, kv_len, table, return_lse=True)
    # (where a sequence's keys are cut depends on the others of the call: equal within the bounds, not to the bit)
    c.table = table.cpu()
    check_attention(c, q, out, lse)
    table[:, 1] = table[:, 0]
    c.table = table.cpu()
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, cu, kv_len, table, return_lse=True)
    check_attention(c, q, out, lse)


def test_only_padding(cuda_device):
    """A step in which no sequence has a new token: nothing is written."""
    import long_context_prefill_moba_b200 as M
    for dt in ("bf16", "f32"):
        for rows in (2, 40):
            c = Cache([(0, 50), (0, 0)], 16, 2, 64, dt, cuda_device, pad=rows, nan=False)
            x = c.rand(rows, 8, 64)
            out = torch.full((rows, 4, 64), 7.0, dtype=c.dtype, device=cuda_device)
            before = c.k_pool.clone()
            M.moba_cache_attention(x[:, :4], c.k_pool, c.v_pool, *c.index, out=out)
            M.moba_cache_append(x[:, 4:6], x[:, 6:], *c.index, c.k_pool, c.v_pool, q=x[:, :4], q_out=out)
            assert (out == 7.0).all() and torch.equal(c.k_pool, before)
            none = torch.empty(0, 4, 64, dtype=c.dtype, device=cuda_device)
            assert M.moba_cache_attention(none, c.k_pool, c.v_pool, *c.index).shape == (0, 4, 64)
            assert M.moba_cache_append(none[:, :2], none[:, 2:], *c.index, c.k_pool, c.v_pool, q=none).shape == (0, 4, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_strides_scale_and_joint_pools(cuda_device, dt, new):
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 200), (new, 50)], 16, 2, 64, dt, cuda_device, joint=True)
    qkv = c.rand(c.rows, 8 + 4, 64)
    q = qkv[:, :8]
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, scale=0.31, return_lse=True)
    check_attention(c, q, out, lse, scale=0.31)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [3, 70])
def test_rows_before_the_first_key(cuda_device, dt, new):
    """More new tokens than keys: the first rows have no key."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, new - 2), (new, 0), (new, new + 1)], 16, 1, 128, dt, cuda_device)
    q = c.rand(c.rows, 4, 128)
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    check_attention(c, q, out, lse)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:, :2]).all()
    assert (out[new:2 * new] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [2, 6, 90, 300])
def test_what_a_row_does_not_see_does_not_reach_it(cuda_device, dt, new):
    """NaN and infinities in keys and values of later tokens, and large visible logits."""
    import long_context_prefill_moba_b200 as M
    L = new + 150
    c = Cache([(new, L)], 16, 2, 64, dt, cuda_device)
    q = c.rand(c.rows, 4, 64)
    want, wlse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    first = new // 2
    poison = [float("nan"), float("inf"), float("-inf")]
    for i, pos in enumerate(range(L - new + first, L)):
        page, slot = int(c.table[0, pos // 16]), pos % 16
        c.v_pool[page, :, slot, i % 64] = poison[i % 3]
        if i % 2:
            c.k_pool[page, :, slot] = poison[(i + 1) % 3]
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:, :first], wlse[:, :first])
    # the first poisoned value (a NaN in channel 0) reaches every row that sees it, and only that channel at first
    assert torch.isnan(out[first:, :, 0]).all()
    assert torch.isfinite(out[first][:, 1:]).all()


@pytest.mark.parametrize("new", [1, 33])
def test_infinite_values_that_are_seen(cuda_device, new):
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 400)], 16, 1, 64, "bf16", cuda_device)
    q = c.rand(c.rows, 4, 64)
    page = int(c.table[0, 2])
    c.v_pool[page, 0, 3, 5] = float("inf")
    c.v_pool[page, 0, 4, 6] = float("-inf")
    out = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index)
    assert (out[..., 5] == float("inf")).all() and (out[..., 6] == float("-inf")).all()
    assert torch.isfinite(out[..., 7:]).all() and torch.isfinite(out[..., :5]).all()


@pytest.mark.parametrize("dt,new", [("bf16", 1), ("bf16", 80), ("f32", 2)])
def test_large_and_growing_logits(cuda_device, dt, new):
    """Logits of some hundreds that grow along the keys: the running maximum moves all the way."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 900)], 32, 1, 128, dt, cuda_device)
    q = c.rand(c.rows, 4, 128)
    for u in range(900):
        c.k_pool[int(c.table[0, u // 32]), 0, u % 32] *= 1 + u / 60
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    check_attention(c, q, out, lse)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 50])
def test_bad_pages_and_lengths_set_the_status(cuda_device, dt, new):
    """Kernel-checked: nothing out of range is followed, the other sequences stay right."""
    import long_context_prefill_moba_b200 as M
    for spoil in ("page", "negative", "length"):
        c = Cache([(new, 100), (new, 90)], 16, 1, 64, dt, cuda_device, max_pages=7)
        q = c.rand(c.rows, 4, 64)
        want = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index)
        cu, kv_len, table = (x.clone() for x in c.index)
        if spoil == "page":
            table[0, 1] = c.pages
        elif spoil == "negative":
            table[0, 1] = -1
        else:
            kv_len[0] = 7 * 16 + 1
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        out = M.moba_cache_attention(q, c.k_pool, c.v_pool, cu, kv_len, table, status=status)
        torch.cuda.synchronize()
        assert int(status) == INTERNAL, spoil
        assert torch.equal(out[new:], want[new:])


def test_offsets_beyond_32_bits(cuda_device):
    """A pool of more than 2^31 elements, the sequences in its last pages."""
    import long_context_prefill_moba_b200 as M
    dev, page, hkv, d = cuda_device, 256, 8, 128
    pages = 2 ** 31 // (page * hkv * d) + 9
    k_pool = torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device=dev)
    v_pool = torch.zeros_like(k_pool)
    for new in (1, 64):
        g = torch.Generator().manual_seed(new)
        k, v, q = (torch.randn(2 * new, h, d, generator=g).to(torch.bfloat16).to(dev) for h in (hkv, hkv, 16))
        cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=dev)
        kv_len = torch.tensor([new, new], dtype=torch.int32, device=dev)
        table = torch.tensor([[pages - 1], [pages - 3]], dtype=torch.int32, device=dev)
        M.moba_cache_append(k, v, cu, kv_len, table, k_pool, v_pool)
        assert torch.equal(k_pool[pages - 1, :, :new].transpose(0, 1), k[:new])
        assert torch.equal(v_pool[pages - 3, :, :new].transpose(0, 1), v[new:])
        out = M.moba_cache_attention(q, k_pool, v_pool, cu, kv_len, table)
        small = M.moba_cache_attention(q, k_pool[-3:].clone(), v_pool[-3:].clone(), cu, kv_len,
                                       torch.tensor([[2], [0]], dtype=torch.int32, device=dev))
        assert torch.equal(out, small)


APPEND = [
    # lens, page, hq (0: no queries), hkv, d, rot, interleaved, norm, dtype, weights, joint
    ([(1, 1)], 16, 4, 1, 128, 128, False, False, "bf16", "bf16", False),
    ([(1, 777), (0, 3), (1, 64), (1, 65)], 64, 32, 8, 128, 128, False, True, "bf16", "f32", True),
    ([(17, 40), (0, 0), (100, 100), (3, 5000)], 32, 6, 3, 64, 32, True, True, "bf16", "bf16", False),
    ([(33, 50), (5, 5)], 16, 0, 2, 64, 64, False, False, "f32", "f32", True),
    ([(1, 9 + i) for i in range(70)], 16, 2, 1, 64, 16, False, True, "f32", "f32", False),
    ([(1, 3) if i % 3 else (0, 8) for i in range(1500)], 16, 1, 1, 64, 64, False, False, "bf16", "bf16", False),
    ([(300, 300)], 256, 8, 8, 128, 0, False, False, "bf16", "bf16", False),
    ([(9, 10 ** 6 + 9)], 4096, 2, 1, 64, 64, False, False, "f32", "f32", False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[8]}-d{c[4]}-rot{c[5]}-p{c[1]}-{len(c[0])}seq")
def test_append(cuda_device, case):
    import long_context_prefill_moba_b200 as M
    lens, page, hq, hkv, d, rot, inter, normed, dt, wt, joint = case
    c = Cache(lens, page, hkv, d, dt, cuda_device, joint=joint, pad=2, nan=False)
    qkv = c.rand(c.rows, hq + 2 * hkv, d)
    q, k, v = (qkv[:, :hq] if hq else None), qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    f = M.moba_rope_inv_freq(rot, 10000.0, cuda_device) if rot else None
    wq, wk = ((1 + 0.5 * torch.randn(d, generator=c.g)).to(DT[wt]).to(cuda_device) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    kb, vb = c.k_pool.clone(), c.v_pool.clone()
    q_out = torch.full((c.rows, hq, d), 7.0, dtype=c.dtype, device=cuda_device) if hq else None
    got = M.moba_cache_append(k, v, *c.index, c.k_pool, c.v_pool, inv_freq=f, q=q, interleaved=inter, eps=1e-5,
                              q_weight=wq if normed and hq else None, k_weight=wk if normed else None, status=status,
                              q_out=q_out)
    torch.cuda.synchronize()
    assert int(status) == 0 and got is q_out
    rows = O.new_tokens(c.cu.numpy(), c.kv_len.numpy())
    pos = np.array([p for _, _, p in rows])
    seq = np.array([b for _, b, _ in rows])
    fn = np64(f) if rot else np.zeros(0)

    def near(x, y, w):
        y = O.norm(y, np64(w), 1e-5) if normed else y
        want = O.rotate(y, pos, fn, inter)
        size = np.abs(y)
        if rot:   # both members of a pair
            i = np.arange(rot // 2)
            ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            size[..., ia] = size[..., ib] = size[..., ia] + size[..., ib]
        assert (np.abs(x - want) <= half_step(c.dtype) * np.abs(want) + 1e-5 * size).all()

    at, slot = c.table.numpy()[seq, pos // page], pos % page
    near(np64(c.k_pool)[at, :, slot], np64(k)[:c.total], wk)
    assert torch.equal(c.v_pool[torch.from_numpy(at).long(), :, torch.from_numpy(slot)], v[:c.total])
    if hq:
        near(np64(q_out)[:c.total], np64(q)[:c.total], wq)
        assert (q_out[c.total:] == 7.0).all()
    # everything else in the pools is as it was
    for p, before in ((c.k_pool, kb), (c.v_pool, vb)):
        rest = p.clone()
        ix = (torch.from_numpy(at).long(), slice(None), torch.from_numpy(slot))
        rest[ix] = before[ix]
        assert torch.equal(rest, before)


def test_append_without_a_page_sets_the_status(cuda_device):
    import long_context_prefill_moba_b200 as M
    for spoil in ("page", "negative", "length", "position"):
        c = Cache([(2, 20), (2, 20)], 16, 1, 64, "bf16", cuda_device, max_pages=2, nan=False)
        k, v, q = c.rand(4, 1, 64), c.rand(4, 1, 64), c.rand(4, 2, 64)
        cu, kv_len, table = (x.clone() for x in c.index)
        kb = c.k_pool.clone()
        if spoil == "page":
            table[0, 1] = c.pages
        elif spoil == "negative":
            table[0, 1] = -1
        elif spoil == "length":
            kv_len[0] = 34
        else:
            kv_len[0] = 0
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        M.moba_cache_append(k, v, cu, kv_len, table, c.k_pool, c.v_pool, status=status, q=q)
        torch.cuda.synchronize()
        assert int(status) == INTERNAL, spoil
        page = int(c.table[1, 1])
        assert torch.equal(c.k_pool[page, :, 2:4].transpose(0, 1), k[2:])
        c.k_pool[page] = kb[page]
        assert torch.equal(c.k_pool, kb)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_serving_a_prompt_in_steps(cuda_device, dt, d):
    """A prompt in chunks, then tokens one by one, as one captured step each kind would serve it: the result at every
    token is the attention of the whole sequence."""
    import long_context_prefill_moba_b200 as M
    dev, hq, hkv, page = cuda_device, 8, 2, 32
    g = torch.Generator().manual_seed(9)
    N = 333
    qkv = torch.randn(N, hq + 2 * hkv, d, generator=g).to(DT[dt]).to(dev)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g)).to(dev), (1 + 0.3 * torch.randn(d, generator=g)).to(dev)
    f = M.moba_rope_inv_freq(d, device=dev)
    pages = -(-N // page)
    table = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32).to(dev)[None]
    k_pool, v_pool = (torch.full((pages + 2, hkv, page, d), float("nan"), dtype=DT[dt], device=dev) for _ in range(2))
    outs, at = [], 0
    for n in [200, 1, 100] + [1] * 32:
        x = qkv[at:at + n]
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        length = torch.tensor([at + n], dtype=torch.int32, device=dev)
        q = M.moba_cache_append(x[:, hq:hq + hkv], x[:, hq + hkv:], cu, length, table, k_pool, v_pool, inv_freq=f, q=x[:, :hq],
                                q_weight=wq, k_weight=wk)
        outs.append(M.moba_cache_attention(q, k_pool, v_pool, cu, length, table))
        at += n
    got = torch.cat(outs)
    assert at == N
    # the training path's norm and rotation, and dense causal MoBA (one block), on the whole sequence
    pos = torch.arange(N, device=dev, dtype=torch.int32)
    q, k = M.moba_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], wq, wk, pos, f)
    c = Cache([(N, N)], page, hkv, d, dt, dev)
    for p, x in ((c.k_pool, k), (c.v_pool, qkv[:, hq + hkv:])):
        for u in range(N):
            p[int(c.table[0, u // page]), :, u % page] = x[u]
    check_attention(c, q, got, None)
    dense = M.moba_forward(q[None], k[None], qkv[None, :, hq + hkv:].contiguous(), N, 1)[0]
    check_attention(c, q, dense, None)


def test_captured_step_is_replayed_with_other_lengths(cuda_device):
    import long_context_prefill_moba_b200 as M
    dev, hq, hkv, d, page = cuda_device, 8, 2, 128, 16
    for new in (1, 40):
        c = Cache([(new, 300), (new, 100)], page, hkv, d, "bf16", dev, nan=False)
        x = c.rand(c.rows, hq + 2 * hkv, d)
        f = M.moba_rope_inv_freq(d, device=dev)

        def step():
            q = M.moba_cache_append(x[:, hq:hq + hkv], x[:, hq + hkv:], *c.index, c.k_pool, c.v_pool, inv_freq=f, q=x[:, :hq])
            return M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index)

        step()
        graphs = []
        for _ in range(2):     # two captured steps, each with its own workspace
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
            graphs.append((graph, out))
        for lens in ([300, 100], [new + 3, 90], [new, 304]):
            c.index[1].copy_(torch.tensor(lens, dtype=torch.int32))
            for graph, out in graphs:
                graph.replay()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(out, want) for _, out in graphs), lens


def test_calls_on_two_streams(cuda_device):
    import long_context_prefill_moba_b200 as M
    cs = [Cache([(n, L), (n, 500)], 32, 2, 128, "bf16", cuda_device, seed=n) for n, L in ((1, 3000), (120, 700))]
    qs = [c.rand(c.rows, 8, 128) for c in cs]
    want = [M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index) for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, c, q in zip(streams, cs, qs):
            with torch.cuda.stream(s):
                got.append(M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))


def test_refusals_with_device_tensors(cuda_device):
    import long_context_prefill_moba_b200 as M
    dev = cuda_device
    c = Cache([(1, 20)], 16, 2, 64, "bf16", dev)
    q = c.rand(1, 4, 64)
    cu, kv_len, table = c.index
    good = dict(q=q, k_pool=c.k_pool, v_pool=c.v_pool, cu_new=cu, kv_len=kv_len, table=table)
    M.moba_cache_attention(**good)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=c.rand(1, 3, 64)), dict(kv_len=kv_len.long()), dict(cu_new=cu[:1]),
                dict(table=table[0]), dict(k_pool=c.k_pool.transpose(1, 2)), dict(v_pool=c.v_pool[:, :1]),
                dict(out=torch.empty(1, 4, 64, device=dev)), dict(table=table.cpu()), dict(q=c.rand(1, 4, 32))):
        with pytest.raises((ValueError, M.MobaError)):
            M.moba_cache_attention(**{**good, **bad})
    k = c.rand(1, 2, 64)
    f = M.moba_rope_inv_freq(64, device=dev)
    good = dict(k=k, v=k, cu_new=cu, kv_len=kv_len, table=table, k_pool=c.k_pool, v_pool=c.v_pool, inv_freq=f)
    for bad in (dict(inv_freq=f.float()), dict(inv_freq=M.moba_rope_inv_freq(8, device=dev)), dict(v=k.float()),
                dict(q=q.float()), dict(q_weight=torch.ones(64, device=dev)), dict(k=c.rand(1, 3, 64)),
                dict(k_weight=torch.ones(32, device=dev)), dict(inv_freq=M.moba_rope_inv_freq(128, device=dev))):
        with pytest.raises((ValueError, M.MobaError)):
            M.moba_cache_append(**{**good, **bad})


@pytest.mark.parametrize("new", [1, 40])
def test_weights_of_a_module_without_gradients(cuda_device, new):
    """Parameters serve under no_grad or inference_mode, or detached; in grad mode the calls refuse them."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 90)], 16, 2, 64, "bf16", cuda_device, nan=False)
    x = c.rand(new, 8, 64)
    w = torch.nn.Parameter(1 + 0.3 * torch.randn(64, generator=c.g).to(cuda_device))

    def step(x, w):
        q = M.moba_cache_append(x[:, 4:6], x[:, 6:], *c.index, c.k_pool, c.v_pool, q=x[:, :4], q_weight=w, k_weight=w)
        return M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index)

    want = step(x, w.detach())
    with torch.no_grad():
        assert torch.equal(step(x, w), want)
    with torch.inference_mode():
        assert torch.equal(step(x, w), want)
    before = c.k_pool.clone()
    with pytest.raises(RuntimeError, match="no gradient"):
        step(x, w)
    with pytest.raises(RuntimeError, match="no gradient"):
        M.moba_cache_attention(x[:, :4].clone().requires_grad_(), c.k_pool, c.v_pool, *c.index)
    torch.cuda.synchronize()
    assert torch.equal(c.k_pool, before)


def test_written_tensors_raise_their_version(cuda_device):
    """A tensor that a backward pass has saved and a call then overwrites is found out by autograd."""
    import long_context_prefill_moba_b200 as M
    for new in (1, 40):
        c = Cache([(new, 90)], 16, 2, 64, "bf16", cuda_device, nan=False)
        x = c.rand(new, 4, 64)
        q = c.rand(new, 4, 64)
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        k_pool, v_pool, out = c.k_pool.clone(), c.v_pool.clone(), torch.empty_like(q)
        at = [t._version for t in (k_pool, v_pool, q, out, status)]
        M.moba_cache_append(x[:, :2], x[:, 2:], *c.index, k_pool, v_pool, q=q, q_out=q, status=status)
        M.moba_cache_attention(q, k_pool, v_pool, *c.index, out=out, status=status)
        assert all(t._version > v for t, v in zip((k_pool, v_pool, q, out, status), at))
        w = torch.ones_like(q, requires_grad=True)
        loss = (w * out).sum()          # saves `out`
        M.moba_cache_attention(q, k_pool, v_pool, *c.index, out=out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        # inputs are only read
        at = q._version
        M.moba_cache_attention(q, k_pool, v_pool, *c.index)
        assert q._version == at


def test_buffers_made_in_inference_mode(cuda_device):
    """They keep no versions, and serve in and out of the mode."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(2, 90)], 16, 2, 64, "bf16", cuda_device, nan=False)
    x = c.rand(2, 8, 64)
    with torch.inference_mode():
        k_pool, v_pool, q_out, out = c.k_pool.clone(), c.v_pool.clone(), torch.empty(2, 4, 64, dtype=c.dtype, device=cuda_device), None

    def step(k_pool, v_pool, q_out):
        q = M.moba_cache_append(x[:, 4:6], x[:, 6:], *c.index, k_pool, v_pool, q=x[:, :4], q_out=q_out)
        return M.moba_cache_attention(q, k_pool, v_pool, *c.index)

    want = step(c.k_pool, c.v_pool, None)
    assert torch.equal(step(k_pool, v_pool, q_out), want)
    with torch.inference_mode():
        assert torch.equal(step(k_pool, v_pool, q_out), want)
    assert torch.equal(k_pool, c.k_pool) and torch.equal(v_pool, c.v_pool)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 50])
def test_one_kv_head_in_slots_before_heads(cuda_device, dt, new):
    """Pools of one head kept as [pages, slots, 1, d]: as the dense ones."""
    import long_context_prefill_moba_b200 as M
    c = Cache([(new, 200), (new, 77)], 16, 1, 64, dt, cuda_device, nan=False)
    x = c.rand(c.rows, 6, 64)
    pools = [torch.empty(c.pages, 16, 1, 64, dtype=c.dtype, device=cuda_device).transpose(1, 2).copy_(p)
             for p in (c.k_pool, c.v_pool)]
    assert pools[0].stride(1) != 16 * 64
    got = []
    for k_pool, v_pool in ((c.k_pool, c.v_pool), pools):
        q = M.moba_cache_append(x[:, 4:5], x[:, 5:], *c.index, k_pool, v_pool, q=x[:, :4])
        got.append(M.moba_cache_attention(q, k_pool, v_pool, *c.index))
    assert torch.equal(*got) and torch.equal(pools[0], c.k_pool) and torch.equal(pools[1], c.v_pool)


def test_calls_from_two_threads(cuda_device):
    """Threads of one process, each with its own stream: the calls give the interpreter's lock back while they run."""
    import threading
    import long_context_prefill_moba_b200 as M
    cs = [Cache([(n, 300), (n, 150)], 32, 2, d, "bf16", cuda_device, seed=d + n) for d in (64, 128) for n in (1, 90)]
    qs = [c.rand(c.rows, 8, c.d) for c in cs]
    got = {}

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got[i] = [M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index) for _ in range(20) for c, q in zip(cs, qs)]
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want = [M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index) for c, q in zip(cs, qs)]
    for i in range(2):
        assert len(got[i]) == 80 and all(torch.equal(x, want[j % 4]) for j, x in enumerate(got[i]))


@pytest.mark.parametrize("dt,d,chunk", [("bf16", 128, 400), ("bf16", 64, 333), ("f32", 128, 300), ("f32", 64, 401)])
def test_a_chunk_among_single_tokens(cuda_device, dt, d, chunk):
    """Few rows a sequence on average, so that the kernels for single tokens take the chunk's long run of row tiles too."""
    import long_context_prefill_moba_b200 as M
    lens = [(1, 200 + 17 * i) for i in range(40)] + [(chunk, chunk + 900)] + [(1, 33)] * 30 + [(0, 5)] * 4
    hq, hkv = 8, 2
    assert sum(n for n, _ in lens) * (hq // hkv) <= 32 * len(lens)
    c = Cache(lens, 32, hkv, d, dt, cuda_device, pad=2)
    q = c.rand(c.rows, hq, d)
    out, lse = M.moba_cache_attention(q, c.k_pool, c.v_pool, *c.index, return_lse=True)
    check_attention(c, q, out, lse, rows=list(range(0, 40, 7)) + list(range(39, c.total, 23)) + [39 + chunk, c.total - 1])
