"""Cases of the serving and training operators beside MoBA attention: the per-head norm of queries and
keys with the position rotation (forward and gradients), the append of keys and values to a paged
cache, and the attention of new tokens over that cache.

`run` computes a case in plain torch operations, or, where the module's `own` is set, with the
library's kernels.  `exact` gives the same outputs in 64 bits, from the formulas.

Formulas (x a head of d numbers at position p, w the norm's weights, f the rotation's frequencies):
  y = x / sqrt(mean(x^2) + eps) * w
  pair i of the rotated part (a, b) -> (a cos(p f_i) - b sin(p f_i), b cos(p f_i) + a sin(p f_i)),
  (a, b) = (y[i], y[i + rot/2]), or (y[2i], y[2i + 1]) where pairs are interleaved
  attention of the new token at position p over its sequence: softmax over the keys at positions
  u <= p of scale <q, k_u>, times v_u; query head h reads kv head h // (hq / hkv)
A sequence's position u is in page table[u // page], slot u % page, of pools [pages, hkv, page, d]."""
import math

import torch

own = False

EPS = 1e-6
BASE = 500000.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # norm and rotation of the queries and keys of one decode step of eight sequences
        dict(name="norm_rope 8 tokens", op="norm_rope", grad=False, tokens=8, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16", far=131072),
        # a training step of a 32K-token sequence: forward, then all gradients
        dict(name="norm_rope train 32768", op="norm_rope", grad=True, tokens=32768, hq=32, hkv=8, d=128,
             rot=128, interleaved=False, dtype="bf16", far=32768),
        # an fp32 training step with head_dim 64, half of it rotated, interleaved pairs, an odd length
        dict(name="norm_rope train f32 5003", op="norm_rope", grad=True, tokens=5003, hq=16, hkv=16, d=64,
             rot=32, interleaved=True, dtype="f32", far=10485760),
        # the cache update of one decode step of 64 sequences
        dict(name="append 64 tokens", op="append", batch=64, new=1, ctx=32768, hq=32, hkv=8, d=128, page=64,
             rot=128, norm=False, dtype="bf16"),
        # chunked prefill of eight prompts, with the per-head norm
        dict(name="append chunks", op="append", batch=8, new=4096, ctx=16384, hq=32, hkv=8, d=128, page=128,
             rot=128, norm=True, dtype="bf16"),
        # fp32, small pages, part of the head rotated, odd lengths
        dict(name="append f32 odd", op="append", batch=5, new=333, ctx=1501, hq=16, hkv=4, d=64, page=16,
             rot=32, norm=False, dtype="f32"),
        # the smallest step: one sequence, one token, a thousand cached tokens
        dict(name="decode 1 x 1000", op="attention", batch=1, new=1, ctx=999, hq=4, hkv=1, d=128, page=16,
             dtype="bf16"),
        # a decode step of 64 sequences of different lengths
        dict(name="decode 64 ragged", op="attention", batch=64, new=1, ctx=16384, hq=32, hkv=8, d=128, page=64,
             dtype="bf16"),
        # a decode step of one 128K-token sequence
        dict(name="decode 1 x 131072", op="attention", batch=1, new=1, ctx=131071, hq=32, hkv=8, d=128, page=256,
             dtype="bf16"),
        # a serving step that mixes chunks of several lengths, head_dim 64
        dict(name="chunks d64 ragged", op="attention", batch=6, new=701, ctx=9000, hq=16, hkv=4, d=64, page=32,
             dtype="bf16"),
        # fp32 chunks
        dict(name="chunks f32", op="attention", batch=3, new=257, ctx=1900, hq=16, hkv=16, d=64, page=64,
             dtype="f32"),
        # chunked prefill deep in a 128K-token prompt
        dict(name="chunk 4096 at 131072", op="attention", batch=1, new=4096, ctx=126976, hq=32, hkv=8, d=128,
             page=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(32, 8), (16, 16), (4, 1), (16, 4), (8, 8), (16, 2)])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = dict(hq=heads[0], hkv=heads[1], d=d, dtype=dtype)
    kind = rng.choice(["norm_rope", "norm_rope", "append", "decode", "decode", "chunk"])
    if kind == "norm_rope":
        return dict(case, op="norm_rope", grad=rng.random() < 0.6, tokens=_log_int(rng, 1, 32768 if dtype == "bf16" else 12000),
                    rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4, far=_log_int(rng, 40000, 10485760))
    case["page"] = rng.choice([16, 32, 64, 128, 256])
    if kind == "append":
        batch = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(3, 16384 // batch))
        return dict(case, op="append", batch=batch, new=new, ctx=_log_int(rng, 1, max(2, 200000 // batch)),
                    rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.5)
    case["op"] = "attention"
    if kind == "decode":
        batch = _log_int(rng, 1, 64)
        return dict(case, batch=batch, new=rng.choice([1, 1, 1, 2, 5]),
                    ctx=_log_int(rng, 100, (500000 if dtype == "bf16" else 60000) // batch))
    batch = _log_int(rng, 1, 8)
    most = 2048 if dtype == "bf16" else 300
    return dict(case, batch=batch, new=_log_int(rng, 16, most // batch + 16),
                ctx=_log_int(rng, 1, (65536 if dtype == "bf16" else 8192) // batch))


# ---- inputs --------------------------------------------------------------------------------
def _lengths(case):
    """(new tokens, total length) of each sequence: they fall off from the case's largest; every fifth of a
    batch of chunks has no new token."""
    got = []
    for b in range(case["batch"]):
        if b == 0:
            new, old = case["new"], case["ctx"]
        else:
            old = case["ctx"] - case["ctx"] * ((b * 37 + 11) % 64) // 80
            new = case["new"] - case["new"] * ((b * 29 + 5) % 64) // 70
            if case["new"] > 16 and b % 5 == 4:
                new = 0
        got.append((new, old + new))
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, hq, hkv, d = TYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = {"case": case}
    if "rot" in case:
        # the rotation's frequencies, in 64 bits
        s["inv_freq"] = BASE ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
    if case["op"] == "norm_rope" or case.get("norm"):
        # weights as after some training: around 1, some channels far from it
        s["q_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dt)
        s["k_weight"] = (1 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(dt)
    if case["op"] == "norm_rope":
        t = case["tokens"]
        # queries, keys and values are parts of one projection's rows
        qkv = normal(t, hq + 2 * hkv, d)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        if case["grad"]:  # consecutive positions of a training sequence, up to the furthest
            s["positions"] = torch.arange(case["far"] - t, case["far"], device=dev, dtype=torch.int32)
            s["dq"], s["dk"] = normal(t, hq, d), normal(t, hkv, d)
        else:
            s["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device=dev, dtype=torch.int32)
        return s

    lens, page = _lengths(case), case["page"]
    total = sum(n for n, _ in lens)
    pages = [-(-length // page) for _, length in lens]
    s["lens"], s["max_pages"] = lens, max(pages)
    ids = torch.randperm(sum(pages) + 3, generator=gen, device=dev).to(torch.int32)  # 3 pages stay free
    table = torch.full((case["batch"], max(pages)), -1, device=dev, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    s["table"] = table
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s["cu_new"] = torch.tensor(cu, device=dev, dtype=torch.int32)
    s["kv_len"] = torch.tensor([length for _, length in lens], device=dev, dtype=torch.int32)
    s["k_pool"], s["v_pool"] = (normal(sum(pages) + 3, hkv, page, d) for _ in range(2))
    if case["op"] == "append":
        qkv = normal(total, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"] = normal(total, hq, d)
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        return _run_norm_rope(state, case)
    if case["op"] == "append":
        return _run_append(state, case)
    return _run_attention(state, case)


def _run_norm_rope(s, case):
    q, k, wq, wk = (s[x] for x in ("q", "k", "q_weight", "k_weight"))
    if case["grad"]:
        q, k, wq, wk = (x.detach().requires_grad_() for x in (q, k, wq, wk))
    if own:
        import long_context_prefill_moba_b200 as M
        outs = M.moba_norm_rope(q, k, wq, wk, s["positions"], s["inv_freq"], eps=EPS, interleaved=case["interleaved"])
    else:
        cs = _angles(s["positions"], s["inv_freq"])
        outs = tuple(_rotated(_normed(x, w), cs, case["interleaved"]).to(x.dtype) for x, w in ((q, wq), (k, wk)))
    if not case["grad"]:
        return outs
    return outs + torch.autograd.grad(outs, (q, k, wq, wk), (s["dq"], s["dk"]))


def _run_append(s, case):
    if own:
        import long_context_prefill_moba_b200 as M
        q = M.moba_cache_append(s["k"], s["v"], s["cu_new"], s["kv_len"], s["table"], s["k_pool"], s["v_pool"],
                                inv_freq=s["inv_freq"], q=s["q"], q_weight=s.get("q_weight"), k_weight=s.get("k_weight"),
                                eps=EPS)
        return q, s["k_pool"], s["v_pool"]
    page = case["page"]
    total = s["q"].shape[0]
    row = torch.arange(total, device=s["q"].device)
    b = torch.searchsorted(s["cu_new"][1:], row, right=True)  # the sequence of each new token
    pos = s["kv_len"][b] - s["cu_new"][b + 1] + row
    cs = _angles(pos, s["inv_freq"])
    q, k = s["q"].float(), s["k"].float()
    if case["norm"]:
        q, k = _normed(q, s["q_weight"]), _normed(k, s["k_weight"])
    where = s["table"][b, pos // page].long()
    s["k_pool"][where, :, pos % page] = _rotated(k, cs, False).to(s["k"].dtype)
    s["v_pool"][where, :, pos % page] = s["v"]
    return _rotated(q, cs, False).to(s["q"].dtype), s["k_pool"], s["v_pool"]


def _run_attention(s, case):
    if own:
        import long_context_prefill_moba_b200 as M
        return M.moba_cache_attention(s["q"], s["k_pool"], s["v_pool"], s["cu_new"], s["kv_len"], s["table"],
                                      return_lse=True)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(hq, s["q"].shape[0], device=out.device, dtype=torch.float32)
    first = 0
    for b, (new, length) in enumerate(s["lens"]):
        if new == 0:
            continue
        at = s["table"][b, :-(-length // page)].long()
        k, v = (p[at].transpose(0, 1).reshape(hkv, -1, d)[:, :length].float() for p in (s["k_pool"], s["v_pool"]))
        key = torch.arange(length, device=out.device)
        step = max(1, (1 << 28) // (hq * length))  # new tokens at a time: a GiB of scores
        for lo in range(0, new, step):
            hi = min(new, lo + step)
            q = s["q"][first + lo:first + hi].float().reshape(hi - lo, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            z = (q.reshape(hkv, -1, d) @ k.transpose(1, 2)).view(hkv, hq // hkv, hi - lo, length) * d ** -0.5
            z = z.masked_fill(key > length - new + torch.arange(lo, hi, device=key.device).unsqueeze(1), -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            o = (p.view(hkv, -1, length) @ v).view(hkv, hq // hkv, hi - lo, d) / total
            out[first + lo:first + hi] = o.permute(2, 0, 1, 3).reshape(hi - lo, hq, d).to(out.dtype)
            lse[:, first + lo:first + hi] = (top + torch.log(total)).view(hq, hi - lo)
        first += new
    return out, lse


def _angles(pos, inv_freq):
    """cos and sin of the rotation, [tokens, 1, rot / 2]: angles in 64 bits, far positions times small steps."""
    a = pos.double()[:, None, None] * inv_freq
    return torch.cos(a).float(), torch.sin(a).float()


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(y, cs, interleaved):
    cos, sin = cs
    half = cos.shape[-1]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, y[..., 2 * half:]), -1)


# ---- what a pass cannot do without ---------------------------------------------------------
def work(case):
    hq, hkv, d, size = case["hq"], case["hkv"], case["d"], SIZE[case["dtype"]]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (hq + hkv) * d
        passes = 5 if case["grad"] else 2  # x, y; and the gradients' x, dy, dx
        return {"bytes": n * size * passes + 4 * case["tokens"], "flops": n * (30 if case["grad"] else 8)}
    lens = [(n, length) for n, length in _lengths(case) if n > 0]
    total = sum(n for n, _ in lens)
    if case["op"] == "append":
        n = total * (hq + 2 * hkv) * d
        return {"bytes": 2 * n * size, "flops": total * (hq + hkv) * d * (8 if case["norm"] else 3)}
    pairs = sum(n * (length - n) + n * (n + 1) // 2 for n, length in lens)
    cached = sum(length for _, length in lens)
    return {"bytes": 2 * cached * hkv * d * size + 2 * total * hq * d * size + 4 * total * hq,
            "flops": 4 * d * hq * pairs}


# ---- the definition in 64 bits -------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        turn = _turns(s["positions"], s["inv_freq"], case["d"], case["interleaved"])
        outs, grads, wgrads = [], [], []
        for x, w, dy in ((s["q"], s["q_weight"], s.get("dq")), (s["k"], s["k_weight"], s.get("dk"))):
            x, w = x.double(), w.double()
            r = (x.square().sum(-1, keepdim=True) / case["d"] + EPS) ** -0.5
            outs.append(_turned(x * r * w, turn, 1))
            if case["grad"]:
                dz = _turned(dy.double(), turn, -1)  # the transposed rotation turns back
                g = dz * w
                grads.append(r * g - x * r ** 3 * (x * g).sum(-1, keepdim=True) / case["d"])
                wgrads.append((dz * x * r).sum((0, 1)))
        return tuple(outs + grads + wgrads)
    page, lens = case["page"], s["lens"]
    if case["op"] == "append":
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
        q_out, first = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device), 0
        for b, (new, length) in enumerate(lens):
            pos = torch.arange(length - new, length, device=q_out.device)
            rows = slice(first, first + new)
            turn = _turns(pos, s["inv_freq"], case["d"], False)
            q, k = s["q"][rows].double(), s["k"][rows].double()
            if case["norm"]:
                q = q * (q.square().mean(-1, keepdim=True) + EPS) ** -0.5 * s["q_weight"].double()
                k = k * (k.square().mean(-1, keepdim=True) + EPS) ** -0.5 * s["k_weight"].double()
            q_out[rows] = _turned(q, turn, 1)
            at = s["table"][b].long()[torch.div(pos, page, rounding_mode="floor")]
            k_pool[at, :, pos % page] = _turned(k, turn, 1)
            v_pool[at, :, pos % page] = s["v"][rows].double()
            first += new
        return q_out, k_pool, v_pool
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(hq, out.shape[0], dtype=torch.float64, device=out.device)
    first = 0
    for b, (new, length) in enumerate(lens):
        at = s["table"][b].long()[torch.arange(length, device=out.device) // page]
        slot = torch.arange(length, device=out.device) % page
        for h in range(hq if new else 0):
            k, v = s["k_pool"][at, h // (hq // hkv), slot].double(), s["v_pool"][at, h // (hq // hkv), slot].double()
            for lo in range(0, new, 2048):
                hi = min(new, lo + 2048)
                z = s["q"][first + lo:first + hi, h].double() @ k.t() / math.sqrt(d)
                last = torch.arange(lo, hi, device=out.device) + (length - new)
                z[torch.arange(length, device=out.device)[None, :] > last[:, None]] = -math.inf
                lse[h, first + lo:first + hi] = torch.logsumexp(z, -1)
                out[first + lo:first + hi, h] = torch.softmax(z, -1) @ v
        first += new
    return out, lse


def _turns(pos, inv_freq, d, interleaved):
    """Each channel's partner, and the cos and signed sin it is turned with, [tokens, 1, d]."""
    half = inv_freq.numel()
    partner = torch.arange(d, device=pos.device)
    sign, which = torch.zeros(d, dtype=torch.float64, device=pos.device), torch.zeros(d, dtype=torch.long, device=pos.device)
    i = torch.arange(half, device=pos.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    partner[a], partner[b] = b, a
    sign[a], sign[b] = -1.0, 1.0
    which[a], which[b] = i, i
    angle = (pos.double()[:, None] * inv_freq[which][None, :] * (sign != 0))[:, None, :]
    return partner, torch.cos(angle), torch.sin(angle) * sign


def _turned(y, turn, way):
    partner, cos, sin = turn
    return y * cos + way * y[..., partner] * sin
