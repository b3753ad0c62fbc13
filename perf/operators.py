"""The prompt and 4-bit cache operators as cases: plain torch forms, the library's calls and a 64-bit form.

Operators (``op`` of a case):

- ``rope``: head norm and rotary embedding of packed projections (``dq.qkv_rope``);
- ``prompt``: causal grouped-head attention of packed sequences (``dq.attention_prompt``);
- ``append``: rows quantised into a paged 4-bit cache, then read back (``dq.kv4_append``, ``dq.kv4_read``);
- ``read``: rows of a paged 4-bit cache as values (``dq.kv4_read``);
- ``decode``: one token a sequence over a paged 4-bit cache (``dq.attention_decode_kv4``).

The 4-bit cache holds 16 keys of one KV head in a block of 2560 bytes:

- bytes 0..1023, key codes: key j at 64 j; its 32-bit word 4 t + g (t, g in 0..3) holds dims
  32 g + 8 t + e (e in 0..7), even e = 2 i at bits 4 i, odd e = 2 i + 1 at bits 16 + 4 i;
- bytes 1024..2047, value codes: 16-bit half (j & 1) of the word at 512 (j >> 3) +
  16 (4 r + ((j >> 1) & 3)) + 4 g holds dims 32 g + 4 r + i (r in 0..7, i in 0..3) at bits 4 i;
- bytes 2048..2303 key and 2304..2559 value scales: at 32 (j >> 1) + 8 g four binary16 values, d of the
  even key, d of the odd key, then z of the even and of the odd key, for dims 32 g .. 32 g + 31.

A value is d (c - 8) + z.  d = f16(f32(max - min) / 15), z = f16(min + 8 d), c = (x - z) / d rounded
to even, + 8, kept in 0..15, each step one 32-bit operation; a group with d = 0 has c = 8.
"""
import math
import random

import numpy as np
import torch

own = False

HD = 128
GROUP = 32
BLOCK_KEYS, BLOCK_BYTES = 16, 2560
EPS, THETA = 1e-6, 1.0e6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases


def listed():
    q = dict(n_q=32, n_kv=8)  # the decode benchmark's heads
    return [
        # one decode token's projections, fp32 as the GEMVs leave them: latency
        dict(name="rope 1 token", op="rope", rows=1, max_ctx=4096, norm=True, type="f32", **q),
        # a long prompt's projections on their way to the prompt attention: bandwidth
        dict(name="rope 8191 tokens", op="rope", rows=8191, max_ctx=8192, norm=True, type="f16", **q),
        # one long prompt from its first token on
        dict(name="prompt 8192", op="prompt", n_seq=1, max_len=8192, min_len=8192, past=0, mix=0, planes=False,
             type="f16", **q),
        # a serving batch of prompts of very different lengths, one-token and empty ones among them
        dict(name="prompt packed ragged", op="prompt", n_seq=12, max_len=2000, min_len=0, past=0, mix=3, planes=False,
             type="bf16", **q),
        # the next 64 tokens of a long conversation against the fp16 cache planes of one layer
        dict(name="prompt 64 after 16000", op="prompt", n_seq=1, max_len=64, min_len=64, past=16000, mix=0, planes=True,
             type="f16", **q),
        # eight sequences' new tokens
        dict(name="append 8 tokens", op="append", rows=8, n_kv=8, page=64, pages=64, type="f32"),
        # a long prompt's keys and values
        dict(name="append 8000 tokens", op="append", rows=8000, n_kv=8, page=64, pages=160, type="f16"),
        # a short shared prefix read back as the next chunk's keys
        dict(name="read 100 tokens", op="read", rows=100, n_kv=8, page=16, pages=64, type="f16"),
        # a long conversation read back for a chunk of a prompt
        dict(name="read 16000 tokens", op="read", rows=16000, n_kv=8, page=64, pages=300, type="bf16"),
        # one conversation of the benchmark's length: latency
        dict(name="decode 1 x 513", op="decode", n_seq=1, max_len=513, min_len=513, mix=0, page=64, type="f32", **q),
        # one very long conversation: the keys split over the whole card
        dict(name="decode 1 x 100001", op="decode", n_seq=1, max_len=100001, min_len=100001, mix=0, page=64, type="f32",
             **q),
        # a serving batch of different lengths
        dict(name="decode 48 ragged", op="decode", n_seq=48, max_len=12000, min_len=1, mix=7, page=32, type="f16", **q),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "append", "read", "decode"])
    n_q, n_kv = rng.choice([(32, 8), (16, 8), (16, 2), (12, 2), (4, 4), (6, 2), (8, 1), (5, 1), (21, 3)])
    if op == "rope":
        rows = _log_int(rng, 1, 8191)
        return dict(op=op, rows=rows, n_q=n_q, n_kv=n_kv, max_ctx=rows + rng.randrange(1, 4096), norm=rng.random() < 0.8,
                    type=rng.choice(["f32", "f16", "bf16"]))
    if op == "prompt":
        n_seq = _log_int(rng, 1, 16)
        longest = _log_int(rng, 1, max(1, 4096 // n_seq))
        return dict(op=op, n_seq=n_seq, max_len=longest, min_len=rng.choice([0, 1, longest]),
                    past=rng.choice([0, 0, _log_int(rng, 1, 4096)]), mix=rng.randrange(1 << 20), planes=rng.random() < 0.3,
                    n_q=n_q, n_kv=n_kv, type=rng.choice(["f16", "bf16"]))
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op in ("append", "read"):
        rows = _log_int(rng, 1, 8000)
        return dict(op=op, rows=rows, n_kv=n_kv, page=page, pages=-(-rows // page) + rng.randrange(1, 30),
                    type=rng.choice(["f32", "f16", "bf16"]))
    n_seq = _log_int(rng, 1, 64)
    longest = _log_int(rng, 1, max(2, 250000 // n_seq // n_kv))
    return dict(op=op, n_seq=n_seq, max_len=longest, min_len=rng.choice([0, 1, longest]), mix=rng.randrange(1 << 20),
                page=page, n_q=n_q, n_kv=n_kv, type=rng.choice(["f32", "f16", "bf16"]))


def _lengths(case):
    r = random.Random(case["mix"])
    lo, hi = case["min_len"], case["max_len"]
    n = [r.randint(lo, hi) for _ in range(case["n_seq"])]
    if lo < hi and len(n) > 2:
        n[1], n[2] = lo, 1
    n[0] = hi
    return n


def _visible(lq, lk):
    """Pairs (query i, key j <= i + lk - lq) of one sequence."""
    return sum(max(0, min(lk, i + lk - lq + 1)) for i in range(lq)) if lk < lq else lq * (lk - lq) + lq * (lq + 1) // 2


def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["n_q"] + 2 * case["n_kv"]
        n = case["rows"] * heads * HD
        turned = case["rows"] * (case["n_q"] + case["n_kv"]) * HD
        return {"bytes": n * (4 + BYTES[case["type"]]) + case["rows"] * (4 + 4 * HD), "flops": turned * 7}
    if op == "prompt":
        n = _lengths(case)
        lk = [a + case["past"] for a in n]
        pairs = sum(_visible(a, b) for a, b in zip(n, lk))
        return {"bytes": 2 * HD * (2 * sum(n) * case["n_q"] + 2 * sum(lk) * case["n_kv"]),
                "flops": 4 * HD * case["n_q"] * pairs}
    if op == "append":  # stored, then read back as fp32
        n = case["rows"] * case["n_kv"]
        return {"bytes": n * (2 * HD * BYTES[case["type"]] + 320 + 2 * HD * 4), "flops": n * 2 * HD * 8}
    if op == "read":
        n = case["rows"] * case["n_kv"]
        return {"bytes": n * (160 + 2 * HD * BYTES[case["type"]]), "flops": n * 2 * HD * 2}
    keys = sum(_lengths(case))
    return {"bytes": keys * case["n_kv"] * 160 + 2 * case["n_seq"] * case["n_q"] * HD * BYTES[case["type"]],
            "flops": keys * case["n_q"] * 4 * HD}


# ------------------------------------------------------ the 4-bit cache's layout


def _quantise(x):
    """fp32 [..., 128] -> d, z fp32 [..., 4] (binary16 values) and codes int32 [..., 128]."""
    g = x.reshape(*x.shape[:-1], HD // GROUP, GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    d = ((hi - lo) / torch.full_like(lo, 15.0)).half().float()  # a divided tensor: a number would be inverted first
    z = (lo + 8.0 * d).half().float()
    t = torch.round((g - z[..., None]) / d[..., None]) + 8.0
    c = torch.where(d[..., None] > 0, t.clamp(0.0, 15.0), torch.full_like(t, 8.0))
    return d, z, c.to(torch.int32).reshape(x.shape)


def _pack(kd, kz, kc, vd, vz, vc):
    """Scales [blocks, 16, 4] and codes [blocks, 16, 128] of keys and values -> uint8 [blocks, 2560]."""
    n = kc.shape[0]
    nib = torch.arange(2, device=kc.device)
    # key codes: [n, key, g, t, i, odd] -> byte 2 odd + (i >> 1), nibble i & 1
    a = kc.reshape(n, 16, 4, 4, 2, 2, 2).permute(0, 1, 3, 2, 6, 4, 5)  # n, key, t, g, odd, i >> 1, i & 1
    ks = (a << (4 * nib)).sum(-1).to(torch.uint8).reshape(n, 1024)
    # value codes: [n, half, quad, odd, g, r, i >> 1, i & 1]
    b = vc.reshape(n, 2, 4, 2, 4, 8, 2, 2).permute(0, 1, 5, 2, 4, 3, 6, 7)  # n, half, r, quad, g, odd, i >> 1, i & 1
    vs = (b << (4 * nib)).sum(-1).to(torch.uint8).reshape(n, 1024)

    def scales(d, z):
        p = torch.stack([d, z], -1).half().reshape(n, 8, 2, 4, 2).permute(0, 1, 3, 4, 2)  # n, pair, g, d|z, odd
        return p.contiguous().view(torch.uint8).reshape(n, 256)

    return torch.cat([ks, vs, scales(kd, kz), scales(vd, vz)], 1)


def _unpack(blocks):
    """uint8 [n, 2560] -> fp32 keys and values [n, 16, 128]."""
    n = blocks.shape[0]
    nib = torch.arange(2, device=blocks.device, dtype=torch.uint8) * 4

    def codes(x):
        return ((x[..., None] >> nib) & 15).float() - 8.0

    def scales(x):
        p = x.contiguous().view(torch.float16).float().reshape(n, 8, 4, 2, 2).permute(3, 0, 1, 4, 2).reshape(2, n, 16, 4, 1)
        return p[0], p[1]

    k = codes(blocks[:, :1024].reshape(n, 16, 4, 4, 2, 2)).permute(0, 1, 3, 2, 5, 6, 4).reshape(n, 16, 4, GROUP)
    v = codes(blocks[:, 1024:2048].reshape(n, 2, 8, 4, 4, 2, 2)).permute(0, 1, 3, 5, 4, 2, 6, 7).reshape(n, 16, 4, GROUP)
    kd, kz = scales(blocks[:, 2048:2304])
    vd, vz = scales(blocks[:, 2304:])
    return (k * kd + kz).reshape(n, 16, HD), (v * vd + vz).reshape(n, 16, HD)


def _rows_of(pool, slots, page):
    """fp32 keys and values [rows, n_kv, 128] of the cache rows ``slots`` (page * page size + offset)."""
    n_kv = pool.shape[1]
    s = slots.long()
    pg, blk, key = s // page, s % page // BLOCK_KEYS, s % BLOCK_KEYS
    at = ((pg[:, None] * n_kv + torch.arange(n_kv, device=s.device)) * (page // BLOCK_KEYS) + blk[:, None]).reshape(-1)
    every, where = torch.unique(at, return_inverse=True)
    k, v = _unpack(pool.reshape(-1, BLOCK_BYTES)[every])
    key = key.repeat_interleave(n_kv)
    shape = (len(slots), n_kv, HD)
    return k[where, key].reshape(shape), v[where, key].reshape(shape)


def _random_pool(gen, pages, n_kv, page):
    """A cache whose every row holds quantised normal keys and values, some channels of the keys larger."""
    n = pages * n_kv * (page // BLOCK_KEYS)
    out = torch.empty((n, BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    wide = 1.0 + 3.0 * (torch.rand(HD, device="cuda", generator=gen) < 0.05).float()
    for a in range(0, n, 1 << 14):
        m = min(n, a + (1 << 14)) - a
        k = torch.randn((m, 16, HD), device="cuda", generator=gen) * wide
        v = torch.randn((m, 16, HD), device="cuda", generator=gen)
        out[a:a + m] = _pack(*_quantise(k), *_quantise(v))
    return out.reshape(pages, n_kv, page // BLOCK_KEYS, BLOCK_BYTES)


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    op, s = case["op"], {"case": case}
    if op == "rope":
        heads = case["n_q"] + 2 * case["n_kv"]
        s["qkv"] = randn(case["rows"], heads * HD)
        s["positions"] = (torch.arange(case["rows"], device="cuda") + seed % (case["max_ctx"] - case["rows"] + 1)).int()
        s["q_norm"], s["k_norm"] = 1 + 0.1 * randn(HD), 1 + 0.1 * randn(HD)
        angle = (torch.arange(case["max_ctx"], device="cuda", dtype=torch.float64)[:, None]
                 / THETA ** (torch.arange(HD // 2, device="cuda", dtype=torch.float64) / (HD // 2)))
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    elif op == "prompt":
        t = TYPES[case["type"]]
        n = _lengths(case)
        lk = [a + case["past"] for a in n]
        if case["planes"]:  # cache planes [n_kv][rows][128], as the decode step keeps them
            k, v = (randn(case["n_kv"], sum(lk) + 16, HD).to(t).transpose(0, 1)[:max(1, sum(lk))] for _ in range(2))
            q = randn(max(1, sum(n)), case["n_q"], HD).to(t)
        else:  # queries, keys and values as three slices of one projection where their counts agree
            a, b = case["n_q"], case["n_kv"]
            if case["past"] == 0:
                qkv = randn(max(1, sum(n)), a + 2 * b, HD).to(t)
                q, k, v = qkv[:, :a], qkv[:, a:a + b], qkv[:, a + b:]
            else:
                q = randn(max(1, sum(n)), a, HD).to(t)
                k, v = randn(max(1, sum(lk)), b, HD).to(t), randn(max(1, sum(lk)), b, HD).to(t)
        s["q"], s["k"], s["v"] = q, k, v
        s["cu_q"] = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(np.cumsum([0] + lk), dtype=torch.int32, device="cuda")
        s["max_q"], s["max_k"] = max(n), max(lk)
    elif op in ("append", "read"):
        rows = case["rows"]
        # the rows of one sequence: consecutive offsets of scattered pages, from an odd offset on
        pages = torch.randperm(case["pages"], device="cuda", generator=gen)
        first = min(seed % 7, case["pages"] * case["page"] - rows)
        at = torch.arange(rows, device="cuda") + first
        s["slots"] = (pages[at // case["page"]] * case["page"] + at % case["page"]).int()
        if op == "append":
            t = TYPES[case["type"]]
            s["k"], s["v"] = randn(rows, case["n_kv"], HD).to(t), randn(rows, case["n_kv"], HD).to(t)
            s["pool"] = torch.zeros((case["pages"], case["n_kv"], case["page"] // BLOCK_KEYS, BLOCK_BYTES),
                                    dtype=torch.uint8, device="cuda")
        else:
            s["pool"] = _random_pool(gen, case["pages"], case["n_kv"], case["page"])
    else:
        n, page = _lengths(case), case["page"]
        wide = max(1, -(-max(n) // page))
        need = [-(-a // page) for a in n]
        pages = sum(need) + 3
        s["pool"] = _random_pool(gen, pages, case["n_kv"], page)
        order = torch.randperm(pages, device="cuda", generator=gen).int()
        first = np.cumsum([0] + need[:-1])
        at = torch.tensor(first, device="cuda")[:, None] + torch.arange(wide, device="cuda")
        s["pages"] = order[at.clamp(max=pages - 1)].contiguous()
        s["n_keys"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["max_keys"] = max(1, max(n))
        s["q"] = randn(case["n_seq"], case["n_q"], HD).to(TYPES[case["type"]])
    return s


# ------------------------------------------------------------- the plain forms


def _plain_rope(s):
    case = s["case"]
    n_q, n_kv = case["n_q"], case["n_kv"]
    x = s["qkv"].reshape(case["rows"], n_q + 2 * n_kv, HD)
    cs = s["rope"][s["positions"].long()][:, None]

    def turned(v, w):
        if case["norm"]:
            v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
        a, b = v[..., :HD // 2], v[..., HD // 2:]
        c, d = cs[..., 0], cs[..., 1]
        return torch.cat([a * c - b * d, b * c + a * d], -1)

    t = TYPES[case["type"]]
    return (turned(x[:, :n_q], s["q_norm"]).to(t), turned(x[:, n_q:n_q + n_kv], s["k_norm"]).to(t),
            x[:, n_q + n_kv:].to(t))


def _plain_prompt(s):
    q, k, v, cu_q, cu_k = s["q"], s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long()
    n_q, n_kv = q.shape[1], k.shape[1]
    max_q, max_k = max(1, s["max_q"]), max(1, s["max_k"])
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    iq, ik = torch.arange(max_q, device=q.device), torch.arange(max_k, device=q.device)
    rows = (cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1)
    cols = (cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)
    qp = q[rows].float().transpose(1, 2).unflatten(1, (n_kv, n_q // n_kv))  # seq, kv, group, i, dim
    kp = k[cols].float().transpose(1, 2)[:, :, None]
    vp = v[cols].float().transpose(1, 2)[:, :, None]
    seen = (ik < lk[:, None])[:, None, :] & (ik[None, None, :] <= (iq[None, :] + (lk - lq)[:, None])[:, :, None])
    seen = seen[:, None, None]
    p = (qp @ kp.transpose(-1, -2)) * (1.0 / math.sqrt(HD))
    p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    o = (p @ vp) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.flatten(1, 2).transpose(1, 2).to(q.dtype)  # seq, i, head, dim
    out = torch.zeros((q.shape[0], n_q, HD), dtype=q.dtype, device=q.device)
    live = iq < lq[:, None]
    out[rows[live]] = o[live]
    return out


def _plain_append(s):
    def kept(x):
        d, z, c = _quantise(x.float())
        return c.sub(8).float() * d.repeat_interleave(GROUP, -1) + z.repeat_interleave(GROUP, -1)

    return kept(s["k"]), kept(s["v"])


def _plain_read(s):
    t = TYPES[s["case"]["type"]]
    k, v = _rows_of(s["pool"], s["slots"], s["case"]["page"])
    return k.to(t), v.to(t)


def _plain_decode(s):
    case, q, pool, n_keys = s["case"], s["q"], s["pool"], s["n_keys"].long()
    n_seq, n_q = q.shape[:2]
    n_kv, per = pool.shape[1:3]
    pages = s["pages"].long()
    blocks = pool[pages.reshape(-1)].transpose(1, 2)  # seq * pages, blocks, kv, bytes
    k, v = _unpack(blocks.reshape(-1, BLOCK_BYTES))
    shape = (n_seq, pages.shape[1] * per, n_kv, BLOCK_KEYS, HD)
    k, v = (x.reshape(shape).transpose(1, 2).reshape(n_seq, n_kv, -1, HD) for x in (k, v))
    qg = q.float().reshape(n_seq, n_kv, n_q // n_kv, HD)
    p = (qg @ k.transpose(-1, -2)) * (1.0 / math.sqrt(HD))
    seen = torch.arange(k.shape[2], device=q.device) < n_keys[:, None]
    p = p.masked_fill(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = (p - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp()
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.reshape(n_seq, n_q, HD).to(q.dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        plain = {"rope": _plain_rope, "prompt": _plain_prompt, "append": _plain_append, "read": _plain_read,
                 "decode": _plain_decode}
        return plain[op](s)
    from quantised_gemv_norm_gb300 import dq

    if op == "rope":
        w = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS) if case["norm"] else {}
        return dq.qkv_rope(s["qkv"], s["positions"], s["rope"], case["n_q"], case["n_kv"], dtype=TYPES[case["type"]], **w)
    if op == "prompt":
        return dq.attention_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    if op == "append":
        dq.kv4_append(s["k"], s["v"], s["slots"], s["pool"])
        return dq.kv4_read(s["pool"], s["slots"], dtype=torch.float32)
    if op == "read":
        return dq.kv4_read(s["pool"], s["slots"], dtype=TYPES[case["type"]])
    return dq.attention_decode_kv4(s["q"], s["pool"], s["pages"], s["n_keys"], s["max_keys"])


# ------------------------------------------------------------------ 64 bits


def _exact_rows(pool, slots, page):
    """fp64 keys and values [rows, n_kv, 128], each code and scale looked up at the place the block's definition gives."""
    s = slots.long()
    j = (s % BLOCK_KEYS)[:, None]
    b = pool[s // page, :, s % page // BLOCK_KEYS]  # rows, n_kv, bytes
    r = torch.arange(len(s), device=s.device)[:, None]
    n = torch.arange(HD, device=s.device)
    g, w = n // 32, n % 32
    e = w % 8
    at = 64 * j + 4 * (4 * (w // 8) + g) + 2 * (e % 2) + e // 4
    kc = (b[r, :, at].long() >> (4 * (e // 2 % 2))[None, :, None]) & 15  # rows, dim, n_kv
    at = 1024 + 512 * (j // 8) + 16 * (4 * (w // 4) + j // 2 % 4) + 4 * g + 2 * (j % 2) + w % 4 // 2
    vc = (b[r, :, at].long() >> (4 * (w % 2))[None, :, None]) & 15
    h = b.contiguous().view(torch.float16)
    at = 16 * (j // 2) + 4 * g + j % 2
    return [(h[r, :, base + at].double() * (c - 8) + h[r, :, base + at + 2].double()).transpose(1, 2)
            for c, base in ((kc, 1024), (vc, 1152))]


def _exact_attention(q, k, v, seen):
    """fp64 softmax(q k^T / sqrt(128)) v of one head; rows that see nothing are zero."""
    a = q @ k.T / math.sqrt(HD)
    a[~seen] = -math.inf
    w = torch.exp(a - a.max(1, keepdim=True).values.nan_to_num(neginf=0.0))
    w[~seen] = 0
    t = w.sum(1, keepdim=True)
    return torch.where(t > 0, (w @ v) / t, torch.zeros_like(t))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        x = s["qkv"].double().reshape(case["rows"], -1, HD)
        out = []
        for a, b, w in ((0, case["n_q"], s["q_norm"]), (case["n_q"], case["n_q"] + case["n_kv"], s["k_norm"])):
            h = x[:, a:b]
            if case["norm"]:
                h = h / torch.sqrt(torch.sum(h ** 2, -1, keepdim=True) / HD + EPS) * w.double()
            z = torch.complex(h[..., :HD // 2], h[..., HD // 2:])
            turn = s["rope"][s["positions"].long()].double()
            z = z * torch.complex(turn[..., 0], turn[..., 1])[:, None]
            out.append(torch.cat([z.real, z.imag], -1))
        return out[0], out[1], x[:, case["n_q"] + case["n_kv"]:]
    if op == "prompt":
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        group = case["n_q"] // case["n_kv"]
        for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
            if a == b or c == d:
                continue
            seen = torch.arange(c, d, device="cuda")[None] - c <= torch.arange(a, b, device="cuda")[:, None] - a + (d - c) - (b - a)
            for h in range(case["n_q"]):
                out[a:b, h] = _exact_attention(q[a:b, h], k[c:d, h // group], v[c:d, h // group], seen)
        return out
    if op == "append":
        got = []
        for x in (s["k"], s["v"]):
            g = x.float().cpu().numpy().reshape(case["rows"], case["n_kv"], 4, GROUP)  # the steps are 32-bit ones
            lo, hi = g.min(-1), g.max(-1)
            d = ((hi - lo) / np.float32(15)).astype(np.float16).astype(np.float32)
            z = (lo + np.float32(8) * d).astype(np.float16).astype(np.float32)
            with np.errstate(divide="ignore", invalid="ignore"):
                c = np.where(d[..., None] > 0, np.clip(np.rint((g - z[..., None]) / d[..., None]), -8, 7), 0)
            y = d.astype(np.float64)[..., None] * c + z.astype(np.float64)[..., None]
            got.append(torch.from_numpy(y.reshape(case["rows"], case["n_kv"], HD)))
        return tuple(got)
    if op == "read":
        return tuple(_exact_rows(s["pool"], s["slots"], case["page"]))
    out = torch.zeros(s["q"].shape, dtype=torch.float64)
    group = case["n_q"] // case["n_kv"]
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        slots = s["pages"][b][at // case["page"]].long() * case["page"] + at % case["page"]
        used, where = torch.unique(slots // case["page"], return_inverse=True)
        k, v = _exact_rows(s["pool"][used], where * case["page"] + slots % case["page"], case["page"])
        q = s["q"][b].double()
        seen = torch.ones((group, n), dtype=torch.bool, device="cuda")
        for g in range(case["n_kv"]):
            out[b, g * group:(g + 1) * group] = _exact_attention(q[g * group:(g + 1) * group], k[:, g], v[:, g], seen).cpu()
    return out
