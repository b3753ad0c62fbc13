"""The operators of a speculative decode step as cases: plain torch forms, the library's calls and a 64-bit form.

A step drafts a tree of tokens for each sequence (its root is the last token that was decided), runs the target
model once over all the nodes, and keeps the path of nodes that the target agrees with.  Operators (``op`` of a case):

- ``append``: a layer's projections through head norm and rotary embedding, queries out, keys and values into a paged
  16-bit cache (``dq.kv16_append``);
- ``attend``: a few new tokens of each sequence, a tree or a chain, over that cache (``dq.attention_tree``); one new
  token a sequence is the ordinary decode step;
- ``verify``: the drafted tokens against the target's logits, from given random numbers (``dq.verify_draft``);
- ``keep``: the accepted nodes' cache rows moved to where a sequence goes on, in all layers (``dq.kv16_keep``).

The cache of a layer is [pages][2: keys, values][KV heads][page size][128]; row j of a sequence is in page
pages[s][j // page size] at offset j % page size.  A sequence has n_past rows and its new tokens' after them.
"""
import math
import random

import numpy as np
import torch

own = False

HD = 128
EPS, THETA = 1e-6, 1.0e6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases


def listed():
    q = dict(n_q=32, n_kv=8)  # the decode benchmark's heads
    one = dict(n_seq=1, min_new=1, page=64, shape="chain")
    return [
        # one token's projections as the vocabulary's GEMVs leave them: latency
        dict(name="append 1 row", op="append", rows=1, max_ctx=4096, norm=True, src="f32", type="f16", page=64, **q),
        # a long prompt's projections into the cache: bandwidth
        dict(name="append 8191 rows", op="append", rows=8191, max_ctx=8192, norm=True, src="f32", type="bf16", page=64, **q),
        # one conversation's next token at the benchmark's length: latency
        dict(name="attend 1 x 1 after 512", op="attend", max_new=1, max_past=512, min_past=512, type="f16", mix=1,
             **one, **q),
        # a drafted tree in one very long conversation: the keys split over the whole card
        dict(name="attend 1 x 16 after 100001", op="attend", max_new=16, max_past=100001, min_past=100001, type="f16",
             mix=2, **(one | dict(min_new=16, shape="tree")), **q),
        # a serving batch of ordinary decode steps of very different lengths
        dict(name="attend 64 x 1 ragged", op="attend", n_seq=64, max_new=1, min_new=1, max_past=12000, min_past=0,
             page=32, shape="chain", type="bf16", mix=3, **q),
        # a serving batch with small drafted trees, some with fewer nodes
        dict(name="attend 32 x 8 ragged", op="attend", n_seq=32, max_new=8, min_new=1, max_past=12000, min_past=1,
             page=64, shape="tree", type="f16", mix=4, **q),
        # few sequences with the largest trees: as much arithmetic as memory
        dict(name="attend 8 x 64", op="attend", n_seq=8, max_new=64, min_new=64, max_past=16000, min_past=4000,
             page=64, shape="tree", type="bf16", mix=5, **q),
        # one conversation's draft of five tokens, with the draft model's probabilities: latency
        dict(name="verify 1 x 6 chain", op="verify", n_seq=1, max_new=6, min_new=6, vocab=151936, probs=True, shape="chain",
             type="f32", greedy=0.0, mix=6),
        # a serving batch of such drafts
        dict(name="verify 64 x 9 chain", op="verify", n_seq=64, max_new=9, min_new=1, vocab=151936, probs=True,
             shape="chain", type="f32", greedy=0.1, mix=7),
        # trees of a draft head's best candidates, a vocabulary of odd size, logits of a 16-bit product
        dict(name="verify 16 x 33 tree", op="verify", n_seq=16, max_new=33, min_new=20, vocab=100003, probs=False,
             shape="tree", type="bf16", greedy=0.25, mix=8),
        # one conversation's accepted nodes in the benchmark's 36 layers: latency
        dict(name="keep 1 x 8", op="keep", n_seq=1, max_new=16, past=600, page=64, layers=36, n_kv=8, type="f16", mix=9),
        # a serving batch's
        dict(name="keep 64 ragged", op="keep", n_seq=64, max_new=64, past=300, page=32, layers=36, n_kv=8, type="bf16", mix=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "verify", "keep"])
    n_q, n_kv = rng.choice([(32, 8), (16, 8), (16, 2), (12, 2), (4, 4), (6, 2), (8, 1), (5, 1), (21, 3)])
    kind, page, mix = rng.choice(["f16", "bf16"]), rng.choice([16, 32, 48, 64, 128, 256]), rng.randrange(1 << 20)
    if op == "append":
        rows = _log_int(rng, 1, 8191)
        return dict(op=op, rows=rows, max_ctx=rows + rng.randrange(1, 4096), norm=rng.random() < 0.8,
                    src=rng.choice(["f32", "f16", "bf16"]), type=kind, page=page, n_q=n_q, n_kv=n_kv)
    if op == "attend":
        n_seq, new = _log_int(rng, 1, 64), rng.choice([1, _log_int(rng, 2, 64)])
        past = _log_int(rng, 1, max(2, 500000 // n_seq // n_kv // max(1, new * n_q // n_kv // 64)))
        return dict(op=op, n_seq=n_seq, max_new=new, min_new=rng.choice([0, 1, new]), max_past=past,
                    min_past=rng.choice([0, 1, past]), page=page, shape=rng.choice(["chain", "tree", "tree", "any"]),
                    type=kind, mix=mix, n_q=n_q, n_kv=n_kv)
    if op == "verify":
        n_seq, new, probs = _log_int(rng, 1, 64), _log_int(rng, 1, 64), rng.random() < 0.5
        return dict(op=op, n_seq=n_seq, max_new=new, min_new=rng.choice([0, 1, new]),
                    vocab=_log_int(rng, 200, max(300, min(151936, 64 * 9 * 151936 // (n_seq * new)))), probs=probs,
                    shape="chain" if probs else rng.choice(["chain", "tree"]), type=rng.choice(["f32", "f16", "bf16"]),
                    greedy=rng.choice([0.0, 0.3, 1.0]), mix=mix)
    return dict(op=op, n_seq=_log_int(rng, 1, 64), max_new=_log_int(rng, 1, 64), past=_log_int(rng, 1, 400), page=page,
                layers=_log_int(rng, 1, 36), n_kv=n_kv, type=kind, mix=mix)


def _counts(case):
    """New tokens and past rows of each sequence."""
    r = random.Random(case["mix"])
    new = [r.randint(case["min_new"], case["max_new"]) for _ in range(case["n_seq"])]
    new[0] = case["max_new"]
    lo, hi = case.get("min_past", 0), case.get("max_past", 0)
    past = [r.randint(lo, hi) for _ in range(case["n_seq"])]
    past[-1] = hi
    return new, past


def _parents(case):
    """Each sequence's tree: its nodes' parents, -1 for the root."""
    r = random.Random(case["mix"] + 1)
    wide = r.choice([2, 4, 8])
    return [[i - 1 if i == 0 or case["shape"] == "chain" else r.randrange(max(0, i - wide), i) for i in range(n)]
            for n in _counts(case)[0]]


def _seen(case):
    """Each sequence's rows' visible nodes, as bit masks."""
    r, out = random.Random(case["mix"] + 2), []
    for p in _parents(case):
        rows = []
        for i, a in enumerate(p):
            rows.append((rows[a] if a >= 0 else 0) | 1 << i)
        if case["shape"] == "any":  # some rows see nothing of the new tokens, some others' tokens
            rows = [x if r.random() < 0.5 else r.choice([0, r.getrandbits(len(p))]) for x in rows]
        out.append(rows)
    return out


def _path(case):
    """Each sequence's accepted nodes: the root, then nodes past the kept ones' places (so that a second call moves the
    same rows), ascending."""
    r, out, most = random.Random(case["mix"]), [], max(1, min(12, case["max_new"] // 2))
    for b in range(case["n_seq"]):
        n = r.randint(1, most) if b else most
        out.append([0] + sorted(r.sample(range(n, case["max_new"]), min(n, case["max_new"] - n + 1) - 1)))
    return out


def work(case):
    op = case["op"]
    if op == "append":
        n, heads = case["rows"] * HD, case["n_q"] + 2 * case["n_kv"]
        return {"bytes": n * heads * (BYTES[case["src"]] + 2) + case["rows"] * (8 + 4 * HD),
                "flops": n * (case["n_q"] + case["n_kv"]) * 7}
    if op == "attend":
        new, past = _counts(case)
        pairs = sum(a * b for a, b in zip(new, past)) + sum(x.bit_count() for rows in _seen(case) for x in rows)
        keys = sum(a + b for a, b in zip(new, past) if a)
        return {"bytes": keys * case["n_kv"] * 4 * HD + sum(new) * case["n_q"] * 4 * HD, "flops": pairs * case["n_q"] * 4 * HD}
    if op == "verify":
        new = _counts(case)[0]
        rows, seqs = sum(new), sum(a > 0 for a in new)
        # every row for its sum; for the sampled token one row of random numbers and one of the draft's
        return {"bytes": case["vocab"] * (rows * BYTES[case["type"]] + seqs * 4 * (2 if case["probs"] else 1)),
                "flops": rows * case["vocab"] * 4}
    moved = sum(i != a for p in _path(case) for i, a in enumerate(p))
    return {"bytes": max(1, moved) * case["layers"] * case["n_kv"] * 2 * 2 * 2 * HD, "flops": 0}


# ------------------------------------------------------------------- inputs


def _randn_into(gen, out, wide=None):
    """Normal numbers, some channels of the keys larger, in pieces."""
    flat = out.view(-1, HD)
    for a in range(0, flat.shape[0], 1 << 20):
        x = torch.randn(flat[a:a + (1 << 20)].shape, device="cuda", generator=gen)
        flat[a:a + (1 << 20)] = x if wide is None else x * wide
    return out


def _tables(gen, past, new, page):
    """A scattered page table for sequences of past + new rows, and how many pages there are."""
    need = [-(-(a + b) // page) for a, b in zip(past, new)]
    wide, total = max(1, max(need)), sum(need) + 2
    order = torch.randperm(total, device="cuda", generator=gen).int()
    first = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    at = first[:, None] + torch.arange(wide, device="cuda")
    return order[at.clamp(max=total - 1)].contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    op, s = case["op"], {"case": case}
    if op == "append":
        rows, page = case["rows"], case["page"]
        s["qkv"] = randn(rows, (case["n_q"] + 2 * case["n_kv"]) * HD).to(TYPES[case["src"]])
        s["positions"] = (torch.arange(rows, device="cuda") + seed % (case["max_ctx"] - rows + 1)).int()
        pages, total = _tables(gen, [seed % 7], [rows], page)
        at = torch.arange(rows, device="cuda") + seed % 7
        s["slots"] = (pages[0][at // page] * page + at % page).int()
        s["pool"] = torch.zeros((total, 2, case["n_kv"], page, HD), dtype=TYPES[case["type"]], device="cuda")
        s["q_norm"], s["k_norm"] = 1 + 0.1 * randn(HD), 1 + 0.1 * randn(HD)
        angle = (torch.arange(case["max_ctx"], device="cuda", dtype=torch.float64)[:, None]
                 / THETA ** (torch.arange(HD // 2, device="cuda", dtype=torch.float64) / (HD // 2)))
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    elif op == "attend":
        new, past = _counts(case)
        t = TYPES[case["type"]]
        s["pages"], total = _tables(gen, past, new, case["page"])
        pool = torch.empty((total, 2, case["n_kv"], case["page"], HD), dtype=t, device="cuda")
        wide = 1.0 + 3.0 * (torch.rand(HD, device="cuda", generator=gen) < 0.05).float()
        s["pool"] = _randn_into(gen, pool, wide)
        s["q"] = randn(max(1, sum(new)), case["n_q"], HD).to(t)
        s["n_past"], s["cu_new"] = ints(past), ints(np.cumsum([0] + new).tolist())
        masks = [x - (1 << 64) if x >> 63 else x for rows in _seen(case) for x in rows]
        s["seen"] = None if case["shape"] == "chain" else torch.tensor(masks or [0], dtype=torch.int64, device="cuda")
        s["even"] = min(new) == max(new)
    elif op == "verify":
        new, vocab = _counts(case)[0], case["vocab"]
        rows, first = max(1, sum(new)), np.cumsum([0] + new)
        parents = _parents(case)
        # a model's logits: most of the mass on a few tokens
        z = 2.0 * randn(rows, vocab)
        top = torch.randint(0, vocab, (rows, 24), device="cuda", generator=gen)
        z.scatter_(1, top, 6.0 + 6.0 * torch.rand((rows, 24), device="cuda", generator=gen))
        s["logits"] = z.to(TYPES[case["type"]])
        of = torch.tensor([first[i] + max(0, a) for i, p in enumerate(parents) for a in p] or [0], device="cuda")
        temp = np.array([0.0 if random.Random(case["mix"] + 9 * i).random() < case["greedy"] else 0.6 + 0.1 * (i % 6)
                         for i in range(case["n_seq"])], np.float32)
        s["temperature"] = torch.tensor(temp, device="cuda")
        tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
        if case["probs"]:
            s["draft_probs"] = torch.empty((rows, vocab), device="cuda")
            hot = torch.tensor(np.maximum(np.repeat(temp, new), 0.3).tolist() or [1.0], device="cuda")[:, None]
            for a in range(0, rows, 64):
                at = of[a:a + 64]
                q = torch.softmax((z[at] + 0.5 * randn(len(at), vocab)) / hot[a:a + 64], -1)
                s["draft_probs"][a:a + 64] = q
                tokens[a:a + 64] = torch.multinomial(q, 1, generator=gen)[:, 0]
        else:
            rank = [sum(b == a for b in p[:i]) for p in parents for i, a in enumerate(p)] or [0]
            best = (z + 0.5 * randn(rows, vocab)).topk(1 + max(rank)).indices
            tokens = best[of, torch.tensor(rank, device="cuda")]
        s["tokens"] = tokens.int()
        s["parents"] = None if case["shape"] == "chain" else ints([a for p in parents for a in p] or [-1])
        s["uniform"] = torch.rand(rows, device="cuda", generator=gen)
        s["noise"] = torch.empty((case["n_seq"], vocab), device="cuda").exponential_(generator=gen).clamp_min_(1e-30)
        s["cu_new"] = ints(first.tolist())
    else:
        path, n = _path(case), case["n_seq"]
        past = [random.Random(case["mix"] + i).randint(0, case["past"]) for i in range(n)]
        s["pages"], total = _tables(gen, past, [case["max_new"]] * n, case["page"])
        pool = torch.empty((case["layers"], total, 2, case["n_kv"], case["page"], HD), dtype=TYPES[case["type"]], device="cuda")
        s["pool"] = _randn_into(gen, pool)
        s["n_past"], s["n_path"] = ints(past), ints([len(p) for p in path])
        s["path"] = ints([p + [-1] * (case["max_new"] - len(p)) for p in path])
    return s


# ------------------------------------------------------------- the plain forms


def _plain_append(s):
    case = s["case"]
    n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
    x = s["qkv"].float().reshape(case["rows"], n_q + 2 * n_kv, HD)
    cs = s["rope"][s["positions"].long()][:, None]

    def turned(v, w):
        if case["norm"]:
            v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
        a, b = v[..., :HD // 2], v[..., HD // 2:]
        c, d = cs[..., 0], cs[..., 1]
        return torch.cat([a * c - b * d, b * c + a * d], -1)

    pool, slots = s["pool"], s["slots"].long()
    pool[slots // page, 0, :, slots % page] = turned(x[:, n_q:n_q + n_kv], s["k_norm"]).to(pool.dtype)
    pool[slots // page, 1, :, slots % page] = x[:, n_q + n_kv:].to(pool.dtype)
    return turned(x[:, :n_q], s["q_norm"]).to(pool.dtype), pool


def _plain_attend(s):
    q, pool, cu = s["q"], s["pool"], s["cu_new"].long()
    n_past, page, dev = s["n_past"].long(), pool.shape[3], q.device
    n_q, n_kv = q.shape[1], pool.shape[2]
    new = cu[1:] - cu[:-1]
    i = torch.arange(max(1, s["case"]["max_new"]), device=dev)
    j = torch.arange(s["pages"].shape[1] * page, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    mask = s["seen"][rows] if s["seen"] is not None else ((2 << i) - 1).expand(len(new), -1)
    node = j - n_past[:, None]  # a key's node, below 0 for the past
    bit = (mask[:, :, None] >> node[:, None].clamp(0, 63)) & 1
    live = (i < new[:, None])[:, :, None]
    seen = (live & ((node < 0)[:, None] | ((node < new[:, None])[:, None] & (bit == 1))))[:, None, None]
    kv = pool[s["pages"].long()].float()  # seq, page, 2, kv, row, dim
    k, v = (kv[:, :, a].transpose(1, 2).flatten(2, 3)[:, :, None] for a in (0, 1))
    qp = q[rows].float().transpose(1, 2).unflatten(1, (n_kv, n_q // n_kv))  # seq, kv, group, i, dim
    p = ((qp @ k.transpose(-1, -2)) * (1.0 / math.sqrt(HD))).masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.flatten(1, 2).transpose(1, 2).to(q.dtype)  # seq, i, head, dim
    out = torch.zeros_like(q)
    out[rows[live[:, :, 0]]] = o[live[:, :, 0]]
    return out


def _plain_verify(s):
    case, cu = s["case"], s["cu_new"].long()
    z, dev = s["logits"], s["logits"].device
    n_seq, width, vocab = case["n_seq"], max(1, case["max_new"]), z.shape[1]
    i = torch.arange(width, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=z.shape[0] - 1)
    new = cu[1:] - cu[:-1]
    live = i < new[:, None]
    parent = s["parents"].long()[rows] if s["parents"] is not None else (i - 1).expand(n_seq, -1)
    parent = torch.where(live & (i > 0), parent, torch.full_like(rows, -1))
    token = s["tokens"].long()[rows]
    temp = s["temperature"].double()
    # softmax of every row in 64 bits, a greedy sequence's at temperature 1
    of_row = torch.repeat_interleave(torch.where(temp > 0, temp, torch.ones_like(temp)), new, output_size=int(z.shape[0]))
    w = z.double()
    best = torch.where(w == w.amax(1, keepdim=True), torch.arange(vocab, device=dev), vocab).amin(1)
    w = (w - w.amax(1, keepdim=True)).div_(of_row[:, None]).exp_()
    total = w.sum(1)
    prow = rows.gather(1, parent.clamp_min(0))
    p = w[prow, token] / total[prow]
    earlier = (parent[:, :, None] == parent[:, None]) & (parent >= 0)[:, None] & (i[:, None] < i)  # i before j, siblings
    again = (earlier & (token[:, :, None] == token[:, None])).any(1)
    if case["probs"]:
        u = s["uniform"].double()[rows] * s["draft_probs"][rows, token].double()
        ok = (u < p) & ~again
    else:
        left = 1.0 - (earlier * (p * ~again)[:, :, None]).sum(1)
        ok = (s["uniform"].double()[rows] * left < p) & ~again
    ok = torch.where((temp > 0)[:, None], ok, best[prow] == token) & (parent >= 0)
    chosen = ok & ~(earlier & ok[:, :, None]).any(1)
    tree = torch.eye(width, device=dev) + (parent[:, :, None] == i)  # row j: itself and its parent
    above = torch.linalg.matrix_power(tree.double(), width) > 0
    on = ~(above & (~chosen & (i > 0))[:, None]).any(2) & live
    n_path = on.sum(1)
    path = torch.where(on, i, width).sort(1).values
    last = (n_path > 0) * path.gather(1, (n_path - 1).clamp_min(0)[:, None]).clamp(max=width - 1)[:, 0]
    path = torch.where(path < width, path, -1)
    row = rows.gather(1, last[:, None])[:, 0]
    r = w[row]
    child = parent == last[:, None]  # the ones that were turned down
    if case["probs"]:
        at = torch.where(child, i, 0).amax(1)
        q = s["draft_probs"][rows.gather(1, at[:, None])[:, 0]].double()
        r = torch.where((at > 0)[:, None], (r - total[row][:, None] * q).clamp_min_(0), r)
    else:
        r = torch.cat([r, r[:, :1]], 1).scatter(1, torch.where(child, token, vocab), 0.0)[:, :vocab]
    score = r.div_(s["noise"].double())
    top = torch.where(score == score.amax(1, keepdim=True), torch.arange(vocab, device=dev), vocab).amin(1)
    top = torch.where((temp > 0) & (score.amax(1) > 0), top, best[row])
    return path.int(), n_path.int(), torch.where(new > 0, top, -1).int()


def _plain_keep(s):
    pool, path, page = s["pool"], s["path"].long(), s["pool"].shape[4]
    i = torch.arange(path.shape[1], device=pool.device)
    src, dst = s["n_past"].long()[:, None] + path, s["n_past"].long()[:, None] + i
    go = (i < s["n_path"].long()[:, None]) & (src != dst)
    seq = torch.arange(path.shape[0], device=pool.device)[:, None].expand_as(src)[go]
    src, dst, pages = src[go], dst[go], s["pages"].long()
    pool[:, pages[seq, dst // page], :, :, dst % page] = pool[:, pages[seq, src // page], :, :, src % page]
    return pool


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "verify": _plain_verify, "keep": _plain_keep}[op](s)
    from quantised_gemv_norm_gb300 import dq

    if op == "append":
        w = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS) if case["norm"] else {}
        return dq.kv16_append(s["qkv"], s["positions"], s["slots"], s["rope"], s["pool"], case["n_q"], **w), s["pool"]
    if op == "attend":
        if s["even"] and case["max_new"]:
            return dq.attention_tree(s["q"], s["pool"], s["pages"], s["n_past"], seen=s["seen"])
        return dq.attention_tree(s["q"], s["pool"], s["pages"], s["n_past"], cu_new=s["cu_new"], max_new=case["max_new"],
                                 seen=s["seen"])
    if op == "verify":
        return dq.verify_draft(s["logits"], s["tokens"], s["uniform"], s["noise"], cu_new=s["cu_new"],
                               max_new=case["max_new"], parents=s["parents"], draft_probs=s.get("draft_probs"),
                               temperature=s["temperature"])
    dq.kv16_keep(s["pool"], s["pages"], s["n_past"], s["path"], s["n_path"])
    return s["pool"]


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "append":
        n_q, n_kv, page = case["n_q"], case["n_kv"], case["page"]
        x = s["qkv"].double().reshape(case["rows"], -1, HD)
        out = []
        for a, b, w in ((0, n_q, s["q_norm"]), (n_q, n_q + n_kv, s["k_norm"])):
            h = x[:, a:b]
            if case["norm"]:
                h = h / torch.sqrt(torch.sum(h ** 2, -1, keepdim=True) / HD + EPS) * w.double()
            turn = s["rope"][s["positions"].long()].double()
            h = torch.complex(h[..., :HD // 2], h[..., HD // 2:]) * torch.complex(turn[..., 0], turn[..., 1])[:, None]
            out.append(torch.cat([h.real, h.imag], -1))
        pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
        slot = s["slots"].tolist()
        page_of, at = torch.tensor([a // page for a in slot]), torch.tensor([a % page for a in slot])
        flat = pool.permute(0, 3, 1, 2, 4)
        flat[page_of.cuda(), at.cuda()] = torch.stack([out[1], x[:, n_q + n_kv:]], 1)
        return out[0], pool
    if op == "attend":
        new, past = _counts(case)
        out, first, group = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0, case["n_q"] // case["n_kv"]
        for b, (n, before, rows) in enumerate(zip(new, past, _seen(case))):
            if n == 0:
                continue
            j = torch.arange(before + n, device="cuda")
            pg, off = s["pages"][b][j // case["page"]].long(), j % case["page"]
            seen = torch.ones((n, before + n), dtype=torch.bool)
            seen[:, before:] = torch.tensor([[bool(x >> c & 1) for c in range(n)] for x in rows])
            seen = seen.cuda()
            for g in range(case["n_kv"]):
                k, v = s["pool"][pg, 0, g, off].double(), s["pool"][pg, 1, g, off].double()
                for h in range(g * group, (g + 1) * group):
                    a = s["q"][first:first + n, h].double() @ k.T / math.sqrt(HD)
                    a[~seen] = -math.inf
                    w = torch.exp(a - a.max(1, keepdim=True).values.nan_to_num(neginf=0.0))
                    w[~seen] = 0
                    t = w.sum(1, keepdim=True)
                    out[first:first + n, h] = torch.where(t > 0, (w @ v) / t, torch.zeros_like(t))
            first += n
        return out
    if op == "verify":
        new, first = _counts(case)[0], 0
        paths, lengths, tokens = [], [], []
        u, tok = s["uniform"].tolist(), s["tokens"].tolist()
        for b, (n, parents) in enumerate(zip(new, _parents(case))):
            temp, cur, path, r = float(s["temperature"][b]), 0, [0], None
            for j in range(1, n):
                if parents[j] != cur:
                    continue
                row, x = s["logits"][first + cur].double(), tok[first + j]
                if temp <= 0:
                    ok = int((row == row.max()).nonzero()[0]) == x
                else:
                    r = torch.softmax(row / temp, 0) if r is None else r
                    q = s["draft_probs"][first + j].double() if case["probs"] else None
                    ok = u[first + j] * (float(q[x]) if case["probs"] else 1.0) < float(r[x])
                if ok:
                    cur, r = j, None
                    path.append(j)
                elif temp > 0:
                    if case["probs"]:
                        r = (r - q).clamp_min(0)
                    else:
                        r = r.clone()
                        r[x] = 0
                    r = r / r.sum()
            if n:
                row = s["logits"][first + cur].double()
                if temp <= 0:
                    score = row
                else:
                    score = (torch.softmax(row / temp, 0) if r is None else r) / s["noise"][b].double()
                tokens.append(int((score == score.max()).nonzero()[0]))
            else:
                path = []
                tokens.append(-1)
            paths.append(path + [-1] * (max(1, case["max_new"]) - len(path)))
            lengths.append(len(path))
            first += n
        return tuple(torch.tensor(x, dtype=torch.int32) for x in (paths, lengths, tokens))
    return None  # rows are moved as they are
