"""GPU tests of the speculative decode step's operators (paged 16-bit append, tree attention, verification, kept rows)
against plain 64-bit forms.

Bounds (per element, u = half a step of the output type, finfo.eps / 2):
  append     a head's scale is off by a few 2^-24 (the squares' sum, the reciprocal root), a turned pair (a, b) by three
             roundings: 2e-6 * hypot(a, b) + u |r|
  attention  probabilities are rounded to the type (u), scores are off by at most about 128 roundings of
             sum |q k| / sqrt(128) (4e-5 of a probability at these inputs):  (u + 4e-5) A + u |r|, A = sum p |v|
  verify     whole numbers, equal: the inputs are drawn so that no decision lies within 2^-24 of its border but by a
             chance of about 1e-6 a decision
  keep       bytes, equal
fp16 results below the normal range are off by half of 2^-24 instead of u |r|: 2^-25 is added for them.
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

HD = 128
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -25
BAD_ARG = 8
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantised_gemv_norm_gb300 import build, dq as dqmod

    build.build()
    dqmod.load()
    yield dqmod
    assert dqmod.device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def within(y, r, slack):
    """|y - r| <= slack + u |r| + TINY, for finite r."""
    u = U[y.dtype]
    d = (y.double() - r).abs() - (slack + u * r.abs() + TINY)
    assert bool((d <= 0).all()), "worst excess %g" % float(d.max())


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def as_i64(masks):
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in masks], dtype=torch.int64, device="cuda")


def tables(counts, page, seed=0, spare=2):
    """A scattered page table for sequences of `counts` rows, and the number of pages."""
    need = [-(-n // page) for n in counts]
    total = sum(need) + spare
    order = list(range(total))
    random.Random(seed).shuffle(order)
    wide, at, rows = max(1, max(need)), 0, []
    for n in need:
        rows.append(order[at:at + n] + [-7] * (wide - n))  # what is past a sequence's last page is never looked at
        at += n
    return i32(rows), total


def tree(n, rng, wide=3):
    """Parents and masks of a random tree of n nodes."""
    parents = [-1] + [rng.randrange(max(0, i - wide), i) for i in range(1, n)]
    seen = []
    for i, a in enumerate(parents):
        seen.append((seen[a] if i else 0) | 1 << i)
    return parents[:n], seen[:n]


# ----------------------------------------------------------------- append


def rope_table(dq, max_ctx):
    return dq.rope_table(max_ctx, 128, 1e6)


def turned(x, table, pos, w, eps):
    """Head norm (w not None) and rotation of fp64 heads [rows, heads, 128]."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    cs = table.double()[pos.long()][:, None]
    a, b = x[..., :64], x[..., 64:]
    r = torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1)
    return r, torch.hypot(a, b).repeat(1, 1, 2)


@pytest.mark.parametrize("src,dtype,rows,n_q,n_kv,norm,page", [
    (F32, F16, 1, 32, 8, True, 64), (F32, BF16, 7, 32, 8, True, 16), (BF16, BF16, 130, 6, 2, False, 48),
    (F16, F16, 33, 5, 1, True, 32), (F16, BF16, 9, 21, 3, True, 256), (F32, F16, 1000, 4, 4, False, 64),
    (BF16, F16, 3, 1, 1, True, 16),
])
def test_append(dq, src, dtype, rows, n_q, n_kv, norm, page):
    g = gen(rows + n_q)
    ctx = 2 * rows + 5
    heads = n_q + 2 * n_kv
    qkv = randn(g, rows, heads * HD + 64, dtype=src)[:, :heads * HD]
    if rows == 1:
        qkv = qkv.clone()
    pos = torch.randperm(ctx, device="cuda", generator=g)[:rows].int()
    pages = -(-rows // page) + 3
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:rows].int()
    off = torch.zeros(rows, dtype=torch.bool, device="cuda")
    pad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    if rows > 2:
        off[1::5] = True
        pad[2::7] = True
        slots[off] = -1
        pos[pad] = -3
    table = rope_table(dq, ctx)
    qn, kn = (1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)) if norm else (None, None)
    pool = randn(g, pages, 2, n_kv, page, HD, dtype=dtype)
    before, out = pool.clone(), randn(g, rows, n_q, HD, dtype=dtype)
    out_before = out.clone()
    dq.kv16_append(qkv, pos, slots, table, pool, n_q, q_norm=qn, k_norm=kn, eps=1e-5, out=out)
    x = qkv.double().reshape(rows, heads, HD)
    p = pos.clamp_min(0)
    q, hq = turned(x[:, :n_q], table, p, qn, 1e-5)
    k, hk = turned(x[:, n_q:n_q + n_kv], table, p, kn, 1e-5)
    if norm:  # the bound is relative to the normed pair
        hq = torch.hypot(q[..., :64], q[..., 64:]).repeat(1, 1, 2)
        hk = torch.hypot(k[..., :64], k[..., 64:]).repeat(1, 1, 2)
    live = ~pad
    within(out[live], q[live], 2e-6 * hq[live])
    assert torch.equal(out[pad], out_before[pad])
    kept = live & ~off
    s = slots.long()[kept]
    within(pool[s // page, 0, :, s % page], k[kept], 2e-6 * hk[kept])
    assert torch.equal(pool[s // page, 1, :, s % page], x[kept][:, n_q + n_kv:].to(dtype))
    untouched = torch.ones((pages, page), dtype=torch.bool, device="cuda")
    untouched[s // page, s % page] = False
    assert torch.equal(pool.transpose(2, 3)[untouched[:, None].expand(-1, 2, -1)],
                       before.transpose(2, 3)[untouched[:, None].expand(-1, 2, -1)])


def test_append_reports_what_it_skips(dq):
    g = gen(3)
    table, qkv = rope_table(dq, 8), randn(g, 3, 3 * HD)
    pool = dq.kv16_pool(2, 1, 16)
    out = torch.full((3, 1, HD), 7.0, dtype=F16, device="cuda")
    dq.kv16_append(qkv, i32([8, 1, 2]), i32([0, 32, 3]), table, pool, 1, out=out)
    assert dq.device_error() == BAD_ARG
    assert bool((out[0] == 7).all()) and not bool((out[1] == 7).all())  # a bad position: nothing; a bad slot: the queries
    assert bool((pool[0, :, :, :3] == 0).all()) and not bool((pool[0, :, :, 3] == 0).all())
    assert bool((pool[1] == 0).all()) and bool((pool[0, :, :, 4:] == 0).all())


# -------------------------------------------------------------- attention


def reference(q, pool, pages, past, new, seen, n_rows=None):
    """fp64 outputs and sum p |v| of every row; rows that see nothing are zero."""
    page, n_kv = pool.shape[3], pool.shape[2]
    n_q = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    first = 0
    for s, (a, n) in enumerate(zip(past, new)):
        if n == 0:
            continue
        j = torch.arange(a + n, device="cuda")
        pg = pages[s].long()[j // page]
        there = (pg >= 0) & (pg < pool.shape[0])
        kv = pool[pg.clamp(0, pool.shape[0] - 1), :, :, j % page].double()  # key, 2, kv, dim
        vis = torch.ones((n, a + n), dtype=torch.bool, device="cuda")
        bits = torch.tensor([[bool(m >> t & 1) for t in range(n)] for m in seen[first:first + n]], device="cuda")
        vis[:, a:] = bits
        vis &= there
        for h in range(n_q):
            k, v = kv[:, 0, h // (n_q // n_kv)], kv[:, 1, h // (n_q // n_kv)]
            for i in range(n):
                w = vis[i]
                if not bool(w.any()):
                    continue
                x = (k[w] @ q[first + i, h].double()) / math.sqrt(HD)
                p = torch.softmax(x, 0)
                out[first + i, h] = p @ v[w]
                mag[first + i, h] = p @ v[w].abs()
        first += n
    return out, mag


def chain_masks(new):
    return [(2 << i) - 1 for n in new for i in range(n)]


def masks_of(new, kind, seed):
    rng = random.Random(seed)
    if kind == "chain":
        return chain_masks(new)
    out = []
    for n in new:
        seen = tree(n, rng)[1]
        if kind == "any":
            seen = [rng.choice([m, 0, rng.getrandbits(64)]) for m in seen]
        out += seen
    return out


def visible_only(masks, new):
    """Bits of tokens that a sequence does not have taken out (they mean nothing)."""
    out, at = [], 0
    for n in new:
        out += [m & ((1 << n) - 1) for m in masks[at:at + n]]
        at += n
    return out


CASES = [
    # past, new, n_q, n_kv, page, kind
    ([0], [1], 4, 4, 16, "chain"),
    ([1], [1], 32, 8, 64, "chain"),
    ([513], [1], 32, 8, 64, "chain"),
    ([15, 16, 17], [1, 1, 1], 8, 2, 16, "chain"),
    ([63, 64, 65, 127, 128], [1, 2, 1, 3, 1], 8, 1, 32, "chain"),
    ([0, 5, 300], [7, 0, 3], 6, 2, 48, "tree"),
    ([200, 0, 33], [16, 16, 16], 8, 2, 64, "any"),
    ([100], [64], 4, 1, 64, "tree"),
    ([0, 1000], [64, 5], 8, 2, 128, "any"),
    ([2000], [5], 21, 3, 256, "tree"),
    ([300], [33], 16, 1, 16, "tree"),
    ([77], [64], 64, 1, 32, "tree"),
    ([3, 900], [2, 31], 40, 1, 64, "any"),
    ([4000, 10, 0, 700], [1, 1, 1, 1], 5, 5, 16, "chain"),
    ([12000], [8], 8, 2, 64, "tree"),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s+%s" % (c[0], c[1]))
def test_attention(dq, case, dtype):
    past, new, n_q, n_kv, page, kind = case
    g = gen(sum(past) + n_q)
    pages, total = tables([a + b for a, b in zip(past, new)], page, seed=len(past))
    pool = randn(g, total, 2, n_kv, page, HD, dtype=dtype)
    q = randn(g, sum(new), n_q, HD, dtype=dtype)
    masks = masks_of(new, kind, 5)
    out = dq.attention_tree(q, pool, pages, i32(past), cu_new=i32([sum(new[:i]) for i in range(len(new) + 1)]),
                            max_new=max(new), seen=None if kind == "chain" else as_i64(masks))
    ref, mag = reference(q, pool, pages, past, new, visible_only(masks, new))
    within(out, ref, (U[dtype] + 4e-5) * mag)


@pytest.mark.parametrize("n_seq,max_new,n_q,n_kv,page,longest", [(70, 1, 8, 2, 32, 400), (40, 5, 4, 2, 16, 300),
                                                                 (300, 2, 2, 1, 16, 40), (9, 64, 4, 1, 64, 500),
                                                                 (150, 20, 4, 2, 16, 60), (40, 40, 8, 2, 32, 200)])
def test_attention_of_batches(dq, n_seq, max_new, n_q, n_kv, page, longest):
    rng = random.Random(n_seq)
    new = [rng.randint(0, max_new) for _ in range(n_seq)]
    past = [rng.choice([0, rng.randint(0, longest)]) for _ in range(n_seq)]
    new[3] = max_new
    g = gen(n_seq)
    pages, total = tables([a + b for a, b in zip(past, new)], page, seed=n_seq)
    pool = randn(g, total, 2, n_kv, page, HD, dtype=F16)
    q = randn(g, sum(new), n_q, HD, dtype=F16)
    masks = masks_of(new, "any", 6)
    out = dq.attention_tree(q, pool, pages, i32(past), cu_new=i32([sum(new[:i]) for i in range(n_seq + 1)]), max_new=max_new,
                            seen=as_i64(masks))
    ref, mag = reference(q, pool, pages, past, new, visible_only(masks, new))
    within(out, ref, (U[F16] + 4e-5) * mag)


@pytest.mark.parametrize("new,n_q", [(1, 8), (8, 8), (24, 8), (64, 16)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_what_is_not_seen_does_not_matter(dq, new, n_q, dtype):
    """NaN and infinities in rows past the end, in unseen new tokens, and a page's other rows."""
    g = gen(new)
    past, page, n_kv = 70, 16, 2
    pages, total = tables([past + new], page)
    pool = randn(g, total, 2, n_kv, page, HD, dtype=dtype)
    q = randn(g, new, n_q, HD, dtype=dtype)
    rng = random.Random(1)
    masks = [rng.getrandbits(new) & ~2 for _ in range(new)]  # token 1 is seen by none
    j = torch.arange(past + new, device="cuda")
    live = torch.zeros((total, page), dtype=torch.bool, device="cuda")
    live[pages[0].long()[j // page], j % page] = True
    clean = dq.attention_tree(q, pool, pages, i32([past]), seen=as_i64(masks))
    ref, mag = reference(q, pool, pages, [past], [new], masks)
    within(clean, ref, (U[dtype] + 4e-5) * mag)
    for bad in (float("nan"), float("inf"), -float("inf")):
        dirty = pool.clone()
        dirty.transpose(2, 3)[~live[:, None].expand(-1, 2, -1)] = bad
        if new > 1:
            at = past + 1
            dirty[pages[0, at // page].long(), :, :, at % page] = bad
        out = dq.attention_tree(q, dirty, pages, i32([past]), seen=as_i64(masks))
        assert torch.equal(out, clean)
    if new > 2:  # an infinite value reaches the rows that see it and no other
        dirty = pool.clone()
        at = past + 2
        dirty[pages[0, at // page].long(), 1, :, at % page, 5] = float("inf")
        out = dq.attention_tree(q, dirty, pages, i32([past]), seen=as_i64(masks))
        sees = torch.tensor([bool(m >> 2 & 1) for m in masks], device="cuda")
        assert torch.equal(out[~sees], clean[~sees])
        assert bool((out[sees][..., 5] == float("inf")).all())
        rest = [i for i in range(HD) if i != 5]
        assert torch.equal(out[sees][..., rest], clean[sees][..., rest])


@pytest.mark.parametrize("dtype,size", [(F16, 100.0), (F16, 6.0e4), (BF16, 1.0e4), (BF16, 1.0e15)])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_scores_far_from_zero(dq, dtype, size, new):
    """A large common part of every score, exact in the products, changes no probability."""
    g = gen(11)
    past, page = 150, 32
    pages, total = tables([past + new], page)
    pool = randn(g, total, 2, 1, page, HD, dtype=dtype)
    q = randn(g, new, 4, HD, dtype=dtype)
    q[..., 0] = size
    pool[:, 0, :, :, 0] = size
    masks = masks_of([new], "tree", 2)
    out = dq.attention_tree(q, pool, pages, i32([past]), seen=as_i64(masks))
    assert bool(torch.isfinite(out).all())
    ref, mag = reference(q, pool, pages, [past], [new], masks)
    # the scores' fp32 sums are off by 2^-24 of their size for each of 128 terms at most
    off = 128 * 2.0 ** -24 * size * size / math.sqrt(HD)
    if off < 0.1:
        within(out, ref, (U[dtype] + 4e-5 + 4 * off) * mag)


@pytest.mark.parametrize("new", [[3, 2], [20, 9], [64, 33]])
def test_rows_of_no_sequence_and_strides(dq, new):
    g = gen(21)
    page, n_kv, n_q = 32, 2, 8
    total = sum(new) + 3
    past = [160 - new[0], 7]  # the first sequence fills its pages to the last row
    pages, n_pages = tables([a + b for a, b in zip(past, new)], page)
    assert pages.shape[1] * page == past[0] + new[0]
    pool = randn(g, n_pages, 2, n_kv, page, HD, dtype=BF16)
    wide = randn(g, total, n_q + 4, 2 * HD, dtype=BF16)
    q = wide[:, 2:2 + n_q, :HD]
    out_wide = randn(g, total, n_q, HD + 8, dtype=BF16)
    before = out_wide.clone()
    out = out_wide[..., :HD]
    first, last = 1, 1 + sum(new)
    dq.attention_tree(q, pool, pages, i32(past), cu_new=i32([1, 1 + new[0], last]), max_new=max(new), out=out)
    ref, mag = reference(q[first:last], pool, pages, past, new, chain_masks(new))
    within(out[first:last], ref, (U[BF16] + 4e-5) * mag)
    assert torch.equal(out_wide[0], before[0]) and torch.equal(out_wide[last:], before[last:])
    assert torch.equal(out_wide[..., HD:], before[..., HD:])
    again = q[first:last].contiguous()  # in place
    dq.attention_tree(again, pool, pages, i32(past), cu_new=i32([0, new[0], sum(new)]), max_new=max(new), out=again)
    assert torch.equal(again, out[first:last])


@pytest.mark.parametrize("new", [1, 8, 40])
def test_a_captured_step_after_copies(dq, new):
    """Lengths and queries written by a copy and by a kernel of the same graph directly before the attention, the output
    read by one directly after it."""
    g = gen(23)
    page, n_kv, n_q, n_seq = 32, 2, 8, 3
    pages, total = tables([300] * n_seq, page)
    pool = randn(g, total, 2, n_kv, page, HD, dtype=F16)
    given_q, given_past = randn(g, n_seq * new, n_q, HD, dtype=F16), i32([0, 0, 0])
    q, n_past = torch.empty_like(given_q), i32([0, 0, 0])
    out, twice = torch.empty_like(q), torch.empty_like(q)
    ws = dq.attention_tree_workspace(n_seq, new, n_q, n_kv)

    def step():
        torch.mul(given_q, 1.0, out=q)
        n_past.copy_(given_past)
        dq.attention_tree(q, pool, pages, n_past, workspace=ws, out=out)
        torch.mul(out, 2.0, out=twice)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            step()
    for past in ([5, 200, 0], [250, 1, 64], [0, 0, 259]):
        given_past.copy_(i32(past))
        given_q.copy_(randn(g, *q.shape, dtype=F16))
        graph.replay()
        ref, mag = reference(given_q, pool, pages, past, [new] * n_seq, chain_masks([new] * n_seq))
        within(out, ref, (U[F16] + 4e-5) * mag)
        assert torch.equal(twice, out * 2)


@pytest.mark.parametrize("new", [1, 8, 40])  # the kernels of few rows, of one and of two query tiles
def test_bad_tables_are_reported(dq, new):
    g = gen(31)
    page = 16
    past, rows = 200 - new, 3 * new
    n_pages = 40
    pool = randn(g, n_pages, 2, 1, page, HD, dtype=F16)
    order = torch.randperm(39, device="cuda", generator=g).int()
    good = order.reshape(3, 13)
    bad = good.clone()
    bad[1, 1], bad[1, 9], bad[2, 4] = 99, -2, 2 ** 31 - 1
    pool[39] = float("nan")  # a page of nobody
    q = randn(g, rows, 4, HD, dtype=F16)
    ref, mag = reference(q, pool, bad, [past] * 3, [new] * 3, chain_masks([new] * 3))
    out = dq.attention_tree(q, pool, bad, i32([past] * 3))
    assert dq.device_error() == BAD_ARG
    within(out, ref, (U[F16] + 4e-5) * mag)  # a bad page's keys take no part
    ref, mag = reference(q, pool, good, [past] * 3, [new] * 3, chain_masks([new] * 3))
    for value in (-1, 13 * page - new + 1, 2 ** 31 - 1, -2 ** 31):
        out = dq.attention_tree(q, pool, good, i32([past, value, past]))
        assert dq.device_error() == BAD_ARG
        assert bool((out[new:2 * new] == 0).all())
        others = torch.cat([torch.arange(new), torch.arange(2 * new, rows)]).cuda()
        within(out[others], ref[others], (U[F16] + 4e-5) * mag[others])
    for cu in ([0, 5 * new, 2 * new, rows], [-1, new, 2 * new, rows], [0, new, 2 * new, 2 ** 31 - 1], [2 * new, new, 0, rows]):
        keep = torch.full_like(q, 3.0)
        dq.attention_tree(q, pool, good, i32([past] * 3), cu_new=i32(cu), max_new=new, out=keep)
        assert dq.device_error() == BAD_ARG
        for s in range(3):
            if cu[s] == s * new and cu[s + 1] == cu[s] + new:
                at = slice(cu[s], cu[s + 1])
                within(keep[at], ref[at], (U[F16] + 4e-5) * mag[at])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_with_whole_segments_of_absent_pages(dq, dtype):
    """Sequences all of whose past pages are outside the pool, beside healthy ones."""
    g = gen(33)
    page, new, past = 32, 20, 416
    pool = randn(g, 30, 2, 2, page, HD, dtype=dtype)
    pages = torch.arange(28, device="cuda", dtype=torch.int32).reshape(2, 14)
    pages[1, :13] = 1000
    q = randn(g, 2 * new, 8, HD, dtype=dtype)
    out = dq.attention_tree(q, pool, pages, i32([past, past]))
    assert dq.device_error() == BAD_ARG
    ref, mag = reference(q, pool, pages, [past, past], [new, new], chain_masks([new, new]))
    within(out, ref, (U[dtype] + 4e-5) * mag)


def test_a_pool_past_32_bit_offsets(dq):
    """Pages whose rows lie beyond 2^32 bytes from the pool's start."""
    g = gen(41)
    page, n_kv = 64, 8
    n_pages = 36000  # 9.4 GB
    pool = torch.zeros((n_pages, 2, n_kv, page, HD), dtype=BF16, device="cuda")
    past, new = [200, 130], [4, 4]
    used = [n_pages - 1, 3, n_pages - 5, 17000], [n_pages - 2, n_pages - 3, 16390]
    for pg in used[0] + used[1]:
        pool[pg] = randn(g, 2, n_kv, page, HD, dtype=BF16)
    pages = i32([used[0], used[1] + [-1]])
    q = randn(g, 8, 16, HD, dtype=BF16)
    out = dq.attention_tree(q, pool, pages, i32(past))
    ref, mag = reference(q, pool, pages, past, new, chain_masks(new))
    within(out, ref, (U[BF16] + 4e-5) * mag)
    # and a store and a move there
    table = rope_table(dq, 512)
    qkv = randn(g, 2, 32 * HD)
    slots = i32([(n_pages - 1) * page + 63, (n_pages - 5) * page + 1])
    dq.kv16_append(qkv, i32([5, 6]), slots, table, pool, 16)
    x = qkv.reshape(2, 32, HD)[:, 24:].to(BF16)
    assert torch.equal(pool[n_pages - 1, 1, :, 63], x[0]) and torch.equal(pool[n_pages - 5, 1, :, 1], x[1])
    was = pool[n_pages - 5, :, :, 1].clone()  # row 129 of sequence 0
    dq.kv16_keep(pool, pages[:1], i32([126]), i32([[0, 3, -1, -1]]), i32([2]))
    assert torch.equal(pool[3, :, :, 63], was)


def test_attention_replayed_with_other_lengths(dq):
    """One captured call, replayed after lengths, masks and pages have changed; another graph on the same workspace."""
    g = gen(51)
    page, n_kv, n_q, n_seq, new = 32, 2, 8, 5, 6
    room = 400
    pages, total = tables([room] * n_seq, page)
    pool = randn(g, total, 2, n_kv, page, HD, dtype=F16)
    q = randn(g, n_seq * new, n_q, HD, dtype=F16)
    n_past, seen = i32([0] * n_seq), as_i64([1] * (n_seq * new))
    ws = dq.attention_tree_workspace(n_seq, new, n_q, n_kv)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dq.attention_tree(q, pool, pages, n_past, seen=seen, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.empty_like(q)
    with torch.cuda.graph(graph):
        dq.attention_tree(q, pool, pages, n_past, seen=seen, workspace=ws, out=out)
    with torch.cuda.graph(other):
        dq.attention_tree(q, pool, pages, n_past, workspace=ws, out=out2)
    rng = random.Random(4)
    for step in range(3):
        past = [rng.choice([0, 1, rng.randint(2, room - new)]) for _ in range(n_seq)]
        masks = masks_of([new] * n_seq, "any", step)
        n_past.copy_(i32(past))
        seen.copy_(as_i64(masks))
        q.copy_(randn(g, *q.shape, dtype=F16))
        graph.replay()
        other.replay()
        ref, mag = reference(q, pool, pages, past, [new] * n_seq, visible_only(masks, [new] * n_seq))
        within(out, ref, (U[F16] + 4e-5) * mag)
        ref, mag = reference(q, pool, pages, past, [new] * n_seq, chain_masks([new] * n_seq))
        within(out2, ref, (U[F16] + 4e-5) * mag)


def test_calls_on_two_streams(dq):
    g = gen(61)
    page, n_kv, n_q = 64, 8, 32
    pages, total = tables([3000, 2000], page)
    pool = randn(g, total, 2, n_kv, page, HD, dtype=BF16)
    qs = [randn(g, 2 * t, n_q, HD, dtype=BF16) for t in (1, 4, 16)]
    want = [dq.attention_tree(q, pool, pages, i32([2900, 1900])) for q in qs]
    torch.cuda.synchronize()
    streams, past = [torch.cuda.Stream() for _ in qs], i32([2900, 1900])
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(dq.attention_tree(q, pool, pages, past))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_workspace_content_does_not_matter(dq):
    g = gen(71)
    pages, total = tables([5000], 64)
    pool = randn(g, total, 2, 8, 64, HD, dtype=F16)
    for t in (1, 4, 16, 64):
        q = randn(g, t, 32, HD, dtype=F16)
        ws = dq.attention_tree_workspace(1, t, 32, 8)
        want = dq.attention_tree(q, pool, pages, i32([4900]), workspace=ws.zero_())
        for fill in (255, 127):
            assert torch.equal(dq.attention_tree(q, pool, pages, i32([4900]), workspace=ws.fill_(fill)), want)
        with pytest.raises(dq.DQError):
            dq.attention_tree(q, pool, pages, i32([4900]), workspace=ws[:ws.numel() - 16])


# ----------------------------------------------------------------- verify


def verify_reference(logits, tokens, uniform, noise, new, parents=None, draft=None, temperature=None):
    """The rules of include/dq.h, one sequence and child after another, in 64 bits."""
    paths, out, first = [], [], 0
    u, tok = uniform.tolist(), tokens.tolist()
    vocab = logits.shape[1]
    for s, n in enumerate(new):
        temp = 1.0 if temperature is None else float(temperature[s])
        if temp > 0:
            temp = min(max(temp, 2.0 ** -60), 2.0 ** 60)
        cur, path, gone, down = 0, [0][:n], [], 0

        def weights(node):
            x = logits[first + node].double()
            x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
            m = x.max()
            if m == -math.inf:
                return None, -1
            w = torch.where(x == m, torch.ones_like(x), torch.exp((x - m) / (temp if temp > 0 else 1.0)))
            return torch.where(x == -math.inf, torch.zeros_like(w), w), int((x == m).nonzero()[0])

        for j in range(1, n):
            parent = j - 1 if parents is None else parents[first + j]
            if parent != cur:
                continue
            w, best = weights(cur)
            x = tok[first + j]
            if w is None or not 0 <= x < vocab:
                take = False
            elif not temp > 0:
                take = x == best
            else:
                p = w / w.sum()
                if draft is not None:
                    take = u[first + j] * float(draft[first + j, x]) < float(p[x])
                    down = 0 if take else j
                else:
                    left = 1.0 - sum(float(p[k]) for k in gone)
                    take = x not in gone and u[first + j] * left < float(p[x])
                    if not take and x not in gone:
                        gone.append(x)
            if draft is not None and temp > 0:
                down = 0 if take else j
            if take:
                cur, gone = j, []
                path.append(j)
        if n:
            w, best = weights(cur)
            if w is None or not temp > 0:
                out.append(best)
            else:
                r = (w - w.sum() * draft[first + down].double()).clamp_min(0) if down else w.clone()
                r[gone] = 0
                score = r / noise[s].double()
                out.append(int((score == score.max()).nonzero()[0]) if float(score.max()) > 0 else best)
        else:
            out.append(-1)
        paths.append(path)
        first += n
    return paths, out


def check_verify(dq, logits, tokens, uniform, noise, new, parents=None, draft=None, temperature=None, max_new=None):
    max_new = max_new or max(new)
    path, n_path, after = dq.verify_draft(
        logits, tokens, uniform, noise, cu_new=i32([sum(new[:i]) for i in range(len(new) + 1)]), max_new=max_new,
        parents=None if parents is None else i32(parents), draft_probs=draft, temperature=temperature)
    paths, want = verify_reference(logits, tokens, uniform, noise, new, parents, draft, temperature)
    assert n_path.tolist() == [len(p) for p in paths]
    assert path.tolist() == [p + [-1] * (max_new - len(p)) for p in paths]
    assert after.tolist() == want
    return paths


def peaked(g, rows, vocab, dtype=F32):
    z = 2.0 * randn(g, rows, vocab)
    top = torch.randint(0, vocab, (rows, min(vocab, 12)), device="cuda", generator=g)
    z.scatter_(1, top, 6.0 + 6.0 * torch.rand(top.shape, device="cuda", generator=g))
    return z.to(dtype)


def exponential(g, *shape):
    return torch.empty(shape, device="cuda").exponential_(generator=g).clamp_min_(1e-30)


@pytest.mark.parametrize("new,vocab,dtype,probs", [
    ([1], 5, F32, False), ([2, 1, 0, 5], 1000, F32, True), ([6] * 20, 4099, F32, True), ([9, 3, 1] * 8, 33333, F16, True),
    ([7] * 12, 151936, F32, True), ([64, 1], 8193, BF16, True), ([5] * 30, 1, F32, False), ([4] * 9, 8192, BF16, False),
    ([64, 30], 24577, F16, False),
])
@pytest.mark.parametrize("temp", [None, 0.7, 0.0])
def test_verify_chains(dq, new, vocab, dtype, probs, temp):
    g = gen(sum(new) + vocab)
    rows = sum(new)
    logits = peaked(g, rows, vocab, dtype)
    q = torch.softmax(torch.cat([logits[:1], logits[:-1]]).float() + 0.4 * randn(g, rows, vocab), -1)
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].int()
    uniform, noise = torch.rand(rows, device="cuda", generator=g), exponential(g, len(new), vocab)
    temperature = None if temp is None else torch.full((len(new),), temp, device="cuda")
    check_verify(dq, logits, tokens, uniform, noise, new, draft=q if probs else None, temperature=temperature)


@pytest.mark.parametrize("new,vocab,dtype", [([33, 20, 1, 0, 64], 50021, F32), ([16] * 10, 1003, BF16), ([40] * 3, 16384, F16)])
def test_verify_trees(dq, new, vocab, dtype):
    g, rng = gen(vocab), random.Random(vocab)
    rows = sum(new)
    logits = peaked(g, rows, vocab, dtype)
    parents, first = [], 0
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    for n in new:
        p = tree(n, rng, wide=4)[0]
        best = (logits[first:first + n].float() + 0.3 * randn(g, n, vocab)).topk(5).indices if n else None
        for i in range(1, n):
            tokens[first + i] = best[p[i], sum(a == p[i] for a in p[:i]) % 5]  # a sixth child repeats the first
        parents += p
        first += n
    uniform, noise = torch.rand(rows, device="cuda", generator=g), exponential(g, len(new), vocab)
    temperature = torch.tensor([0.0 if i % 3 == 1 else 0.5 + 0.2 * i for i in range(len(new))], device="cuda")
    paths = check_verify(dq, logits, tokens, uniform, noise, new, parents=parents, temperature=temperature, max_new=64)
    assert max(len(p) for p in paths) > 1


def test_verify_repeated_and_missing_tokens(dq):
    """Children with the same token, tokens outside the vocabulary, a root alone, all candidates rejected."""
    g, vocab = gen(5), 300
    logits = peaked(g, 6, vocab)
    parents = [-1, 0, 0, 0, 0, 4]
    top = int(logits[0].argmax())
    noise, uniform = exponential(g, 1, vocab), torch.full((6,), 0.999999, device="cuda")
    for tokens in ([0, 7, 7, 7, 9, 1], [0, -1, vocab, 7, -5, 3], [0, top, top, 2 ** 31 - 1, top, 1]):
        check_verify(dq, logits, i32(tokens), uniform, noise, [6], parents=parents)
        check_verify(dq, logits, i32(tokens), uniform * 0, noise, [6], parents=parents)


def test_verify_logits_at_the_ends(dq):
    """Infinities, NaN, rows without any finite logit, equal logits."""
    g, vocab = gen(6), 9000
    inf, nan = float("inf"), float("nan")
    rows = peaked(g, 8, vocab)
    rows[0, 5:] = -inf
    rows[1] = -inf
    rows[2] = nan
    rows[3, ::7] = nan
    rows[4, [11, 8500]] = inf
    rows[5] = 3.0
    rows[6] = -inf
    rows[6, 8999] = -5.0
    rows[7, 17] = 3.0e38
    noise = exponential(g, 8, vocab)
    for temp in (None, torch.full((8,), 0.3, device="cuda"), torch.zeros(8, device="cuda"),
                 torch.tensor([1e-30, 1e30, inf, nan, -1.0, 1e-42, 1.0, 2.0], device="cuda")):
        check_verify(dq, rows, i32([0] * 8), torch.zeros(8, device="cuda"), noise, [1] * 8, temperature=temp)
        draft = torch.softmax(peaked(g, 8, vocab), -1)
        tokens = torch.multinomial(draft, 1, generator=g)[:, 0].int()
        uniform = torch.rand(8, device="cuda", generator=g)
        check_verify(dq, rows, tokens, uniform, noise[:4], [2] * 4, draft=draft, temperature=None if temp is None else temp[:4])
        check_verify(dq, rows, tokens, uniform, noise[:1], [8], parents=[-1, 0, 0, 1, 1, 2, 2, 3],
                     temperature=None if temp is None else temp[:1])


def test_verify_reports_bad_trees(dq):
    g, vocab = gen(7), 500
    logits, noise, uniform = peaked(g, 4, vocab), exponential(g, 2, vocab), torch.zeros(4, device="cuda")
    tokens = logits.argmax(1).int()
    for parents in ([-1, 1, 0, 2], [-1, 0, 5, -2]):
        path, n_path, after = dq.verify_draft(logits, tokens, uniform, noise[:1], parents=i32(parents))
        assert dq.device_error() == BAD_ARG
        paths, want = verify_reference(logits, tokens, uniform, noise[:1], [4],
                                       [a if 0 <= a < i else -9 for i, a in enumerate(parents)])
        assert path[0, :len(paths[0])].tolist() == paths[0] and after.tolist() == want
    for cu in ([0, 3, 2], [0, 5, 6], [-2, 2, 4], [0, 4, 4 + 2 ** 30]):
        path, n_path, after = dq.verify_draft(logits, tokens, uniform, noise, cu_new=i32(cu), max_new=4)
        assert dq.device_error() == BAD_ARG
        for s in range(2):
            ok = 0 <= cu[s] <= cu[s + 1] <= 4
            assert (n_path[s].item() > 0) == (ok and cu[s] < cu[s + 1])
            if not ok:
                assert path[s].tolist() == [-1] * 4 and after[s].item() == -1


def test_verify_leaves_rows_of_no_sequence(dq):
    """Logits before the first and after the last sequence have no part in anything, NaN or not."""
    g, vocab = gen(10), 4100
    logits = peaked(g, 9, vocab)
    logits[0], logits[7:] = float("nan"), float("inf")
    tokens, uniform, noise = logits.argmax(1).int(), torch.rand(9, device="cuda", generator=g), exponential(g, 2, vocab)
    path, n_path, after = dq.verify_draft(logits, tokens, uniform, noise, cu_new=i32([1, 5, 7]), max_new=6)
    paths, want = verify_reference(logits[1:7], tokens[1:7], uniform[1:7], noise, [4, 2])
    assert after.tolist() == want and n_path.tolist() == [len(p) for p in paths]
    assert path.tolist() == [p + [-1] * (6 - len(p)) for p in paths]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_verify_strides_and_streams(dq, dtype):
    g, vocab = gen(8), 10007
    wide = peaked(g, 12, vocab + 9, dtype)
    logits = wide[:, 3:3 + vocab]  # rows of any alignment
    q = torch.softmax(randn(g, 12, vocab + 1), -1)[:, :vocab]
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].int()
    uniform, noise = torch.rand(12, device="cuda", generator=g), exponential(g, 3, vocab + 5)[:, :vocab]
    check_verify(dq, logits, tokens, uniform, noise, [4] * 3, draft=q)
    want = dq.verify_draft(logits, tokens, uniform, noise, draft_probs=q)
    ws = dq.verify_draft_workspace(12, vocab).fill_(255)
    side, out = torch.cuda.Stream(), [torch.empty_like(x) for x in want]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dq.verify_draft(logits, tokens, uniform, noise, draft_probs=q, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dq.verify_draft(logits, tokens, uniform, noise, draft_probs=q, workspace=ws, out=out)
    for _ in range(2):
        uniform.copy_(torch.rand(12, device="cuda", generator=g))
        graph.replay()
        for a, b in zip(out, dq.verify_draft(logits, tokens, uniform, noise, draft_probs=q)):
            assert torch.equal(a, b)


def test_verified_tokens_are_distributed_as_drawn(dq):
    """20000 sequences of one drafted token each: the token that follows the root has the target's distribution whether
    the draft was accepted or not (each count within five deviations)."""
    g, vocab, n = gen(9), 8, 20000
    row, draft = randn(g, 2, vocab), torch.softmax(1.5 * randn(g, 1, vocab), -1)
    p = torch.softmax(row[0].double(), -1)
    logits = row.repeat(n, 1)
    for probs in (draft.repeat(2 * n, 1), None):
        tokens = torch.multinomial(draft[0], 2 * n, replacement=True, generator=g).int()
        uniform, noise = torch.rand(2 * n, device="cuda", generator=g), exponential(g, n, vocab)
        path, n_path, after = dq.verify_draft(logits, tokens, uniform, noise, draft_probs=probs)
        first = torch.where(n_path == 2, tokens[1::2], after).long()
        count = torch.bincount(first, minlength=vocab).double()
        assert bool(((count - n * p).abs() <= 5 * torch.sqrt(n * p * (1 - p)) + 1).all())


# ------------------------------------------------------------------- keep


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layers,page,n_kv", [(None, 16, 1), (1, 64, 2), (5, 32, 8)])
def test_keep(dq, layers, page, n_kv, dtype):
    g, rng = gen(page), random.Random(page)
    past = [0, 15, 100, 31, 7]
    paths = [[0], [0, 2, 3, 7, 20], [0, 1, 2, 3], [], [0, 1, 3, 4, 5, 9, 10, 11, 12, 40, 41, 63]]
    pages, total = tables([a + 64 for a in past], page, seed=3)
    pool = randn(g, *([layers] if layers else []), total, 2, n_kv, page, HD, dtype=dtype)
    want, src = pool.clone().unflatten(0, (1, -1)) if not layers else pool.clone(), pool.clone()
    src = src if layers else src.unflatten(0, (1, -1))
    for s, p in enumerate(paths):
        for i, node in enumerate(p):
            a, b = past[s] + node, past[s] + i
            want[:, pages[s, b // page].long(), :, :, b % page] = src[:, pages[s, a // page].long(), :, :, a % page]
    path = i32([p + [rng.choice([-1, 1000]) for _ in range(64 - len(p))] for p in paths])
    dq.kv16_keep(pool, pages, i32(past), path, i32([len(p) for p in paths]))
    assert torch.equal(pool if layers else pool.unflatten(0, (1, -1)), want)


def test_keep_reports_what_it_skips(dq):
    g, page = gen(2), 16
    pages = i32([[0, 1], [2, 9], [3, 4], [5, 6], [7, 7]])
    pool = randn(g, 8, 2, 1, page, HD, dtype=F16)
    before = pool.clone()
    # a node past the tree; a row in a bad page; more rows than pages; a bad count; a bad length
    path = i32([[0, 4, 2], [0, 3, 0], [0, 2, 0], [0, 1, 2], [0, 2, 2]])
    n_path, past = i32([3, 2, 2, 4, 2]), i32([0, 13, 30, 0, -1])
    dq.kv16_keep(pool, pages, past, path, n_path)
    assert dq.device_error() == BAD_ARG
    assert torch.equal(pool, before)


# ---------------------------------------------------------- all together


def test_a_step_as_it_is_used(dq):
    """Two layers: a prompt stored, then steps of a drafted tree (append, attention, verification, kept rows); after each
    step the cache is what storing the accepted tokens one after the other would have left, and one token's attention over
    it agrees with 64 bits."""
    g, rng = gen(100), random.Random(100)
    n_q, n_kv, page, layers, vocab, n_seq, nodes = 8, 2, 32, 2, 5000, 3, 12
    heads, ctx = n_q + 2 * n_kv, 400
    table, qn, kn = rope_table(dq, ctx), 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    embed = [randn(g, vocab, heads * HD) for _ in range(layers)]  # a token's projections in each layer
    prompt = [rng.randint(5, 90) for _ in range(n_seq)]
    pages, total = tables([300] * n_seq, page)
    pool = dq.kv16_pool(total, n_kv, page, dtype=BF16, n_layers=layers)
    text = [[rng.randrange(vocab) for _ in range(n)] for n in prompt]

    def slots_of(s, rows):
        t = pages[s].tolist()
        return [t[j // page] * page + j % page for j in rows]

    for l in range(layers):
        toks = torch.tensor(sum(text, []), device="cuda")
        pos = sum([list(range(n)) for n in prompt], [])
        slots = sum([slots_of(s, range(n)) for s, n in enumerate(prompt)], [])
        dq.kv16_append(embed[l][toks], i32(pos), i32(slots), table, pool[l], n_q, q_norm=qn, k_norm=kn)
    n_past, root = i32(prompt), [rng.randrange(vocab) for _ in range(n_seq)]
    for step in range(4):
        past = n_past.tolist()
        trees = [tree(nodes, rng) for _ in range(n_seq)]
        drafted = [[root[s]] + [rng.randrange(vocab) for _ in range(nodes - 1)] for s in range(n_seq)]
        depth = []
        for p, _ in trees:
            d = [0] * nodes
            for i in range(1, nodes):
                d[i] = d[p[i]] + 1
            depth.append(d)
        toks = torch.tensor(sum(drafted, []), device="cuda")
        pos = i32(sum([[past[s] + d for d in depth[s]] for s in range(n_seq)], []))
        slots = i32(sum([slots_of(s, range(past[s], past[s] + nodes)) for s in range(n_seq)], []))
        seen = as_i64(sum([t[1] for t in trees], []))
        for l in range(layers):
            q = dq.kv16_append(embed[l][toks], pos, slots, table, pool[l], n_q, q_norm=qn, k_norm=kn)
            out = dq.attention_tree(q, pool[l], pages, n_past, seen=seen)
            ref, mag = reference(q, pool[l], pages, past, [nodes] * n_seq, sum([t[1] for t in trees], []))
            within(out, ref, (U[BF16] + 4e-5) * mag)
        logits = randn(g, n_seq * nodes, vocab)
        for s in range(n_seq):  # the target likes one of each node's children, where it has any
            for i in range(nodes):
                kids = [j for j in range(1, nodes) if trees[s][0][j] == i]
                if kids and rng.random() < 0.8:
                    logits[s * nodes + i, drafted[s][rng.choice(kids)]] = 20.0
        path, n_path, after = dq.verify_draft(logits, toks.int(), torch.rand(n_seq * nodes, device="cuda", generator=g),
                                              exponential(g, n_seq, vocab), parents=i32(sum([t[0] for t in trees], [])))
        dq.kv16_keep(pool, pages, n_past, path, n_path)
        n_past += n_path
        for s in range(n_seq):
            text[s] += [drafted[s][i] for i in path[s].tolist()[:n_path[s].item()]]
        root = after.tolist()
        lengths = n_past.tolist()
        assert [len(t) for t in text] == lengths and max(n_path.tolist()) > 1
        for l in range(layers):
            plain = dq.kv16_pool(total, n_kv, page, dtype=BF16)
            all_toks = torch.tensor(sum(text, []), device="cuda")
            all_slots = sum([slots_of(s, range(n)) for s, n in enumerate(lengths)], [])
            dq.kv16_append(embed[l][all_toks], i32(sum([list(range(n)) for n in lengths], [])), i32(all_slots), table, plain,
                           n_q, q_norm=qn, k_norm=kn)
            at = torch.tensor(all_slots, device="cuda")
            assert torch.equal(pool[l][at // page, :, :, at % page], plain[at // page, :, :, at % page])
            one = randn(g, n_seq, n_q, HD, dtype=BF16)
            got = dq.attention_tree(one, pool[l], pages, n_past - 1)
            ref, mag = reference(one, pool[l], pages, [n - 1 for n in lengths], [1] * n_seq, [1] * n_seq)
            within(got, ref, (U[BF16] + 4e-5) * mag)
