"""GPU tests of the prompt and 4-bit cache attention at the ends of their number ranges: probabilities far below the
largest one, scores far from zero, value scales of very different sizes in one cache.

The bounds are those of test_gpu_prompt_kv4.py; what is added to them stands at each test.
"""
import math

import pytest
import torch

from test_gpu_prompt_kv4 import (BAD_ARG, build_cache, decode_ref, decode_slack, dq, gen, HD, i32, prompt_ref,
                                 quantise_ref, randn, starts, U, within)

pytestmark = pytest.mark.gpu
assert dq  # the fixture


def sink_inputs(g, below, n, queries, n_q, n_kv, dtype):
    """q, k, v whose key 0 has a value of zero and 2^below times the usual probability of the n - 1 others."""
    q, k, v = randn(g, queries, n_q, HD), 0.25 * randn(g, n, n_kv, HD), randn(g, n, n_kv, HD)
    q[..., 0] = 16.0
    k[..., 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = below * math.log(2.0) * math.sqrt(HD) / 16.0
    v[0] = 0.0
    return q.to(dtype), k.to(dtype), v.to(dtype)


# One query tile's keys split over blocks (8 heads on 2), or not (80 blocks already).
@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (80, 80)])
@pytest.mark.parametrize("below", [18, 24, 26])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompt_small_probabilities_beside_a_large_one(dq, below, n_q, n_kv, dtype):
    # An fp16 probability is one of steps of 2^-24 below 2^-14, with the largest at 2^7: 2^-26 of it is 32 steps, each
    # key's rounding half a step at most, 2^-32 of the largest.  The keys' probabilities spread over 8 steps and more,
    # so the roundings are independent: six of their standard deviations, 2^-32 / sqrt(3) sqrt(sum v^2), are allowed.
    n, queries = 16001, 3
    q, k, v = sink_inputs(gen(below + n_q), below, n, queries, n_q, n_kv, dtype)
    cu, ck = [0, queries], [0, n]
    y = dq.attention_prompt(q, k, v, i32(cu), i32(ck))
    r, size = prompt_ref(q, k, v, cu, ck)
    spread = (v.double() ** 2).sum(0).sqrt().repeat_interleave(n_q // n_kv, 0)
    slack = (U[dtype] + 4e-5) * size + 6 * 2.0 ** -32 / math.sqrt(3) * spread
    within(y, r, slack)
    # an infinity that a query sees with such a probability is there, whether or not its tile has masked keys
    v[100, 0, 5], v[n - queries, 0, 6] = math.inf, -math.inf
    y = dq.attention_prompt(q, k, v, i32(cu), i32(ck))
    group = n_q // n_kv
    assert bool((y[:, :group, 5] == math.inf).all()) and bool((y[:, :group, 6] == -math.inf).all())
    r[:, :group, 5:7], y[:, :group, 5:7] = 0, 0
    within(y, r, slack)


def one_key_rows(scores, gap):
    """Rows [queries, heads] whose largest score leaves the next one behind by more than ``gap``."""
    top = scores.topk(2, -1).values
    return top[..., 0] - top[..., 1] > gap


@pytest.mark.parametrize("lq,lk", [(200, 200), (5, 3000)])
@pytest.mark.parametrize("dtype,scale", [
    (torch.float16, 300.0), (torch.float16, 4000.0), (torch.float16, 16000.0), (torch.bfloat16, 300.0),
    (torch.bfloat16, 1e6), (torch.bfloat16, 1e8), (torch.bfloat16, 1e17),
])
def test_prompt_scores_far_from_zero(dq, lq, lk, dtype, scale):
    # Scores of +-4 scale^2: one key takes the whole weight wherever the fp32 scores (off by at most 128 2^-24 of
    # sum |q k| / sqrt(128), 5.5e-5 scale^2) tell the two largest apart, and is the output: A's rounded probability alone.
    g = gen(int(math.log2(scale) * 16) + lk)
    q, k = (randn(g, n, h, HD).mul(scale).clamp(-6e4 if dtype == torch.float16 else -1e38, 6e4 if dtype == torch.float16
                                                 else 1e38).to(dtype) for n, h in ((lq, 4), (lk, 2)))
    v = randn(g, lk, 2, HD, dtype=dtype)
    cu, ck = [0, lq], [0, lk]
    y = dq.attention_prompt(q, k, v, i32(cu), i32(ck))
    r, size = prompt_ref(q, k, v, cu, ck)
    s = torch.einsum("ihd,jhd->ihj", q.double(), k.double().repeat_interleave(2, 1)) / math.sqrt(HD)
    seen = torch.arange(lk, device="cuda")[None] <= torch.arange(lq, device="cuda")[:, None] + lk - lq
    clear = one_key_rows(s.masked_fill(~seen[:, None], -math.inf), 1e-3 * scale ** 2)
    assert float(clear.double().mean()) > 0.9
    assert bool(torch.isfinite(y).all())
    within(y[clear], r[clear], U[dtype] * size[clear])


@pytest.mark.parametrize("n_q,lq,lk", [(4, 70, 70), (127, 3, 3), (4, 5, 3000)])
def test_prompt_a_row_far_from_zero_changes_no_other(dq, n_q, lq, lk):
    g = gen(n_q + lk)
    q, k, v = (randn(g, n, h, HD, dtype=torch.float16) for n, h in ((lq, n_q), (lk, 1), (lk, 1)))
    cu, ck = i32([0, lq]), i32([0, lk])
    want = dq.attention_prompt(q, k, v, cu, ck)
    q2 = q.clone()
    q2[1, 2] *= 16000
    y = dq.attention_prompt(q2, k, v, cu, ck)
    assert not torch.equal(y[1, 2], want[1, 2])
    y[1, 2] = want[1, 2]
    assert torch.equal(y, want)
    for _ in range(10):  # whatever an earlier call left in shared memory
        dq.attention_prompt(q2.flip(0).contiguous(), k, v, cu, ck)
        assert torch.equal(dq.attention_prompt(q, k, v, cu, ck), want)


@pytest.mark.parametrize("n", [200, 6000])
@pytest.mark.parametrize("dtype,scale", [
    (torch.float32, 1e5), (torch.float32, 1e9), (torch.float32, 1e20), (torch.float32, 1e37), (torch.float16, 15000.0),
    (torch.bfloat16, 1e9), (torch.bfloat16, 1e20), (torch.bfloat16, 1e37),
])
def test_decode_scores_far_from_zero(dq, n, dtype, scale):
    # Scores of +-4 scale, off by at most 6e-5 scale (two parts: (2^-21 + 128 2^-24) sum |q k| / sqrt(128); 16-bit
    # queries: 2e-5): where the two largest are further apart than that, one key is the output.
    pool, table, ks, vs, zs = build_cache(dq, n, [n], 2, 64)
    q = randn(gen(n + 1), 1, 8, HD).mul(scale).to(dtype)
    if dtype == torch.float16:
        q = q.clamp(-65504, 65504)
    y = dq.attention_decode_kv4(q, pool, table, i32([n]), n)
    r, size = decode_ref(q, ks, vs, [n])
    s = torch.einsum("hd,jhd->hj", q[0].double(), ks[0].repeat_interleave(4, 1)) / math.sqrt(HD)
    clear = one_key_rows(s, 1e-3 * scale)[None]
    assert float(clear.double().mean()) > 0.8
    assert bool(torch.isfinite(y).all())
    slack = decode_slack(q, ks, vs, zs, [n], size)
    within(y[clear], r[clear], slack[clear])


@pytest.mark.parametrize("n", [200, 6000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_large_queries_over_equal_keys(dq, n, dtype):
    # every score is zero, whatever the queries' size
    g = gen(n)
    k, v = torch.zeros(n, 2, HD, device="cuda"), randn(g, n, 2, HD)
    pages = -(-n // 64)
    pool, table = dq.kv4_pool(pages, 2, 64), torch.arange(pages, device="cuda").int()[None]
    slots = torch.arange(n, device="cuda").int()
    dq.kv4_append(k, v, slots, pool)
    kk, vv = (x.double() for x in dq.kv4_read(pool, slots, dtype=torch.float32))
    z = torch.from_numpy(quantise_ref(v.cpu().numpy())[1]).cuda().double().repeat_interleave(32, -1)
    q = randn(g, 1, 8, HD).mul(1e37).to(dtype)
    y = dq.attention_decode_kv4(q, pool, table, i32([n]), n)
    r, size = decode_ref(torch.zeros_like(q), [kk], [vv], [n])
    within(y, r, decode_slack(torch.zeros_like(q), [kk], [vv], [z], [n], size))


def test_calls_repeat_to_the_bit(dq):
    g = gen(91)
    lq = [300, 1, 900, 40]
    q, k, v = (randn(g, sum(lq), h, HD, dtype=torch.bfloat16) for h in (8, 2, 2))
    pool, table, _, _, _ = build_cache(dq, 92, [5000, 3, 800], 2, 64)
    x, n = randn(g, 3, 8, HD, dtype=torch.float16), i32([5000, 3, 800])
    few, fk = randn(g, 6, 8, HD, dtype=torch.float16), randn(g, 9000, 2, HD, dtype=torch.float16)

    def all_three():
        return (dq.attention_prompt(q, k, v, i32(starts(lq))), dq.attention_prompt(few, fk, fk, i32([0, 6]), i32([0, 9000])),
                dq.attention_decode_kv4(x, pool, table, n, 5000))

    want = all_three()
    for _ in range(20):
        for a, b in zip(all_three(), want):
            assert torch.equal(a, b)


# ----------------------------------------------------- value scales of all sizes


def scales_slack(q, keys, values, value_scales, value_z, lengths, dtype):
    """The usual bound with B = sum p (|v - z| + |z|) in place of A, and what fp16's smallest step leaves of a key's
    products: (8 + |z|) max(2^-34, D 2^-36) of the sequence's largest probability, D the KV head's largest scale."""
    parts = [(v - z).abs() + z.abs() for v, z in zip(values, value_z)]
    b = decode_ref(q, keys, parts, lengths)[0]
    slack = 2e-5 * b if dtype == torch.float32 else (6e-5 + 2.0 ** -11) * b
    for i, n in enumerate(lengths):
        group = q.shape[1] // keys[i].shape[1]
        s = torch.einsum("hd,jhd->hj", q[i].double(), keys[i].repeat_interleave(group, 1)) / math.sqrt(HD)
        top = torch.softmax(s, 1).amax(1)[:, None]
        most = value_scales[i].amax((0, 2)).repeat_interleave(group)[:, None]
        step = torch.maximum(torch.full_like(most, 2.0 ** -34), most * 2.0 ** -36)
        slack[i] += step * top * (8 + value_z[i].abs()).sum(0).repeat_interleave(group, 0)
    return slack


def decode_case(dq, k, v, q, copies):
    """One sequence's rows, read by ``copies`` sequences with queries of their own."""
    n, n_kv = k.shape[:2]
    pages = -(-n // 64)
    pool = dq.kv4_pool(pages, n_kv, 64)
    table = torch.arange(pages, device="cuda").int()[None].repeat(copies, 1)
    slots = torch.arange(n, device="cuda").int()
    dq.kv4_append(k, v, slots, pool)
    kk, vv = (x.double() for x in dq.kv4_read(pool, slots, dtype=torch.float32))
    assert bool(torch.isfinite(vv).all())
    d, z = (torch.from_numpy(x).cuda().double() for x in quantise_ref(v.cpu().numpy())[:2])
    y = dq.attention_decode_kv4(q, pool, table, i32([n] * copies), n)
    assert dq.device_error() == 0
    keys, values, lengths = [kk] * copies, [vv] * copies, [n] * copies
    r, _ = decode_ref(q, keys, values, lengths)
    within(y, r, scales_slack(q, keys, values, [d] * copies, [z.repeat_interleave(32, -1)] * copies, lengths, q.dtype))


# 240 keys: one block, whose warps each take cache blocks of the first and of the last keys; 600: splits of 128 keys;
# 20 sequences of 8 KV heads: splits of 512 keys
@pytest.mark.parametrize("n,copies,n_kv", [(240, 1, 2), (600, 1, 2), (1500, 20, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("small", [1.0, 1e-3])
def test_decode_scales_that_grow_along_the_keys(dq, n, copies, n_kv, dtype, small):
    # ordinary values, then scales of 100, then one of 40000 (fp16's last binade), all in one KV head
    g = gen(n + copies)
    k, v = randn(g, n, n_kv, HD), randn(g, n, n_kv, HD) * small
    a, b = 9 * n // 16, 14 * n // 16
    v[a:b, 0, 3], v[a:b, 0, 4] = 750.0, -750.0
    v[b:, 0, 70], v[b:, 0, 90] = 3e5, -3e5
    decode_case(dq, k, v, (0.3 * randn(g, copies, 4 * n_kv, HD)).to(dtype), copies)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_decode_scales_that_fall_along_the_keys(dq, dtype):
    # the largest scale first: the later keys' products stay under its lower cap
    g = gen(7)
    k, v = randn(g, 250, 2, HD), randn(g, 250, 2, HD)
    v[0, :, 3], v[0, :, 4] = 3e5, -3e5
    decode_case(dq, k, v, randn(g, 1, 8, HD).to(dtype), 1)


@pytest.mark.parametrize("n", [250, 6000])
@pytest.mark.parametrize("below", [12, 20])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_decode_small_probabilities_beside_a_large_one(dq, n, below, dtype):
    q, k, v = sink_inputs(gen(below + n), below, n, 1, 8, 2, torch.float32)
    decode_case(dq, k, v, q.to(dtype), 1)


# ------------------------------------------------------------------ large batches


def test_decode_scratch_of_a_large_batch(dq):
    # one result of 132 numbers a query head for every 1024 keys of three blocks an SM, and one more a sequence
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for n_seq, n_q, n_kv, most in ((256, 32, 8, 131072), (1024, 32, 8, 131072), (64, 64, 64, 20000), (300, 8, 1, 1 << 20)):
        need = dq.load().dq_attention_decode_kv4_workspace_bytes(n_seq, n_q, n_kv, most)
        pairs = max(n_seq * n_kv, 3 * sms)
        splits = most / 1024 * 3 * sms / pairs
        assert need <= 528 * (n_q // n_kv) * n_seq * n_kv * (1.1 * splits + 1), (n_seq, n_q, n_kv, most)


@pytest.mark.parametrize("n_q,n_kv,dtype", [(32, 8, torch.float16), (24, 8, torch.float32)])
def test_decode_large_batch(dq, n_q, n_kv, dtype):
    # 1600 pairs of a sequence and a KV head: the splits hold more than 1024 keys
    lengths = [4000, 3333] + [1, 0, 17, 100, 257] * 39 + [2500, 16, 1100]
    pool, table, ks, vs, zs = build_cache(dq, n_q, lengths, n_kv, 64)
    q = randn(gen(n_q), len(lengths), n_q, HD, dtype=dtype)
    r, size = decode_ref(q, ks, vs, lengths)
    slack = decode_slack(q, ks, vs, zs, lengths, size)
    for most in (4000, table.shape[1] * 64):
        within(dq.attention_decode_kv4(q, pool, table, i32(lengths), most), r, slack)
    assert dq.device_error() == 0


# ------------------------------------------------------------------- bad offsets


@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 600, 100, 1000], None),  # rows of two sequences, more block tiles than valid offsets can need
    ([0, 600, 100, 1000], [0, 600, 100, 1000]), ([0, 1000, 0, 1000, 0, 1000, 0], None), ([0, 300, 1001, 1000], None),
    ([-5, 300, 600, 1000], None), ([0, 300, 600, 1000], [0, 300, 1001, 1000]), ([0, 300, 600, 1000], [0, 700, 2, 1000]),
    ([0, 300, 600, 1000], [-2147483648, 2147483647, 0, 1000]),
])
def test_prompt_bad_offsets_touch_nothing_outside(dq, cu_q, cu_k):
    g = gen(17)
    n = 1000
    q, k, v = (randn(g, n, h, HD, dtype=torch.float16) for h in (8, 2, 2))
    wide = torch.full((n + 400, 10, HD), 5.0, dtype=torch.float16, device="cuda")
    dq.attention_prompt(q, k, v, i32(cu_q), None if cu_k is None else i32(cu_k), out=wide[200:-200, 1:9])
    assert dq.device_error() == BAD_ARG
    assert bool((wide[:200] == 5).all()) and bool((wide[-200:] == 5).all())
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 9] == 5).all())
    # the next call is not affected
    y = dq.attention_prompt(q, k, v, i32([0, 300, 600, 1000]))
    r, size = prompt_ref(q, k, v, [0, 300, 600, 1000], [0, 300, 600, 1000])
    within(y, r, (U[q.dtype] + 4e-5) * size)


# ------------------------------------------------ into the decode step's fp16 planes


def test_prompt_into_the_fp16_planes_and_a_token_after_it(dq):
    # a prompt's keys and values copied into a layer's planes: the prompt attention reads them there, and the
    # single-token attention goes on from them (fp64 form: normwise 1e-4, that call's own bound)
    g = gen(19)
    n, n_q, n_kv, ctx = 90, 32, 8, 128
    table = dq.rope_table(ctx)
    wq, wk = 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    norms = dict(q_norm=wq, k_norm=wk)
    x = randn(g, n + 1, (n_q + 2 * n_kv) * HD)
    pos = torch.arange(n + 1, device="cuda").int()
    q, k, v = dq.qkv_rope(x[:n], pos[:n], table, n_q, n_kv, **norms)
    planes = torch.full((2, n_kv, ctx, HD), math.nan, dtype=torch.float16, device="cuda")
    planes[0, :, :n], planes[1, :, :n] = k.transpose(0, 1), v.transpose(0, 1)
    cu = i32([0, n])
    rows = planes.transpose(1, 2)
    assert torch.equal(dq.attention_prompt(q, rows[0][:n], rows[1][:n], cu), dq.attention_prompt(q, k, v, cu))
    new = x[n].reshape(-1, HD)
    planes[1, :, n] = new[n_q + n_kv:].half()
    y = dq.attention_decode_rope(new[:n_q].contiguous(), new[n_q:n_q + n_kv].contiguous(), planes[0], planes[1], wq, wk,
                                 table, n + 1)
    q1, _, _ = dq.qkv_rope(x[n:], pos[n:], table, n_q, n_kv, dtype=torch.float32, **norms)
    r, _ = decode_ref(q1, [rows[0][:n + 1].double()], [rows[1][:n + 1].double()], [n + 1])
    assert float((y.double() - r[0]).norm() / r.norm()) <= 1e-4
    assert dq.device_error() == 0
