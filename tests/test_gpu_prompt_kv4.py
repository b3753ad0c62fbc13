"""GPU tests of the prompt, packed-row and 4-bit cache operators against plain 64-bit forms.

Bounds (per element, u = half a step of the output type: 2^-25 in fp32 terms of finfo.eps / 2):
  rope       a head's scale is off by a few 2^-24 (the squares' sum, the reciprocal root), a turned pair (a, b) by
             three roundings: 2e-6 * hypot(a, b), + u |r|
  prompt     probabilities are rounded to the type (u), scores are off by at most about 128 roundings of
             sum |q k| / sqrt(128) (4e-5 of a probability at these inputs):  (u + 4e-5) A + u |r|, A = sum p |v|
  read       one rounding of the exact d (c - 8) + z: u |r|
  decode     fp32: two-part operands (2^-22 of sum |q k|) and fp32 sums: 2e-5 A + u |r|.  16-bit: the probabilities are
             one fp16 number each in the products p d (c - 8) and p z, half a step 2^-11 either: 2^-11 B more, with
             B = sum p (|v - z| + |z|); scores from uncentred codes, fp32 sums of up to 15 d sum |q| / sqrt(128) per group
             (d about 0.3: 41 at these inputs), four roundings of 2^-23 each: 2e-5, twice that of a probability: 6e-5 A
fp16 results below the normal range are off by half of 2^-24 instead of u |r|: 2^-25 is added for them.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HD = 128
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -25
BAD_ARG = 8


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


# ------------------------------------------------------------------- rope


def rope_ref(x, pos, w, table, eps):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    cs = table[pos.long()].double()[:, None]
    a, b, c, s = x[..., :64], x[..., 64:], cs[..., 0], cs[..., 1]
    size = torch.hypot(a, b)
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)


@pytest.mark.parametrize("rows,n_q,n_kv,dtype,norm", [
    (1, 32, 8, torch.float32, True), (7, 5, 1, torch.float16, True), (65, 3, 3, torch.bfloat16, True),
    (33, 12, 2, torch.float16, False), (700, 21, 3, torch.float32, False), (2050, 32, 8, torch.float16, True),
    (2, 1, 1, torch.bfloat16, True),
])
def test_qkv_rope(dq, rows, n_q, n_kv, dtype, norm):
    g = gen(rows)
    heads = n_q + 2 * n_kv
    wide = randn(g, rows, heads * HD + 12) * 3  # a row stride wider than the heads
    pos = torch.randint(0, 5000, (rows,), device="cuda", generator=g).int()
    pos[0] = 4999
    table = dq.rope_table(5000)
    wq, wk = (1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)) if norm else (None, None)
    q, k, v = dq.qkv_rope(wide, pos, table, n_q, n_kv, q_norm=wq, k_norm=wk, dtype=dtype)
    x = wide[:, :heads * HD].reshape(rows, heads, HD)
    for y, lo, hi, w in ((q, 0, n_q, wq), (k, n_q, n_q + n_kv, wk)):
        r, size = rope_ref(x[:, lo:hi], pos, w, table, 1e-6)
        within(y, r, 2e-6 * size)
    assert torch.equal(v, x[:, n_q + n_kv:].to(dtype))


def test_qkv_rope_leaves_padding_rows_and_reports_far_positions(dq):
    g = gen(3)
    x = randn(g, 6, 4 * HD)
    table = dq.rope_table(16)
    out = tuple(torch.full((6, n, HD), 7.0, device="cuda") for n in (2, 1, 1))
    pos = i32([3, -1, 15, -2147483648, 0, -5])
    dq.qkv_rope(x, pos, table, 2, 1, dtype=torch.float32, out=out)
    assert dq.device_error() == 0
    for o in out:
        assert bool((o[[1, 3, 5]] == 7).all()) and not bool((o[[0, 2, 4]] == 7).any())
    before = [o.clone() for o in out]
    dq.qkv_rope(x, i32([16, -1, -1, 2147483647, -1, -1]), table, 2, 1, dtype=torch.float32, out=out)
    assert dq.device_error() == BAD_ARG
    for o, b in zip(out, before):
        assert torch.equal(o, b)


def test_qkv_rope_matches_the_single_token_attention_inputs(dq):
    # attention_decode_rope writes the same key row; the squares are summed in another order, so a value
    # next to a border between two fp16 numbers may round to either: one step apart
    g = gen(4)
    x = randn(g, 1, 48 * HD)
    wq, wk = 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    table = dq.rope_table(64, theta=1e6)
    _, k, _ = dq.qkv_rope(x, i32([0]), table, 32, 8, q_norm=wq, k_norm=wk, dtype=torch.float16)
    planes = torch.zeros(2, 8, 64, HD, dtype=torch.float16, device="cuda")
    dq.attention_decode_rope(x[0, :32 * HD].reshape(32, HD), x[0, 32 * HD:40 * HD].reshape(8, HD), planes[0], planes[1],
                             wq, wk, table, 1)
    a, b = planes[0, :, 0].double(), k[0].double()
    assert bool(((a - b).abs() <= 2 * U[torch.float16] * b.abs() + 2 * TINY).all())


# ------------------------------------------------------------------ prompt


def prompt_ref(q, k, v, cu_q, cu_k):
    """(out, A) in 64 bits; rows of no sequence are NaN."""
    n_q, n_kv = q.shape[1], k.shape[1]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    size = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        i, j = torch.arange(b - a, device=q.device)[:, None], torch.arange(d - c, device=q.device)[None]
        seen = j <= i + (d - c) - (b - a)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            kk, vv = k[c:d, g].double(), v[c:d, g].double()
            s = (q[a:b, h].double() @ kk.T) / math.sqrt(HD)
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True) if d > c else torch.zeros(b - a, 1, dtype=torch.float64, device=q.device)
            p = torch.exp(s - top.nan_to_num(neginf=0.0))
            p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
            out[a:b, h], size[a:b, h] = p @ vv, p @ vv.abs()
    return out, size


def starts(lengths):
    return [0] + list(np.cumsum(lengths))


def check_prompt(dq, q, k, v, lq, lk=None, **kw):
    cu_q = starts(lq)
    cu_k = starts(lk) if lk is not None else cu_q
    y = dq.attention_prompt(q, k, v, i32(cu_q), None if lk is None else i32(cu_k), **kw)
    r, size = prompt_ref(q, k, v, cu_q, cu_k)
    live = cu_q[-1]
    within(y[:live], r[:live], (U[q.dtype] + 4e-5) * size[:live])
    return y


@pytest.mark.parametrize("n_q,n_kv", [(32, 8), (5, 1), (21, 3), (4, 4), (16, 2), (71, 1), (12, 4)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompt_head_layouts(dq, n_q, n_kv, dtype):
    g = gen(n_q)
    lq = [150, 1, 0, 37]
    t = sum(lq)
    check_prompt(dq, randn(g, t, n_q, HD, dtype=dtype), randn(g, t, n_kv, HD, dtype=dtype),
                 randn(g, t, n_kv, HD, dtype=dtype), lq)


@pytest.mark.parametrize("lq", [[1], [2], [31], [32], [33], [63, 65], [127], [128], [129], [255, 1, 257], [511], [513], [1030],
                                [0, 0, 5, 0], [1] * 70])
def test_prompt_lengths(dq, lq):
    g = gen(sum(lq))
    t = sum(lq)
    qkv = randn(g, t, 8 + 2 * 2, HD, dtype=torch.float16)  # slices of one projection
    check_prompt(dq, qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], lq)


@pytest.mark.parametrize("lq,lk", [
    ([1], [1000]), ([64], [1064]), ([64], [5000]), ([3, 1, 0, 130], [200, 129, 50, 131]), ([100], [64]), ([300, 7], [1, 0]),
    ([5], [0]), ([16, 16], [4096, 17]), ([200], [328]),
])
def test_prompt_key_lengths(dq, lq, lk):
    # more keys than queries (a cached prefix), fewer (first rows see nothing), none at all
    g = gen(sum(lk) + 1)
    n_q, n_kv = 16, 4
    q = randn(g, sum(lq), n_q, HD, dtype=torch.bfloat16)
    k, v = (randn(g, max(1, sum(lk)), n_kv, HD, dtype=torch.bfloat16) for _ in range(2))
    y = check_prompt(dq, q, k, v, lq, lk)
    at = 0
    for a, b in zip(lq, lk):
        assert bool((y[at:at + max(0, a - b)] == 0).all())
        at += a


@pytest.mark.parametrize("n", [128, 129, 700])
def test_prompt_many_sequences(dq, n):
    # more sequences than one look at the offsets takes (128), some of them empty or without keys
    g = gen(n)
    lq, lk = [i * 7 % 5 for i in range(n)], [i * 5 % 11 for i in range(n)]
    q, k, v = (randn(g, sum(x), h, HD, dtype=torch.float16) for x, h in ((lq, 4), (lk, 2), (lk, 2)))
    check_prompt(dq, q, k, v, lq, lk)
    assert dq.device_error() == 0
    bad = starts(lq)
    bad[3] = sum(lq) + 1  # far from the end, where the search begins: reported all the same
    dq.attention_prompt(q, k, v, i32(bad), i32(starts(lk)))
    assert dq.device_error() == BAD_ARG


def test_prompt_over_cache_planes_and_into_a_strided_output(dq):
    g = gen(9)
    planes = randn(g, 2, 4, 700, HD, dtype=torch.float16)  # [k or v][n_kv][max_ctx][128]
    wide = torch.full((50, 26, HD), 3.0, dtype=torch.float16, device="cuda")
    q = randn(g, 50, 16, HD, dtype=torch.float16)
    k, v = planes[0].transpose(0, 1)[:600], planes[1].transpose(0, 1)[:600]
    y = check_prompt(dq, q, k, v, [50], [600], out=wide[:, 4:20])
    assert y.data_ptr() == wide[:, 4:].data_ptr()
    assert bool((wide[:, :4] == 3).all()) and bool((wide[:, 20:] == 3).all())


@pytest.mark.parametrize("scale", [20.0, 60.0])
def test_prompt_with_peaked_scores(dq, scale):
    # a softmax that few keys share, its maximum rising along the keys
    g = gen(int(scale))
    lq = [400]
    q, k = randn(g, 400, 8, HD, dtype=torch.float16), randn(g, 400, 2, HD, dtype=torch.float16)
    v = randn(g, 400, 2, HD, dtype=torch.float16)
    k = (k * torch.linspace(0.01, 1, 400, device="cuda")[:, None, None]).half()
    q = (q * scale).half()
    cu = starts(lq)
    y = dq.attention_prompt(q, k, v, i32(cu))
    r, size = prompt_ref(q, k, v, cu, cu)
    # a score s is off by up to 128 roundings (2^-24 each) of sum |q k| / sqrt(128) <= 128 * 4 scale / 11.3
    # (|k| <= 1 by its ramp times a few): 128 * 2^-24 * 45 scale = 3.5e-4 scale, twice (numerator and sum)
    within(y, r, (U[q.dtype] + 7e-4 * scale) * size)


def test_prompt_masked_infinities_and_nans_take_no_part(dq):
    g = gen(11)
    lq = [200, 100]
    t = 330  # 30 rows of no sequence
    q, k, v = (randn(g, t, n, HD, dtype=torch.float16) for n in (8, 2, 2))
    clean = dq.attention_prompt(q, k, v, i32(starts(lq)))
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    for x in (k2, v2, q2):
        x[300:] = float("nan")
    v2[300:310], k2[300:310] = float("inf"), float("-inf")
    # the last key of the first sequence: only its last query sees it
    v2[199, 0, 5], v2[199, 1, 7], k2[199, 1] = float("nan"), float("inf"), float("nan")
    # a key in the middle of the second sequence: queries from 260 on see it
    v2[260, 0, 3], v2[260, 0, 4] = float("-inf"), float("nan")
    y = dq.attention_prompt(q2, k2, v2, i32(starts(lq)))
    want = clean.clone()
    assert torch.equal(y[:199], clean[:199]) and torch.equal(y[200:260], clean[200:260])
    assert bool(torch.isnan(y[199, :4, 5]).all()) and bool(torch.isnan(y[199, 4:]).all())
    keep = torch.ones(HD, dtype=torch.bool, device="cuda")
    keep[5] = False
    assert torch.equal(y[199, :4][:, keep], want[199, :4][:, keep])
    late = y[260:300, :4]
    assert bool((late[..., 3] == float("-inf")).all()) and bool(torch.isnan(late[..., 4]).all())
    keep[5], keep[3], keep[4] = True, False, False
    assert torch.equal(late[..., keep], want[260:300, :4][..., keep])
    assert torch.equal(y[260:300, 4:], want[260:300, 4:])


def test_prompt_split_keys_with_infinities_and_nans(dq):
    # few queries over many keys: several blocks share the keys of one query tile
    g = gen(14)
    lk, n = 3000, 10
    q, k, v = randn(g, n, 8, HD, dtype=torch.bfloat16), *(randn(g, lk, 2, HD, dtype=torch.bfloat16) for _ in range(2))
    cu, ck = i32([0, n]), i32([0, lk])
    clean = dq.attention_prompt(q, k, v, cu, ck)
    r, size = prompt_ref(q, k, v, [0, n], [0, lk])
    within(clean, r, (U[q.dtype] + 4e-5) * size)
    v2 = v.clone()
    v2[lk - 3, 0, 9] = float("inf")  # seen by the last three queries
    v2[lk - 1, 1, 100] = float("nan")  # by the last one
    v2[100, 1, 7] = float("-inf")  # by all
    y = dq.attention_prompt(q, k, v2, cu, ck)
    want = clean.clone()
    want[n - 3:, :4, 9] = float("inf")
    want[n - 1, 4:, 100] = float("nan")
    want[:, 4:, 7] = float("-inf")
    assert torch.equal(torch.nan_to_num(y, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


def test_prompt_leaves_other_rows_and_reports_bad_offsets(dq):
    g = gen(12)
    q, k, v = (randn(g, 60, n, HD, dtype=torch.bfloat16) for n in (4, 2, 2))
    out = torch.full_like(q, 9.0)
    dq.attention_prompt(q, k, v, i32([5, 20, 20, 41]), out=out)  # rows before the first and after the last
    assert dq.device_error() == 0
    assert bool((out[:5] == 9).all()) and bool((out[41:] == 9).all()) and not bool((out[5:41] == 9).all(-1).any())
    r, size = prompt_ref(q, k, v, [5, 20, 20, 41], [5, 20, 20, 41])
    within(out[5:41], r[5:41], (U[q.dtype] + 4e-5) * size[5:41])
    for cu in ([0, 20, 10, 30], [0, 20, 61, 30], [-3, 10, 20, 30]):
        out.fill_(9.0)
        dq.attention_prompt(q, k, v, i32(cu), out=out)
        assert dq.device_error() == BAD_ARG
    dq.attention_prompt(q, k, v, i32([0, 20, 40]), cu_k=i32([0, 30, 20]), out=out)
    assert dq.device_error() == BAD_ARG


def test_prompt_offsets_past_32_bits(dq):
    # the last rows of a plane of 5 GB; only they are written and read
    g = gen(13)
    rows = 1 << 24
    big = torch.empty(rows, 1, 160, dtype=torch.float16, device="cuda")[..., :HD]
    big[-300:] = randn(g, 300, 1, HD, dtype=torch.float16)
    q = randn(g, 20, 4, HD, dtype=torch.float16)
    y = dq.attention_prompt(q, big, big, i32([0, 20]), i32([rows - 300, rows]))
    r, size = prompt_ref(q, big[-300:], big[-300:], [0, 20], [0, 300])
    within(y, r, (U[q.dtype] + 4e-5) * size)


# --------------------------------------------------------------- 4-bit cache


def quantise_ref(x):
    """numpy fp32 steps of the format -> (d, z fp64 [..., 4], codes [..., 128], values fp64)."""
    g = x.reshape(*x.shape[:-1], 4, 32).astype(np.float32)
    lo, hi = g.min(-1), g.max(-1)
    with np.errstate(all="ignore"):
        d = ((hi - lo) / np.float32(15)).astype(np.float16)
        z = (lo + np.float32(8) * d.astype(np.float32)).astype(np.float16)
        bad = ~(np.isfinite(d) & np.isfinite(z) & np.isfinite(g).all(-1))
        d, z = (np.where(bad, np.float16(np.nan), a) for a in (d, z))
        t = np.rint((g - z.astype(np.float32)[..., None]) / d.astype(np.float32)[..., None]) + 8
        c = np.where((d > 0)[..., None], np.clip(np.nan_to_num(t, nan=8.0), 0, 15), 8).astype(np.int64)
        val = d.astype(np.float64)[..., None] * (c - 8) + z.astype(np.float64)[..., None]
    return d, z, c.reshape(x.shape), val.reshape(x.shape)


def block_bytes_ref(dk, zk, ck, dv, zv, cv):
    """One row's contribution, byte by byte from the header's definition: {(byte, nibble or None): value}."""
    def put(j):
        got = {}
        for n in range(HD):
            g, t, e, r, i = n // 32, n % 32 // 8, n % 8, n % 32 // 4, n % 4
            bit = 4 * (e // 2) + 16 * (e % 2)
            got[64 * j + 4 * (4 * t + g) + bit // 8, bit // 4 % 2] = int(ck[n])
            base = 1024 + 512 * (j // 8) + 16 * (4 * r + j // 2 % 4) + 4 * g + 2 * (j % 2)
            got[base + i // 2, i % 2] = int(cv[n])
        for base, d, z in ((2048, dk, zk), (2304, dv, zv)):
            for g in range(4):
                for s, x in ((0, d), (4, z)):
                    for b, byte in enumerate(np.float16(x[g]).tobytes()):
                        got[base + 32 * (j // 2) + 8 * g + 2 * (j % 2) + s + b, None] = byte
        return got
    return put


def rows_for(seed, rows, n_kv, dtype):
    g = gen(seed)
    k, v = randn(g, rows, n_kv, HD, dtype=dtype), randn(g, rows, n_kv, HD, dtype=dtype)
    k[:, :, 3] *= 20  # an outlier channel
    k[0, 0, :32] = 0.75  # a constant group
    v[-1, -1, 32:64] = 0
    v[0, 0, 64:96] *= 1e-6 if dtype != torch.float16 else 1e-3  # scales below fp16's normal range
    return k, v


@pytest.mark.parametrize("rows,n_kv,page,dtype", [
    (1, 8, 64, torch.float32), (17, 1, 16, torch.float16), (100, 3, 48, torch.bfloat16), (33, 2, 256, torch.float32),
    (500, 8, 64, torch.float16),
])
def test_append_and_read(dq, rows, n_kv, page, dtype):
    k, v = rows_for(rows, rows, n_kv, dtype)
    pages = -(-rows // page) + 2
    slots = torch.randperm(pages * page, device="cuda", generator=gen(1))[:rows].int()
    pool = dq.kv4_pool(pages, n_kv, page)
    dq.kv4_append(k, v, slots, pool)
    raw = pool.cpu().numpy()
    refs = [quantise_ref(x.float().cpu().numpy()) for x in (k, v)]
    for r in range(0, rows, max(1, rows // 7)):
        s = int(slots[r])
        for g in range(n_kv):
            b = raw[s // page, g, s % page // 16]
            want = block_bytes_ref(*[refs[0][i][r, g] for i in range(3)], *[refs[1][i][r, g] for i in range(3)])(s % 16)
            for (at, nib), x in want.items():
                got = int(b[at]) if nib is None else int(b[at]) >> (4 * nib) & 15
                assert got == x, (r, g, at, nib)
    unused = torch.ones(pages * page, dtype=torch.bool)
    unused[slots.cpu().long()] = False
    for out in (torch.float32, torch.float16, torch.bfloat16):
        for y, (_, _, _, val) in zip(dq.kv4_read(pool, slots, dtype=out), refs):
            within(y.cpu(), torch.from_numpy(val), 0.0)
    for y in dq.kv4_read(pool, torch.nonzero(unused).flatten().int().cuda(), dtype=torch.float32):
        assert bool((y == 0).all())  # rows that no slot names were not touched


def test_append_takes_strides_and_every_row_of_a_page(dq):
    g = gen(21)
    n_kv, page = 2, 32
    qkv = randn(g, 64, 4 + 2 * n_kv, HD, dtype=torch.bfloat16)
    planes = randn(g, n_kv, 64, HD, dtype=torch.bfloat16).transpose(0, 1)
    slots = torch.arange(64, device="cuda").flip(0).int()
    a, b = dq.kv4_pool(2, n_kv, page), dq.kv4_pool(2, n_kv, page)
    dq.kv4_append(qkv[:, 4:4 + n_kv], planes, slots, a)
    dq.kv4_append(qkv[:, 4:4 + n_kv].contiguous(), planes.contiguous(), slots, b)
    assert torch.equal(a, b)
    k, v = dq.kv4_read(a, slots, dtype=torch.float32)
    for y, x in ((k, qkv[:, 4:4 + n_kv]), (v, planes)):
        within(y, torch.from_numpy(quantise_ref(x.float().cpu().numpy())[3]).cuda(), 0.0)


def test_append_non_finite_groups_are_nan_and_spread_no_further(dq):
    x = randn(gen(22), 4, 1, HD)
    x[0, 0, 5], x[1, 0, 40], x[2, 0, 70] = float("nan"), float("inf"), float("-inf")
    x[3, 0, 100], x[3, 0, 1] = 3e6, 30000.0  # a scale past fp16's range; a large one within it
    pool, slots = dq.kv4_pool(1, 1, 16), i32([0, 1, 2, 3])
    dq.kv4_append(x, x, slots, pool)
    for y in dq.kv4_read(pool, slots, dtype=torch.float32):
        nan = torch.isnan(y).reshape(4, 4, 32)
        want = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
        want[0, 0] = want[1, 1] = want[2, 2] = want[3, 3] = True
        assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)
        r = torch.from_numpy(quantise_ref(x.cpu().numpy())[3]).cuda()
        ok = ~torch.isnan(y)
        within(y[ok], r[ok], 0.0)


def test_append_and_read_skip_padding_and_report_slots_past_the_pool(dq):
    k = randn(gen(23), 5, 2, HD)
    pool = dq.kv4_pool(2, 2, 16)
    dq.kv4_append(k, k, i32([-1, 3, -7, 31, -2147483648]), pool)
    assert dq.device_error() == 0
    out = tuple(torch.full((4, 2, HD), 5.0, device="cuda") for _ in range(2))
    dq.kv4_read(pool, i32([3, -1, 31, 3]), dtype=torch.float32, out=out)
    r = torch.from_numpy(quantise_ref(k.cpu().numpy())[3]).cuda()
    for y in out:
        within(y[[0, 2, 3]], r[[1, 3, 1]], 0.0)
        assert bool((y[1] == 5).all())
    before = pool.clone()
    dq.kv4_append(k, k, i32([32, -1, 2147483647, -1, -1]), pool)
    assert dq.device_error() == BAD_ARG and torch.equal(pool, before)
    dq.kv4_read(pool, i32([32, -1, 40, -1]), dtype=torch.float32, out=out)
    assert dq.device_error() == BAD_ARG


# ------------------------------------------------------------------- decode


def decode_ref(q, k, v, n_keys):
    """q [n_seq, n_q, 128], k, v lists of fp64 [n, n_kv, 128] -> (out, A)."""
    out, size = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape, dtype=torch.float64,
                                                                                       device=q.device)
    for b, n in enumerate(n_keys):
        if n == 0:
            continue
        group = q.shape[1] // k[b].shape[1]
        kk, vv = (x[:n].repeat_interleave(group, 1).transpose(0, 1) for x in (k[b], v[b]))
        s = (kk @ q[b].double()[..., None])[..., 0] / math.sqrt(HD)
        p = torch.softmax(s, 1)[:, None]
        out[b], size[b] = (p @ vv)[:, 0], (p @ vv.abs())[:, 0]
    return out, size


def build_cache(dq, seed, lengths, n_kv, page, spare=2):
    """A pool whose pages are scattered over the sequences; unused rows hold NaN scales."""
    g = gen(seed)
    need = [max(1, -(-n // page)) for n in lengths]
    pages = sum(need) + spare
    pool = torch.full((pages, n_kv, page // 16, 2560), 0xFF, dtype=torch.uint8, device="cuda")
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((len(lengths), max(need) + 1), -12345, dtype=torch.int32, device="cuda")
    ks, vs, zs, at = [], [], [], 0
    for b, n in enumerate(lengths):
        mine = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine
        if n == 0:
            ks.append(None), vs.append(None), zs.append(None)
            continue
        k, v = randn(g, n, n_kv, HD), randn(g, n, n_kv, HD)
        j = torch.arange(n, device="cuda")
        slots = (mine[j // page] * page + j % page).int()
        dq.kv4_append(k, v, slots, pool)
        kk, vv = dq.kv4_read(pool, slots, dtype=torch.float32)  # exact: checked above
        ks.append(kk.double()), vs.append(vv.double())
        z = torch.from_numpy(quantise_ref(v.cpu().numpy())[1].astype(np.float64)).cuda()
        zs.append(z.repeat_interleave(32, -1))
    return pool, table, ks, vs, zs


def decode_slack(q, ks, vs, zs, lengths, size):
    if q.dtype == torch.float32:
        return 2e-5 * size
    parts = [None if v is None else (v - z).abs() + z.abs() for v, z in zip(vs, zs)]
    return 6e-5 * size + 2.0 ** -11 * decode_ref(q, ks, parts, lengths)[0]


@pytest.mark.parametrize("n_q,n_kv,lengths,page,dtype", [
    (32, 8, [513], 64, torch.float32), (32, 8, [1], 16, torch.float32), (5, 1, [0, 1, 15, 16, 17], 16, torch.float16),
    (21, 3, [31, 32, 33, 100], 32, torch.bfloat16), (4, 4, [257, 3, 64], 48, torch.float32),
    (16, 2, [1000, 0, 4097, 129], 128, torch.float32), (32, 8, [60] * 40, 64, torch.float16),
    (8, 1, [20000], 256, torch.float32), (2, 1, [5000, 10], 16, torch.float32), (7, 1, [300], 16, torch.float32),
    (12, 2, [2047, 2048, 2049, 511, 512], 64, torch.bfloat16), (64, 64, [200], 64, torch.float32),
])
def test_decode(dq, n_q, n_kv, lengths, page, dtype):
    pool, table, ks, vs, zs = build_cache(dq, sum(lengths), lengths, n_kv, page)
    q = randn(gen(31), len(lengths), n_q, HD, dtype=dtype)
    r, size = decode_ref(q, ks, vs, lengths)
    for most in (max(1, max(lengths)), table.shape[1] * page):  # the split goes by the bound, the result does not
        y = dq.attention_decode_kv4(q, pool, table, i32(lengths), most)
        assert dq.device_error() == 0
        within(y, r, decode_slack(q, ks, vs, zs, lengths, size))
    for b, n in enumerate(lengths):
        assert n > 0 or bool((y[b] == 0).all())
    assert torch.equal(dq.attention_decode_kv4(q, pool, table, i32(lengths)), y)  # the same call, the same bits


def test_decode_peaked_and_shared_pages(dq):
    # two sequences over the same pages (a fork), queries large enough that one key takes most of the weight
    pool, table, ks, vs, zs = build_cache(dq, 41, [700], 2, 64)
    q = randn(gen(42), 2, 8, HD) * 12
    both = table.repeat(2, 1)
    y = dq.attention_decode_kv4(q, pool, both, i32([700, 350]), 700)
    r, size = decode_ref(q, ks * 2, vs * 2, [700, 350])
    # a score is off by at most (2^-21 + 128 * 2^-24) * sum |q k| / sqrt(128), sum |q k| <= 128 * 12 here
    within(y, r, 2 * 8.2e-6 * 128 * 12 / 11.3 * size)


def test_decode_small_values_beside_an_outlier_channel(dq):
    # Equal scores: every p_j is the same 2^e, e = cap - 3 or more.  The outlier's scale is below 16, which lowers
    # the cap of 12 to 11: 600 products p d of the small groups are off by at most half of 2^-24 (fp16's smallest, the
    # second part's step) times |c - 8| <= 8 each, over a sum of 600 2^8: 2^-22 2^-8 = 2^-30 beside the usual bound.
    # In the outlier's own group v is a difference: its bound goes by B = sum p (|v - z| + |z|) in place of A.
    g = gen(51)
    n, page = 600, 64
    k, v = randn(g, n, 2, HD), randn(g, n, 2, HD) * 1e-4
    v[:, :, 3] = 400 * torch.rand(n, 2, device="cuda", generator=g) - 200  # one a group: d = |v| / 15
    pool, table = dq.kv4_pool(10, 2, page), torch.arange(10, device="cuda").int()[None]
    slots = torch.arange(n, device="cuda").int()
    dq.kv4_append(k, v, slots, pool)
    kk, vv = (x.double() for x in dq.kv4_read(pool, slots, dtype=torch.float32))
    d, z = quantise_ref(v.cpu().numpy())[:2]
    assert 8 < float(d.max()) < 16
    z = torch.from_numpy(z.astype(np.float64)).cuda().repeat_interleave(32, -1)
    q = torch.zeros(1, 8, HD, device="cuda")
    y = dq.attention_decode_kv4(q, pool, table, i32([n]), n)
    r, size = decode_ref(q, [kk], [vv], [n])
    parts = decode_ref(q, [kk], [(vv - z).abs() + z.abs()], [n])[0]
    within(y[..., 32:], r[..., 32:], 2e-5 * size[..., 32:] + 2.0 ** -30)
    within(y[..., :32], r[..., :32], 2e-5 * parts[..., :32])


def test_decode_masked_rows_may_hold_anything(dq):
    pool, table, ks, vs, zs = build_cache(dq, 43, [70, 0, 5], 2, 64)  # unused rows: NaN scales, all codes 15
    q = randn(gen(44), 3, 4, HD)
    r, size = decode_ref(q, ks, vs, [70, 0, 5])
    within(dq.attention_decode_kv4(q, pool, table, i32([70, 0, 5]), 128), r, 2e-5 * size)
    x = torch.full((1, 2, HD), float("nan"), device="cuda")
    seen = table[0, 0] * 64 + 3
    dq.kv4_append(x, x, seen.reshape(1).int(), pool)
    y = dq.attention_decode_kv4(q, pool, table, i32([3, 0, 5]), 128)  # not seen
    assert not bool(torch.isnan(y).any())
    y = dq.attention_decode_kv4(q, pool, table, i32([4, 0, 5]), 128)  # seen: that sequence alone
    assert bool(torch.isnan(y[0]).all()) and not bool(torch.isnan(y[1:]).any())


def test_decode_reports_bad_counts_and_pages(dq):
    pool, table, ks, vs, zs = build_cache(dq, 45, [70, 40, 9], 2, 32)
    q = randn(gen(46), 3, 4, HD)
    r, size = decode_ref(q, ks, vs, [70, 40, 9])
    for bad in (-1, 97, 2147483647):
        y = dq.attention_decode_kv4(q, pool, table, i32([70, bad, 9]), 96)
        assert dq.device_error() == BAD_ARG
        assert bool((y[1] == 0).all())
        within(y[[0, 2]], r[[0, 2]], 2e-5 * size[[0, 2]])
    for bad in (-1, pool.shape[0], 2147483647):
        t = table.clone()
        t[1, 0] = bad
        y = dq.attention_decode_kv4(q, pool, t, i32([70, 40, 9]), 96)
        assert dq.device_error() == BAD_ARG
        within(y[[0, 2]], r[[0, 2]], 2e-5 * size[[0, 2]])
        rest, rsize = decode_ref(q[1:2], [ks[1][32:]], [vs[1][32:]], [8])
        within(y[1:2], rest, 2e-5 * rsize)


def test_decode_in_place(dq):
    pool, table, ks, vs, zs = build_cache(dq, 47, [300], 2, 32)
    q = randn(gen(48), 1, 8, HD)
    want = dq.attention_decode_kv4(q, pool, table, i32([300]), 300)
    dq.attention_decode_kv4(q, pool, table, i32([300]), 300, out=q)
    assert torch.equal(q, want)


# ------------------------------------------------------- workspaces and devices


def test_workspaces_are_checked(dq):
    import ctypes

    lib = dq.load()
    g = gen(71)
    # one query tile over many keys: split, so a workspace is needed
    q, k, v = randn(g, 4, 8, HD, dtype=torch.float16), *(randn(g, 4000, 2, HD, dtype=torch.float16) for _ in range(2))
    need = lib.dq_attention_prompt_workspace_bytes(1, 4, 4000, 8, 2)
    assert need > 0
    cu, ck, out = i32([0, 4]), i32([0, 4000]), torch.empty_like(q)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")

    def call(w, n):
        d = dq._Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 1024, 128, 256, 128, 256, 128, 1024, 128,
                       cu.data_ptr(), ck.data_ptr(), dq.TYPE_F16, 1, 4, 4000, 8, 2, 128, w, n)
        return lib.dq_attention_prompt(ctypes.byref(d), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))

    assert call(None, 0) == -1 and call(ws.data_ptr(), need - 1) == -2 and call(ws.data_ptr() + 8, need) == -3
    ws.fill_(0xFF)  # its content is of no meaning
    assert call(ws.data_ptr(), need) == 0
    assert torch.equal(out, dq.attention_prompt(q, k, v, cu, ck))
    with pytest.raises(dq.DQError):
        dq.attention_prompt(q, k, v, cu, ck, workspace=ws[:64])

    pool, table, _, _, _ = build_cache(dq, 72, [2000], 2, 64)
    x, n = randn(g, 1, 8, HD), i32([2000])
    ws = dq.attention_decode_kv4_workspace(1, 8, 2, 2000)
    assert ws is not None
    want = dq.attention_decode_kv4(x, pool, table, n, 2000)
    ws.fill_(0xFF)
    assert torch.equal(dq.attention_decode_kv4(x, pool, table, n, 2000, workspace=ws), want)
    with pytest.raises(dq.DQError):
        dq.attention_decode_kv4(x, pool, table, n, 2000, workspace=ws[:64])


def test_tensors_off_the_current_device_are_refused(dq):
    g = gen(73)
    q, k = randn(g, 4, 8, HD, dtype=torch.float16), randn(g, 4, 2, HD, dtype=torch.float16)
    cu, pool, slots = i32([0, 4]), dq.kv4_pool(1, 2, 16), i32([0, 1, 2, 3])
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k.cpu(), k, cu)
    with pytest.raises(ValueError):
        dq.attention_prompt(q, k, k, cu.cpu())
    with pytest.raises(ValueError):
        dq.kv4_append(k, k, slots.cpu(), pool)
    with pytest.raises(ValueError):
        dq.kv4_read(pool.cpu(), slots)
    with pytest.raises(ValueError):
        dq.attention_decode_kv4(q, pool, torch.zeros(4, 1, dtype=torch.int32), slots, 16)
    with pytest.raises(ValueError):
        dq.qkv_rope(randn(g, 4, 4 * HD), slots, dq.rope_table(16), 2, 1, q_norm=torch.ones(HD), k_norm=torch.ones(HD))


def test_two_streams_at_once(dq):
    # calls without a shared workspace do not meet, whichever streams they run on
    g = gen(74)
    pool, table, _, _, _ = build_cache(dq, 75, [3000, 700], 2, 64)
    n = i32([3000, 700])
    x = [randn(g, 2, 8, HD) for _ in range(4)]
    q = [randn(g, 700, 8, HD, dtype=torch.bfloat16) for _ in range(4)]
    k = [randn(g, 700, 2, HD, dtype=torch.bfloat16) for _ in range(4)]
    cu = i32([0, 33, 700])
    want = [(dq.attention_decode_kv4(a, pool, table, n, 3000), dq.attention_prompt(b, c, c, cu)) for a, b, c in zip(x, q, k)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        got = []
        for i in range(4):
            with torch.cuda.stream(streams[i % 2]):
                got.append((dq.attention_decode_kv4(x[i], pool, table, n, 3000), dq.attention_prompt(q[i], k[i], k[i], cu)))
        torch.cuda.synchronize()
        for (a, b), (c, d) in zip(got, want):
            assert torch.equal(a, c) and torch.equal(b, d)


def test_first_call_may_be_captured(tmp_path):
    # a fresh process whose first use of the kernels is inside a capture
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys; sys.path.insert(0, %r)
import torch
from quantised_gemv_norm_gb300 import dq
dq.load()
q = torch.randn(70, 8, 128, device='cuda').half(); k = torch.randn(70, 2, 128, device='cuda').half()
cu = torch.tensor([0, 70], dtype=torch.int32, device='cuda')
x = torch.randn(70, 12 * 128, device='cuda'); pos = torch.arange(70, dtype=torch.int32, device='cuda')
table = torch.ones(128, 64, 2, device='cuda'); pool = dq.kv4_pool(2, 2, 64); pages = pos[:2].reshape(1, 2)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = dq.attention_prompt(q, k, k, cu)
    a, b, c = dq.qkv_rope(x, pos, table, 8, 2)
    dq.kv4_append(b, c, pos, pool)
    d, e = dq.kv4_read(pool, pos)
    z = dq.attention_decode_kv4(a[:1].float(), pool, pages, pos[69:], 128)
g.replay(); torch.cuda.synchronize()
assert torch.equal(y, dq.attention_prompt(q, k, k, cu))
assert torch.equal(z, dq.attention_decode_kv4(a[:1].float(), pool, pages, pos[69:], 128))
assert dq.device_error() == 0
print('captured')
""" % root
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------- all together


def test_prompt_then_tokens(dq):
    """Two prompts through head norm and rotation, prompt attention and the store; then tokens over the stored cache, and
    a second piece of the first prompt over its rows read back."""
    g = gen(51)
    n_q, n_kv, page = 8, 2, 32
    lens = [70, 33]
    t = sum(lens)
    table = dq.rope_table(256)
    wq, wk = 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    norms = dict(q_norm=wq, k_norm=wk)
    qkv = randn(g, t, (n_q + 2 * n_kv) * HD)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    q, k, v = dq.qkv_rope(qkv, pos, table, n_q, n_kv, dtype=torch.float16, **norms)
    check_prompt(dq, q, k, v, lens)
    pages = i32([[4, 1, 6, 2], [0, 5, -1, -1]])
    pool = dq.kv4_pool(8, n_kv, page)
    seq = torch.repeat_interleave(torch.arange(2), torch.tensor(lens)).cuda()
    slots = (pages[seq, (pos // page).long()] * page + pos % page).int()
    dq.kv4_append(k, v, slots, pool)
    keys, values = dq.kv4_read(pool, slots, dtype=torch.float32)
    hist = [(keys[:70].double(), values[:70].double()), (keys[70:].double(), values[70:].double())]
    for step in range(3):
        n = [70 + step, 33 + step]
        x = randn(g, 2, (n_q + 2 * n_kv) * HD)
        at = i32(n)
        q1, k1, v1 = dq.qkv_rope(x, at, table, n_q, n_kv, dtype=torch.float32, **norms)
        new = (pages[torch.arange(2, device="cuda"), (at // page).long()] * page + at % page).int()
        dq.kv4_append(k1, v1, new, pool)
        kk, vv = dq.kv4_read(pool, new, dtype=torch.float32)
        hist = [(torch.cat([a, kk[i:i + 1].double()]), torch.cat([b, vv[i:i + 1].double()]))
                for i, (a, b) in enumerate(hist)]
        y = dq.attention_decode_kv4(q1, pool, pages, at + 1, 128)
        r, size = decode_ref(q1, [h[0] for h in hist], [h[1] for h in hist], [m + 1 for m in n])
        within(y, r, 2e-5 * size)
    back = torch.arange(70, device="cuda")
    rows = (pages[0, back // page] * page + back % page).int()
    kc, vc = dq.kv4_read(pool, rows, dtype=torch.float16)
    x = randn(g, 20, (n_q + 2 * n_kv) * HD)
    q2, k2, v2 = dq.qkv_rope(x, torch.arange(70, 90).int().cuda(), table, n_q, n_kv, dtype=torch.float16, **norms)
    check_prompt(dq, q2, torch.cat([kc, k2]), torch.cat([vc, v2]), [20], [90])
    assert dq.device_error() == 0


def test_captured_into_a_graph_and_replayed_on_another_stream(dq):
    g = gen(61)
    n_q, n_kv, page = 8, 2, 32
    pool, table, _, _, _ = build_cache(dq, 62, [300, 45], n_kv, page, spare=4)
    n_keys = i32([300, 45])
    x = randn(g, 2, (n_q + 2 * n_kv) * HD)
    rope = dq.rope_table(512)
    q, k, v = (torch.empty(2, n, HD, device="cuda") for n in (n_q, n_kv, n_kv))
    ws = dq.attention_decode_kv4_workspace(2, n_q, n_kv, 320)
    pq, pk, pv = (randn(g, 300, n, HD, dtype=torch.float16) for n in (n_q, n_kv, n_kv))
    cu = i32([0, 299, 300])
    slots = i32([table[0, 9].item() * page + 12, table[1, 1].item() * page + 13])

    def step():
        dq.qkv_rope(x, n_keys, rope, n_q, n_kv, dtype=torch.float32, out=(q, k, v))
        dq.kv4_append(k, v, slots, pool)
        return dq.attention_decode_kv4(q, pool, table, n_keys, 320, workspace=ws), dq.attention_prompt(pq, pk, pv, cu)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2):
        x.copy_(randn(gen(seed), *x.shape))
        pq.copy_(randn(gen(seed), *pq.shape, dtype=torch.float16))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got_now = [y.clone() for y in got]
        want = step()
        for a, b in zip(got_now, want):
            assert torch.equal(a, b)
