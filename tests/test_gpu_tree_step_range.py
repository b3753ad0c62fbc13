"""GPU tests of the tree attention over its number range: scores far from zero on both sides of the size from which their
reference is subtracted first, in batches whose blocks go through several key tiles and items.

Queries and keys are such that a score is a sum of multiples of 1/16 below 2^17: exact in fp32 in any order.  What is left
of the bound is then, relative to sum p |v|,
  u + 4e-5       as in every test of the attention, and
  2 * 2^-23 X ln 2   X = |m| log2(e) / sqrt(128), for a row whose largest score is at most 32768: there the tensor-core
                 kernel has c s and c m rounded (2^-24 X each) before their difference is taken, which is in the numerator
                 and in the sum of the probabilities."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HD = 128
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F16, BF16 = torch.float16, torch.bfloat16
C = 1.4426950408889634 / math.sqrt(HD)


@pytest.fixture(scope="module")
def dq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantised_gemv_norm_gb300 import build, dq as dqmod

    build.build()
    dqmod.load()
    yield dqmod
    assert dqmod.device_error() == 0


def quarters(g, *shape):
    """Multiples of 1/4 in -1.5 .. 1.5."""
    return torch.randint(-6, 7, shape, device="cuda", generator=g).float() / 4


def inputs(n_seq, past, new, n_q, sizes, dtype, step, seed):
    """One KV head; row r's queries have dim 0 = sizes[r % len], the keys 127.5: scores around 127.5 size, growing by
    `step` from one 128 keys to the next."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    keys, page = past + new, 32
    wide = -(-keys // page)
    pages = torch.randperm(n_seq * wide, device="cuda", generator=g).int().reshape(n_seq, wide)
    kv = torch.randn((n_seq * wide, 2, 1, page, HD), device="cuda", generator=g)
    j = torch.arange(wide * page, device="cuda")
    k = torch.randn((n_seq, wide * page, HD), device="cuda", generator=g)
    k[..., 0] = 127.5
    k[..., 1] = step * (j // 128)
    k[..., 2:8] = quarters(g, n_seq, wide * page, 6)
    kv[pages.long(), 0, 0] = k.reshape(n_seq, wide, page, HD)
    pool = kv.to(dtype)
    q = torch.zeros((n_seq * new, n_q, HD), device="cuda")
    at = torch.arange(n_seq * new * n_q, device="cuda").reshape(-1, n_q)
    q[..., 0] = torch.tensor(sizes, device="cuda", dtype=torch.float32)[at % len(sizes)]
    q[..., 1] = 1
    q[..., 2:8] = quarters(g, n_seq * new, n_q, 6)
    return pool, q.to(dtype), pages


def reference(q, pool, pages, past, new):
    """fp64 outputs, sum p |v| and the largest score of every row, chains."""
    n_seq, n_q = pages.shape[0], q.shape[1]
    kv = pool[pages.long()].double()  # seq, page, 2, 1, row, dim
    k, v = (kv[:, :, a, 0].flatten(1, 2)[:, :past + new] for a in (0, 1))
    qs = q.double().reshape(n_seq, new, n_q, HD).flatten(1, 2)
    s = qs @ k.transpose(1, 2)
    i = torch.arange(new, device="cuda").repeat_interleave(n_q)
    s.masked_fill_(torch.arange(past + new, device="cuda")[None, :] > past + i[:, None], -math.inf)
    m = s.amax(-1)
    p = torch.softmax(s / math.sqrt(HD), -1)
    return (p @ v).reshape(q.shape), (p @ v.abs()).reshape(q.shape), m.reshape(q.shape[:2])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [1, 9, 40])  # the kernels of few rows, of one and of two query tiles
@pytest.mark.parametrize("n_seq", [1, 160])  # a key tile a block, and six of each sequence
@pytest.mark.parametrize("step", [0, 40, 80])  # of 62.7 on, the reference follows from tile to tile
def test_scores_far_from_zero_are_exact(dq, dtype, new, n_seq, step):
    past, n_q = 700, 4
    sizes = [512, 256, -512, 128, -256, 0, 256.0, 255]  # 512: far; 256: 32640, past 32768 some tiles on
    pool, q, pages = inputs(n_seq, past, new, n_q, sizes, dtype, step, 7 + new)
    n_past = torch.full((n_seq,), past, dtype=torch.int32, device="cuda")
    ref, mag, m = reference(q, pool, pages, past, new)
    far = m.abs() > 32768
    assert bool(far.any()) and bool((~far).any())
    if step:
        crossing = (m > 32768) & (m < 33300)
        assert bool(crossing.any())
    out = dq.attention_tree(q, pool, pages, n_past)
    u = U[dtype]
    off = torch.where(far, 0.0, 2 * 2.0 ** -23 * m.abs() * C * math.log(2))
    d = (out.double() - ref).abs() - ((u + 4e-5 + off)[..., None] * mag + u * ref.abs() + 2.0 ** -25)
    assert bool((d <= 0).all()), "worst excess %g" % float(d.max())
