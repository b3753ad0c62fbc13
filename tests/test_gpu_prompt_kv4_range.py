"""GPU tests of the prompt and 4-bit cache attention at the ends of their number ranges: probabilities far below the
largest one, scores far from zero, value scales of very different sizes in one cache.

The bounds are those of test_gpu_prompt_kv4.py; what is added to them stands at each test.
"""
import math

import pytest
import torch

from test_gpu_prompt_kv4 import dq, gen, HD, i32, prompt_ref, randn, U, within

pytestmark = pytest.mark.gpu
assert dq  # the fixture


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
