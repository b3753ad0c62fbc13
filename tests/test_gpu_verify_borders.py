"""GPU tests of the verification where a decision lies within a 32-bit rounding of its border.

The kernel's sums of weights are good to about 2^-22 in its first pass; where that does not settle a decision it takes
the sum again to 2^-38 and a place's weight to 2^-52.  The inputs here put decisions 2^-20 to 2^-30 of their numbers
from the border, where 64-bit arithmetic (2^-52) settles them and a 32-bit sum does not.  Outputs are whole numbers:
equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

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


def randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def exponential(g, *shape):
    return torch.empty(shape, device="cuda").exponential_(generator=g).clamp_min_(1e-30)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def weights(row, temp=1.0):
    x = row.double()
    return torch.exp((x - x.max()) / temp)


def best(score):
    """The place of the largest, the lowest of equal ones."""
    return int((score == score.max()).nonzero()[0])


def spread(g, rows, vocab, dtype):
    """Logits over a range of about 20, with ties in 16 bits."""
    return (3.0 * randn(g, rows, vocab)).to(dtype)


@pytest.mark.parametrize("n_seq,vocab", [(1, 20000), (40, 5003), (330, 700)])  # 16 blocks a sequence, 4, 1
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_next_token_among_near_ratios(dq, n_seq, vocab, dtype):
    """noise = the weight rounded to 32 bits: every ratio is 1 but for 2^-24, and one is the largest."""
    g = gen(n_seq)
    logits = spread(g, n_seq, vocab, dtype)
    noise = torch.stack([weights(r).float() for r in logits])
    want = [best(weights(r) / e.double()) for r, e in zip(logits, noise)]
    after = dq.verify_draft(logits, i32([0] * n_seq), torch.zeros(n_seq, device="cuda"), noise)[2]
    assert after.tolist() == want


@pytest.mark.parametrize("n_seq,vocab", [(1, 20000), (40, 5003), (330, 700)])
@pytest.mark.parametrize("small", [0, 22])
def test_residual_of_a_draft_that_is_the_target(dq, n_seq, vocab, small):
    """The draft's probabilities are the target's, rounded to 32 bits, but at the drafted token (rejected) and, with
    `small`, at every 20th: what is left of the others is rounding, +-2^-25 of it, and their noise is as small."""
    g = gen(100 + n_seq)
    logits = spread(g, 2 * n_seq, vocab, F32)
    draft = torch.zeros((2 * n_seq, vocab), device="cuda")
    noise = exponential(g, n_seq, vocab)
    tokens, want = [], []
    for s in range(n_seq):
        w = weights(logits[2 * s])
        p = w / w.sum()
        x = best(p)
        q = p.float()
        if small:
            noise[s] *= 2.0 ** -small
            noise[s, ::20] *= 2.0 ** small
            q[::20] *= 0.7
        q[x] = 8.0 * p[x]
        draft[2 * s + 1] = q
        tokens += [0, x]
        r = (w - w.sum() * q.double()).clamp_min(0)
        want.append(best(r / noise[s].double()))
        assert float(r.max()) > 0
    path, n_path, after = dq.verify_draft(logits, i32(tokens), torch.full((2 * n_seq,), 0.9, device="cuda"), noise,
                                          draft_probs=draft)
    assert n_path.tolist() == [1] * n_seq
    assert after.tolist() == want


@pytest.mark.parametrize("n_seq,vocab", [(1, 20000), (40, 5003), (330, 700)])
def test_nothing_left_of_the_target(dq, n_seq, vocab):
    """A draft that is nowhere below the target, by 2^-22 of it: no residual, so the largest logit."""
    g = gen(200 + n_seq)
    logits = spread(g, 2 * n_seq, vocab, F32)
    draft = torch.zeros((2 * n_seq, vocab), device="cuda")
    noise = exponential(g, n_seq, vocab) * 1e-6
    tokens, want = [], []
    for s in range(n_seq):
        w = weights(logits[2 * s])
        p = w / w.sum()
        x = int(p.topk(2).indices[1])
        q = p.float() * (1 + 2.0 ** -22)
        q[x] = 8.0 * p[x]
        assert bool((q.double() > p).all())
        draft[2 * s + 1] = q
        tokens += [0, x]
        want.append(best(p))
    path, n_path, after = dq.verify_draft(logits, i32(tokens), torch.full((2 * n_seq,), 0.9, device="cuda"), noise,
                                          draft_probs=draft)
    assert n_path.tolist() == [1] * n_seq
    assert after.tolist() == want


def test_residual_below_the_normal_range(dq):
    """All but one token's weights are around 2^-137; the draft covers that one, so the residual is theirs."""
    g, vocab, n_seq = gen(300), 3000, 3
    logits = -95.0 + randn(g, 2 * n_seq, vocab)
    logits[:, 77] = 0.0
    draft = torch.zeros((2 * n_seq, vocab), device="cuda")
    draft[:, 77], draft[:, 5] = 1.0, 1e-3
    noise = exponential(g, n_seq, vocab)
    want = []
    for s in range(n_seq):
        w = weights(logits[2 * s])
        r = (w - w.sum() * draft[2 * s + 1].double()).clamp_min(0)
        want.append(best(r / noise[s].double()))
    assert 77 not in want and 5 not in want
    path, n_path, after = dq.verify_draft(logits, i32([0, 5] * n_seq), torch.full((2 * n_seq,), 0.9, device="cuda"), noise,
                                          draft_probs=draft)
    assert n_path.tolist() == [1] * n_seq
    assert after.tolist() == want
