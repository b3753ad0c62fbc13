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


@pytest.mark.parametrize("small", [2.0 ** -127, 2.0 ** -130, 2.0 ** -149])
def test_noise_below_the_normal_range(dq, small):
    """A token of weight 2^-115 and less with the smallest noise: its ratio is as large as another's, not infinite."""
    vocab, n_seq = 1000, 24
    logits = torch.full((n_seq, vocab), -float("inf"), device="cuda")
    noise = torch.ones((n_seq, vocab), device="cuda")
    logits[:, 10], noise[:, 10] = 0.0, 2.0 ** -10
    logits[:, 900], noise[:, 900] = -80.0 - 0.25 * torch.arange(n_seq, device="cuda"), small
    want = [best(weights(r) / e.double()) for r, e in zip(logits, noise)]
    after = dq.verify_draft(logits, i32([0] * n_seq), torch.zeros(n_seq, device="cuda"), noise)[2]
    assert after.tolist() == want


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gap", [6, 12])
def test_a_child_after_a_likely_one(dq, dtype, gap):
    """A first child of probability 1 - 2^-gap is rejected; the second's random number is 2^-20 beside p / (1 - p(first))."""
    g, vocab, n_seq = gen(400 + gap), 1000, 64
    logits = randn(g, 3 * n_seq, vocab).to(dtype)
    uniform = torch.full((3 * n_seq,), 1 - 2.0 ** -24, device="cuda")
    tokens, want = [], []
    for s in range(n_seq):
        row = logits[3 * s]
        rest = torch.logsumexp(row.double(), 0)
        row[500] = float(rest) + gap * math.log(2.0)
        row[10 + s] = row[:500].float().max() + 2
        w = weights(row)
        p = w / w.sum()
        border = float(w[10 + s] / (w.sum() - w[500]))
        assert border < 0.9 and float(p[500]) < 1 - 2.0 ** -14
        u = torch.tensor(border * (1 + 2.0 ** -20 * (-1) ** s)).float()
        uniform[3 * s + 2] = u
        assert (float(u) < border) == (s % 2 == 1) and abs(float(u) / border - 1) > 2.0 ** -21
        tokens += [0, 500, 10 + s]
        want.append(2 if float(u) < border else 1)
    noise = exponential(g, n_seq, vocab)
    path, n_path, after = dq.verify_draft(logits, i32(tokens), uniform, noise, parents=i32([-1, 0, 0] * n_seq))
    assert n_path.tolist() == want
    assert path.tolist() == [[0, 2, -1] if n == 2 else [0, -1, -1] for n in want]


def test_chain_tokens_beside_their_border(dq):
    """uniform * q is 2^-23 beside p, for the second and the third node of chains."""
    g, vocab, n_seq = gen(500), 4000, 64
    logits = spread(g, 3 * n_seq, vocab, F32)
    draft = torch.softmax(spread(g, 3 * n_seq, vocab, F32), -1)
    uniform, tokens, want = torch.zeros(3 * n_seq, device="cuda"), [], []
    for s in range(n_seq):
        tokens.append(0)
        taken = []
        for j in (1, 2):
            w = weights(logits[3 * s + j - 1])
            x = int(w.topk(20).indices[(s + j) % 20])
            p = float(w[x] / w.sum())
            u = torch.tensor(0.25 + 0.5 * ((s * 7 + j) % 11) / 11).float()
            draft[3 * s + j, x] = p / float(u) * (1 + 2.0 ** -23 * (1 if s * (2 * j - 1) // 2 % 2 else -1))
            q = float(draft[3 * s + j, x])
            if float(u) * q == p:
                q = 0.0
            uniform[3 * s + j] = u
            tokens.append(x)
            taken.append(float(u) * q < p)
        want.append(1 + taken[0] + (taken[0] and taken[1]))
    assert len(set(want)) == 3
    noise = exponential(g, n_seq, vocab)
    assert dq.verify_draft(logits, i32(tokens), uniform, noise, draft_probs=draft)[1].tolist() == want


def test_rejected_mass_of_everything(dq):
    """A random number of 2 rejects whatever it is asked about: where the rejected tokens have all of the probability, the
    last child, whose weight is 0, is not accepted for a rounding of what is left."""
    g, vocab, n_seq = gen(600), 64, 2000
    logits = torch.full((8 * n_seq, vocab), -float("inf"), device="cuda")
    logits[:, 1:7] = 2 * randn(g, 8 * n_seq, 6)
    tokens = i32([0, 1, 2, 3, 4, 5, 6, 7] * n_seq)
    noise = exponential(g, n_seq, vocab)
    path, n_path, after = dq.verify_draft(logits, tokens, torch.full((8 * n_seq,), 2.0, device="cuda"), noise,
                                          parents=i32([-1] + [0] * 7).repeat(n_seq))
    assert n_path.tolist() == [1] * n_seq
    assert after.tolist() == logits[::8].argmax(1).tolist()  # nothing is left: the largest logit


def wide_trees():
    star = [-1] + [0] * 63
    breadth4 = [-1] + [(i - 1) // 4 for i in range(1, 64)]
    breadth8 = [-1] + [(i - 1) // 8 for i in range(1, 64)]
    chains = [-1] + [0] * 10 + list(range(1, 54))  # ten children, a chain below each
    return {"star": star, "breadth4": breadth4, "breadth8": breadth8, "chains": chains}


@pytest.mark.parametrize("name", ["star", "breadth4", "breadth8", "chains"])
def test_wide_trees(dq, name):
    """Nodes with many children, some of them with a sibling's token or none of the vocabulary."""
    parents, n, n_seq, vocab = wide_trees()[name], 64, 24, 3001
    g = gen(len(name))
    logits = spread(g, n * n_seq, vocab, F32)
    uniform, noise = torch.rand(n * n_seq, device="cuda", generator=g), exponential(g, n_seq, vocab)
    uniform[: n * n_seq // 2] = 0.99 + 0.0099 * uniform[: n * n_seq // 2]
    tokens, paths, after = [], [], []
    for s in range(n_seq):
        rows = logits[n * s:n * (s + 1)]
        top = rows.float().topk(40).indices.tolist()
        count, mine = [0] * n, [0]
        for i in range(1, n):
            k = count[parents[i]]
            count[parents[i]] += 1
            mine.append(-1 if k % 11 == 10 else top[parents[i]][k % 9 + k // 2 % 31])
        u = uniform[n * s:n * (s + 1)].tolist()
        cur, path = 0, [0]
        while True:
            w = weights(rows[cur])
            p, gone, step = w / w.sum(), [], None
            for j in range(cur + 1, n):
                x = mine[j]
                if parents[j] != cur or x < 0 or x in gone:
                    continue
                if u[j] * (1.0 - sum(float(p[k]) for k in gone)) < float(p[x]):
                    step = j
                    break
                gone.append(x)
            if step is None:
                break
            cur = step
            path.append(cur)
        p = p.clone()
        p[gone] = 0
        tokens += mine
        paths.append(path + [-1] * (n - len(path)))
        after.append(best(p / noise[s].double()))
    got = dq.verify_draft(logits, i32(tokens), uniform, noise, parents=i32(parents * n_seq))
    assert got[0].tolist() == paths
    assert got[2].tolist() == after


def test_tokens_after_candidates_are_distributed_as_drawn(dq):
    """20000 sequences of a root and three fixed candidates for its successor, the last of them after the second: the first
    two tokens have the target's distribution, whatever was accepted (each count within five deviations)."""
    g, vocab, n = gen(700), 8, 20000
    rows = randn(g, 4, vocab)
    p = torch.softmax(rows.double(), -1)
    uniform, noise = torch.rand(4 * n, device="cuda", generator=g), exponential(g, n, vocab)
    path, n_path, after = dq.verify_draft(rows.repeat(n, 1), i32([0, 3, 5, 6] * n), uniform, noise,
                                          parents=i32([-1, 0, 0, 2] * n))
    one, two = path[:, 1] == 1, path[:, 1] == 2
    first = torch.where(one, 3, torch.where(two, 5, after)).long()
    assert bool((n_path[~two] == 1 + one[~two].int()).all())

    def drawn(tokens, p):
        n = len(tokens)
        count = torch.bincount(tokens.long(), minlength=vocab).double()
        assert bool(((count - n * p).abs() <= 5 * torch.sqrt(n * p * (1 - p)) + 1).all())

    drawn(first, p[0])
    drawn(after[one], p[1])
    both = two & (path[:, 2] == 3)
    drawn(torch.where(both, 6, after)[two], p[2])
    drawn(after[both], p[3])
