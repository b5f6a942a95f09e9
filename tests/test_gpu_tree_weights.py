"""Attention whose weights lie far apart: one key that takes nearly all of a row's
weight and holds nothing, before many keys whose small weights make up the output, and
scores that rise along the cache.

Tolerances, per element, beside those of test_gpu_tree.py's head (scores, exponentials
and sums in 32 bits): 16-bit weights and results are rounded by u = eps/2 of the type
relative to their value.  float16's weights are taken relative to a reference that puts
the largest at 2^9 or above, so that the half step of the type's smallest numbers, 2^-25,
is at most 2^-34 of it: n keys add at most n 2^-34 max|v|, and the result's own smallest
half step 2^-25."""
import pytest
import torch

import draft_token_verification_vocab_amd as sv

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
PAGE, D = 16, 64


def attend(dt, scores, values, T, heads):
    """tree_attention of T nodes with `heads` query heads on one key head over cached
    positions of given scores (the nodes' own are -100), and the definition in 64 bits:
    all rows are alike, so (out [T, heads, D], lse, want [D], want lse, mass, high)."""
    n = scores.shape[0]
    pages = -(-(n + T) // PAGE)
    keys, pool = torch.zeros(pages * PAGE, D), torch.zeros(pages * PAGE, D)
    keys[:n, 0] = scores
    keys[n:, 0] = -100.0
    pool[:n] = values
    keys, pool = keys.to(dt), pool.to(dt)
    s, v = keys[:n, 0].double(), pool[:n].double()
    w = torch.softmax(s, 0)
    lse = torch.logsumexp(s, 0)

    def paged(x):
        return x.view(pages, 1, PAGE, D).cuda()
    q = torch.zeros(1, T, heads, D, dtype=dt)
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    got = sv.tree_attention(q.cuda(), paged(keys), paged(pool), table,
                            torch.tensor([n], dtype=torch.int32).cuda(), scale=1.0, lse=True)
    return (got[0][0].cpu().double(), got[1][0].cpu().double(), w @ v, lse, w @ v.abs(),
            v.abs().amax(0))


def check(dt, scores, values, T, heads):
    out, lse, want, want_lse, mass, high = attend(dt, scores, values, T, heads)
    n, u = scores.shape[0], torch.finfo(dt).eps / 2
    ds = (D + 8) * 2.0 ** -23 * scores.abs().max().item()
    rel = 2 * ds + 2.0 ** -21 + n * 2.0 ** -23 + 16 * 2.0 ** -22
    t = mass * rel + want.abs() * 2.0 ** -23
    if dt != F32:
        t = t + 2 * u * mass            # the weights and their sum
    if dt == F16:
        t = t + n * 2.0 ** -34 * high
    t = t + u * (want.abs() + t) + (2.0 ** -25 if dt == F16 else 0.0)
    assert torch.isfinite(out).all()
    off = (out - want).abs()
    assert (off <= t).all(), (off / t).max()
    assert ((lse - want_lse).abs() <= ds + rel + 2.0 ** -21 * (1 + want_lse.abs())).all()


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,heads", [(1, 1), (9, 8), (70, 4)])   # one and two row tiles to a wave
@pytest.mark.parametrize("n,sink", [(400, 17.5), (8000, 18.0), (40000, 15.5), (40000, 19.0)])
@pytest.mark.parametrize("at", [0.0, 0.6, 1.0])
def test_a_key_of_nearly_all_weight_that_holds_nothing(dt, T, heads, n, sink, at):
    g = torch.Generator().manual_seed(n)
    scores = torch.zeros(n)
    values = 0.5 + torch.rand(n, D, generator=g)
    where = int(at * (n - 1))
    scores[where] = sink
    values[where] = 0.0
    check(dt, scores, values, T, heads)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,heads", [(1, 1), (70, 4)])
@pytest.mark.parametrize("step", [0.0625, 4.0, 4.25, 11.0])
def test_scores_that_rise(dt, T, heads, step):
    """By a step to every 64 keys: below, about and above what the weights' reference
    lets pass (2^6, 4.16 in these scores), of the largest values."""
    g = torch.Generator().manual_seed(7)
    n = 1500
    scores = (step * (torch.arange(n) // 64)).clamp(max=200.0) - 60.0
    values = (2.0 * torch.rand(n, D, generator=g) - 1.0) * 60000.0
    check(dt, scores, values, T, heads)
