"""The README's draft-model example, run as it is printed: on the CPU over the
64-bit definitions, on the GPU over the package."""
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import draft_ref as ref

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")

# a tree may be shipped without its documents
pytestmark = pytest.mark.skipif(not os.path.exists(README), reason="README.md is not here")


def example():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "distill_loss" in b]
    assert len(found) == 1
    return found[0]


class Definitions:
    """The package's calls as the example makes them, over oracle.draft_ref."""

    @staticmethod
    def rows(t):
        return t.reshape(-1, t.shape[-1]).float().numpy()

    def row_topk(self, x, k, *, temperature=1.0):
        got = ref.row_topk(self.rows(x), k, temperature)
        lead = x.shape[:-1]
        return {"values": torch.from_numpy(got[0]).float().reshape(lead + (k,)),
                "ids": torch.from_numpy(got[1]).reshape(lead + (k,)),
                "lse": torch.from_numpy(got[2]).float().reshape(lead)}

    def both(self, x, ids, values, lse, g, temperature, keep):
        def flat(t):
            return None if t is None else t.reshape(-1).numpy()
        loss, grad = ref.distill(self.rows(x), ids.reshape(-1, ids.shape[-1]).numpy(),
                                 self.rows(values).astype(np.float64), flat(lse), temperature,
                                 flat(keep), flat(g))
        return (torch.from_numpy(loss).reshape(x.shape[:-1]),
                torch.from_numpy(grad).reshape(x.shape).to(x.dtype))

    def distill_loss(self, x, ids, values, lse, *, temperature=1.0):
        return self.both(x, ids, values, lse, None, temperature, None)[0], lse

    def distill_grad(self, x, ids, values, lse, g, *, temperature=1.0):
        return self.both(x, ids, values, lse, g, temperature, None)[1]

    def distill_step(self, x, ids, values, lse, g, *, temperature=1.0, keep=None, out=None):
        loss, grad = self.both(x, ids, values, lse, g, temperature, keep)
        return loss, grad if out is None else out.copy_(grad)

    def beam_select(self, x, scores, n, *, ended=None, eos=-1):
        got = ref.beam_select(x.float().numpy(), scores.double().numpy(), n, 1.0, ended.numpy(),
                              eos)
        return dict(zip(("scores", "parents", "tokens", "ended"), map(torch.from_numpy, got)))

    def beam_reorder(self, parents, states, *, lengths=None):
        for s in states:
            s.copy_(torch.from_numpy(ref.beam_reorder(parents.numpy(), s.numpy(), s.numpy(),
                                                      lengths.numpy())))
        return states


class Recorded:
    """Notes the arguments and results of the distillation calls."""

    def __init__(self, calls):
        self.calls, self.seen = calls, []

    def __getattr__(self, name):
        fn = getattr(self.calls, name)
        if not name.startswith("distill"):
            return fn

        def call(student, *args, **kw):
            before = student.clone()
            got = fn(student, *args, **kw)
            self.seen.append((name, before, kw.get("temperature", 1.0), kw.get("keep"), got))
            return got
        return call


def run_example(calls, dev):
    g = torch.Generator().manual_seed(3)
    B, K, W, V = 3, 2, 3, 64
    recorded = Recorded(calls)
    target = 4 * torch.randn(B, K + 1, V, generator=g)
    names = dict(
        sv=recorded, K=K, W=W, eos=1, target=target.to(dev),
        draft=(target[:, :K] + torch.randn(B, K, V, generator=g)).to(dev),
        grad_loss=torch.rand(B, K, generator=g).to(dev), weights=torch.rand(B, K, generator=g).to(dev),
        keep=torch.tensor([[1, 1], [1, 0], [0, 0]], dtype=torch.uint8, device=dev),
        logits=torch.randn(B, W, V, generator=g).to(dev),
        scores=-torch.rand(B, W, generator=g).to(dev),
        ended=torch.zeros(B, W, dtype=torch.uint8, device=dev),
        caches=[torch.randn(B, W, 2, 5, 4, generator=g).to(dev)],
        used=torch.tensor([5, 3, 0], dtype=torch.int32, device=dev))
    exec(example(), names)
    # Every loss is the divergence of the teacher's 20 likeliest tokens and one
    # bucket for its others from the student's, both at the call's temperature.
    assert [s[0] for s in recorded.seen] == ["distill_loss", "distill_grad", "distill_step"]
    for name, student, T, keep, got in recorded.seen:
        if name == "distill_grad":
            continue
        p = torch.softmax(target[:, :K].double() / T, -1)
        log_q = torch.log_softmax(student.cpu().double() / T, -1)
        top = p.topk(20, -1)
        rest = 1 - top.values.sum(-1)
        left = log_q.exp().scatter(-1, top.indices, 0.0).sum(-1)
        listed = (top.values * (top.values.log() - log_q.gather(-1, top.indices))).sum(-1)
        bucket = rest.log() - left.log()
        want = listed + rest * bucket
        # Both normalisers come from float32 sums, off by e: 64 terms whose
        # exponents (at most 7 in the mean) are off by three half steps, exp2 by one
        # step, five additions by half a step each.  The teacher's is a float32
        # below 2^5 besides, off by half a step, 2^-20.  A factor 1 + d on the
        # listed masses moves the loss by d (listed - P * bucket).
        h = 2.0 ** -24
        e = (math.log(2) * 3 * 7 + 7) * h
        tol = 2 * e + (e + 2.0 ** -20) * (listed.abs() + bucket.abs()) + want.abs() * h
        if keep is not None:
            want = want * keep.cpu()
        assert ((got[0].cpu().double() - want).abs() <= tol).all(), name


def test_example_over_the_definitions():
    run_example(Definitions(), "cpu")


@pytest.mark.gpu
def test_example():
    import draft_token_verification_vocab_amd as sv
    run_example(sv, "cuda:0")
