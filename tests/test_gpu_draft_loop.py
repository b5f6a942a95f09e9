"""The draft-model calls as they are used together: drafting by beams, verifying
the draft, recording the target's top logits and training the draft model on
them; the same calls recorded in HIP graphs and enqueued on other streams."""
import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, D = 4099, 32
S = 4104  # row stride


class BagModel:
    """Logits from the mean embedding of a history: enough of a language model
    to draft with, and its gradient is one product."""

    def __init__(self, seed, dtype=torch.float32):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.embed = torch.randn(V, D, generator=g, device=DEV)
        self.weight = torch.randn(D, S, generator=g, device=DEV)
        self.weight[:, V:] = 0
        self.dtype = dtype

    def hidden(self, history):
        return self.embed[history.long()].mean(dim=-2)

    def logits(self, history):
        return (self.hidden(history) @ self.weight).to(self.dtype).contiguous()


def draft_by_beams(model, prompt, W, K, eos):
    """K beam steps from prompts [B, P]; the histories, scores and a cache that
    holds each position's token are reordered with the beams."""
    B, P = prompt.shape
    history = prompt.new_zeros(B, W, P + K)
    history[:, :, :P] = prompt[:, None]
    cache = torch.zeros(B, W, 2, P + K, 4, dtype=torch.bfloat16, device=DEV)
    scores = torch.full((B, W), float("-inf"), device=DEV)
    scores[:, 0] = 0.0
    ended = torch.zeros(B, W, dtype=torch.uint8, device=DEV)
    for i in range(K):
        n = P + i
        logits = model.logits(history[:, :, :n])
        r = sv.beam_select(logits, scores, W, vocab=V, ended=ended, eos=eos)
        want = ref.beam_select(logits[..., :V].float().cpu().numpy(),
                               scores.double().cpu().numpy(), W, 1.0, ended.cpu().numpy(), eos)
        assert np.array_equal(r["parents"].cpu().numpy(), want[1])
        assert np.array_equal(r["tokens"].cpu().numpy(), want[2])
        used = torch.full((B,), n, dtype=torch.int32, device=DEV)
        sv.beam_reorder(r["parents"], [cache], lengths=used)
        sv.beam_reorder(r["parents"], [history], lengths=used, position_dim=2)
        history[:, :, n] = r["tokens"]
        cache[:, :, :, n] = (r["tokens"] % 97).to(torch.bfloat16)[:, :, None, None]
        scores, ended = r["scores"], r["ended"]
    # what was written to the cache followed its beam
    assert torch.equal(cache[:, :, 1, P:, 3].float(), (history[:, :, P:] % 97).float())
    return history, scores


def test_draft_verify_record_and_train():
    B, P, K, W, k = 6, 5, 4, 4, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    prompt = torch.randint(0, V, (B, P), generator=g, device=DEV, dtype=torch.int32)
    draft_model, target_model = BagModel(2), BagModel(3)
    history, scores = draft_by_beams(draft_model, prompt, W, K, eos=7)
    assert (scores[:, :1] >= scores).all()
    best = history[:, 0].contiguous()                 # the best beam is the draft
    tokens = best[:, P:].contiguous()
    steps = torch.stack([target_model.logits(best[:, :P + j]) for j in range(K + 1)], 1)
    drafts = torch.stack([draft_model.logits(best[:, :P + j]) for j in range(K)], 1)
    r = sv.verify(steps, drafts, tokens, seed=5, vocab=V, stats=True)
    # record the target's rows at the verified positions and train on them
    top = sv.row_topk(steps, k, vocab=V)
    assert torch.allclose(top["lse"], r.target_lse, rtol=1e-6, atol=1e-5)
    assert torch.equal(top["ids"][..., 0], r.target_argmax)
    keep = (torch.arange(K, device=DEV) <= r.accepted_len[:, None]).to(torch.uint8)
    ids, values = top["ids"][:, :K].contiguous(), top["values"][:, :K].contiguous()
    lse = r.target_lse[:, :K].contiguous()
    weight = torch.full((B, K), 1.0 / float(keep.sum()), device=DEV)
    loss, grad = sv.distill_step(drafts, ids, values, lse, weight, vocab=V, keep=keep)
    torch.cuda.synchronize()
    args = [t.reshape((B * K,) + t.shape[2:]).double().cpu().numpy()
            for t in (drafts[..., :V], ids, values, lse, keep, weight)]
    want_l, want_g = ref.distill(args[0], args[1].astype(np.int64), args[2], args[3], 1.0,
                                 args[4], args[5])
    assert np.allclose(loss.cpu().numpy().ravel(), want_l, rtol=1e-6, atol=1e-5)
    assert np.allclose(grad[..., :V].cpu().numpy().reshape(B * K, V), want_g, rtol=1e-4,
                       atol=1e-7 * np.abs(want_g).max())
    assert not grad[..., V:].any() and not grad[keep == 0].any()
    # one descent step along the weight's gradient: its directional derivative
    hidden = torch.stack([draft_model.hidden(best[:, :P + j]) for j in range(K)], 1)
    dw = torch.einsum("nd,ns->ds", hidden.reshape(-1, D), grad.reshape(-1, S))
    eps = 1e-3 / dw.norm()

    def total(sign):
        w = draft_model.weight.double() - sign * eps.double() * dw.double()
        x = (hidden.reshape(-1, D).double() @ w)[:, :V].cpu().numpy()
        l, _ = ref.distill(x, args[1].astype(np.int64), args[2], args[3], 1.0, args[4])
        return float((l * args[5]).sum())
    slope = (total(1) - total(-1)) / 2
    assert abs(slope + float(eps * dw.square().sum())) <= 1e-4 * abs(slope)


def inputs(seed, B=3, W=4, k=8):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)
    return dict(logits=(3 * normal(B, W, S)).to(torch.bfloat16),
                student=(3 * normal(B, W, S)).to(torch.bfloat16),
                scores=-5 - normal(B, W).abs(), cache=normal(B, W, 2, 6, 8),
                weight=normal(B, W).abs())


def calls(x, k=8):
    """Every draft-model call on one set of inputs, each feeding the next."""
    top = sv.row_topk(x["logits"], k, vocab=V)
    loss, state = sv.distill_loss(x["student"], top["ids"], top["values"], top["lse"], vocab=V)
    grad = sv.distill_grad(x["student"], top["ids"], top["values"], state, x["weight"], vocab=V)
    loss2, grad2 = sv.distill_step(x["student"], top["ids"], top["values"], None, x["weight"],
                                   vocab=V)
    sel = sv.beam_select(x["logits"], x["scores"], 4, vocab=V)
    out = torch.zeros_like(x["cache"])
    sv.beam_reorder(sel["parents"], [x["cache"]], [out])
    return [top["values"], top["ids"], top["lse"], loss, grad, loss2, grad2, sel["scores"],
            sel["parents"], sel["tokens"], sel["ended"], out]


def same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.is_floating_point() else x,
                           y.view(torch.int16) if y.is_floating_point() else y)
               for x, y in zip(a, b))


def test_recorded_in_graphs_and_replayed():
    a, b = inputs(1), inputs(2)
    eager = [[t.clone() for t in calls(x)] for x in (a, b)]
    graphs, outs, bufs = [], [], []
    for x in (a, b):  # two graphs, each with workspaces of its own
        buf = {n: t.clone() for n, t in x.items()}
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls(buf)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(buf))
        graphs.append(g)
        bufs.append(buf)
    for rep in range(4):
        for i, g in enumerate(graphs):
            src = (a, b)[(i + rep) % 2]  # new contents in place
            for n, t in bufs[i].items():
                t.copy_(src[n])
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, g in zip(streams, graphs):  # both at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        mixed = calls(a)  # eager work between the replays
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert same(mixed, eager[0])
        for i in range(2):
            assert same(outs[i], eager[(i + rep) % 2]), (rep, i)


def test_calls_on_another_stream():
    x = inputs(4)
    want = [t.clone() for t in calls(x)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = {n: t * 1 for n, t in x.items()}  # inputs made on that stream
        got = calls(late)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same(got, want)


def test_refusals_of_the_binding():
    x = inputs(6)
    top = sv.row_topk(x["logits"], 8, vocab=V)
    with pytest.raises(sv.SpecVerifyError):
        sv.row_topk(x["logits"], 129, vocab=V)
    with pytest.raises(sv.SpecVerifyError):
        sv.row_topk(x["logits"], 4, vocab=S + 1)
    with pytest.raises(TypeError):
        sv.row_topk(x["logits"].half(), 4)
    with pytest.raises(ValueError):
        sv.row_topk(x["logits"][..., :V], 4)             # not contiguous
    with pytest.raises(ValueError):
        sv.distill_loss(x["student"], top["ids"].long(), top["values"], vocab=V)
    with pytest.raises(ValueError):
        sv.distill_loss(x["student"], top["ids"], top["values"][..., :7].contiguous(), vocab=V)
    _, state = sv.distill_loss(x["student"], top["ids"], top["values"], vocab=V)
    with pytest.raises(ValueError):
        sv.distill_grad(x["student"], top["ids"], top["values"], state[:-1], vocab=V)
    with pytest.raises(ValueError):
        sv.distill_step(x["student"], top["ids"], top["values"], vocab=V,
                        out=torch.empty_like(x["student"], dtype=torch.float32))
    with pytest.raises(ValueError):
        sv.beam_select(x["logits"], x["scores"][:, :3].contiguous(), 4, vocab=V)
    with pytest.raises(sv.SpecVerifyError):
        sv.beam_select(x["logits"], x["scores"], 65, vocab=V)
    p = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        sv.beam_reorder(p, [x["cache"][:, :3]])
    with pytest.raises(ValueError):
        sv.beam_reorder(p, [x["cache"]], [x["cache"].double()])
    with pytest.raises(ValueError):
        sv.beam_reorder(p[:, :2].contiguous(), [x["cache"]])  # fewer beams, in place
    with pytest.raises(ValueError):
        sv.beam_reorder(p, [x["cache"]], lengths=p[:, 0].contiguous(), position_dim=5)
    flat = x["cache"].reshape(-1)
    one, two = flat[:48].view(3, 4, 4), flat[4:52].view(3, 4, 4)
    with pytest.raises(sv.SpecVerifyError):
        sv.beam_reorder(p, [one], [two])                 # overlapping buffers


def test_autograd_sees_what_the_calls_overwrite():
    """exp keeps its result for its backward pass: once a call has written there,
    that pass has to be refused, not to go on with other values."""
    x = inputs(8)
    top = sv.row_topk(x["logits"], 8, vocab=V)
    teacher = top["ids"], top["values"]

    def result(t):
        return t.float().clone().requires_grad_().exp()
    student = result(x["student"] / 8)
    version = student._version
    _, state = sv.distill_loss(student, *teacher, vocab=V)
    sv.distill_grad(student, *teacher, state, vocab=V)
    sv.distill_step(student, *teacher, vocab=V)
    assert student._version == version
    student.sum().backward()                         # nothing was written
    writes = [lambda t: sv.distill_grad(t, *teacher, state, vocab=V, out=t),
              lambda t: sv.distill_step(t, *teacher, vocab=V, out=t),
              lambda t: sv.beam_reorder(torch.zeros(3, 4, dtype=torch.int32, device=DEV), [t]),
              lambda t: sv.beam_reorder(torch.zeros(3, 4, dtype=torch.int32, device=DEV),
                                        [torch.zeros_like(t)], [t])]
    for write in writes:
        student = result(x["student"] / 8)
        write(student)
        with pytest.raises(RuntimeError, match="inplace"):
            student.sum().backward()
