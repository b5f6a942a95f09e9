"""Distillation loss and gradient on the GPU against their 64-bit definitions
and against differences, within bounds that follow from the arithmetic."""
import math

import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H = 2.0 ** -24  # half a float32 step, relative


def sum_error(V):
    """Relative error of the sum over the unlisted entries: every exponent d is
    off by three half steps of |d| (log2(e), its division by T, the fused
    product) and the terms' mean |d| is at most log2 V + 1; exp2 by one step; the
    five additions within a chunk by half a step each (beyond it the sums are
    double)."""
    return math.log(2) * 3 * H * (math.log2(max(V, 2)) + 1) + 7 * H


def bounds(x, ids, logits, lse, T, keep, grad_loss, loss, grad, dtype):
    """(loss bound [R], gradient bound [R, V])."""
    R, V = x.shape
    e = sum_error(V)
    g = np.ones(R) if grad_loss is None else np.abs(grad_loss)
    tol_l, tol_g = np.zeros(R), np.zeros((R, V))
    step = 2.0 ** -9 * 2 if dtype == "bf16" else H  # half a step of the type
    for r in range(R):
        if not np.isfinite(loss[r]):
            continue
        seen = ref.visible(x[r])
        listed = [(i, t) for i, t in zip(ids[r], logits[r]) if 0 <= i < V and t > ref.MASKED]
        if (keep is not None and not keep[r]) or not listed or not seen.any():
            continue
        at = np.array([i for i, _ in listed])
        t = np.array([v for _, v in listed], np.float64)
        t = t / T if lse is not None else (t - t.max()) / T
        norm = ref.log_sum_exp(t, np.ones(len(t), bool)) if lse is None else float(lse[r])
        P = np.exp(t - norm).sum()
        rest = max(0.0, 1.0 - P) if lse is not None else 0.0
        mass = P + rest
        z = (np.where(seen, x[r], 0.0) - x[r][seen].max()) / T
        q = np.where(seen, np.exp(z - ref.log_sum_exp(z, seen)), 0.0)
        outside = seen.copy()
        outside[at] = False
        # each logarithm of a sum carries the sum's relative error
        tol_l[r] = 2 * mass * e + abs(loss[r]) * H
        d = np.zeros(V)
        share = q * mass
        if outside.any():
            d[outside] = np.abs(z[outside] - z[outside].max()) / math.log(2)
            share[outside] += rest * np.exp(z[outside] - ref.log_sum_exp(z, outside))
        tol_g[r] = g[r] / T * share * (2 * e + math.log(2) * 4 * H * d + 6 * H)
        tol_g[r] += np.abs(grad[r]) * step + 2.4e-38
    return tol_l, tol_g


def padded(x, stride, dtype):
    t = torch.full(x.shape[:-1] + (stride,), float("nan"), dtype=DT[dtype])
    t[..., :x.shape[-1]] = torch.from_numpy(x).to(DT[dtype])
    return t


def check(x, ids, logits, lse=None, *, dtype="f32", T=1.0, keep=None, grad_loss=None,
          stride=None):
    """Loss, gradient and the fused step of one batch; returns the fused step's
    host arrays."""
    R, V = x.shape
    per = 8 if dtype == "bf16" else 4
    S = stride or -(-V // per) * per
    T = float(np.float32(T))
    student = padded(x, S, dtype)
    xs = student[:, :V].float().numpy()

    def dev(a, dt):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dt).to(DEV)
    si, sl = dev(ids, torch.int32), dev(logits, torch.float32)
    sz, sk, sg = dev(lse, torch.float32), dev(keep, torch.uint8), dev(grad_loss, torch.float32)
    sd = student.to(DEV)
    loss, state = sv.distill_loss(sd, si, sl, sz, temperature=T, vocab=V, keep=sk)
    grad = sv.distill_grad(sd, si, sl, state, sg, temperature=T, vocab=V)
    loss2, grad2 = sv.distill_step(sd, si, sl, sz, sg, temperature=T, vocab=V, keep=sk)
    place = sd.clone()
    sv.distill_grad(place, si, sl, state, sg, temperature=T, vocab=V, out=place)
    place2 = sd.clone()
    sv.distill_step(place2, si, sl, sz, sg, temperature=T, vocab=V, keep=sk, out=place2)
    alone, none = sv.distill_loss(sd, si, sl, sz, temperature=T, vocab=V, keep=sk, state=False)
    torch.cuda.synchronize()
    assert none is None

    def same(a, b):
        return torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(loss, alone) and same(grad, place) and same(grad2, place2)
    assert torch.equal(sd.cpu().view(torch.int16), student.view(torch.int16))

    f64 = [None if a is None else np.asarray(a, np.float64) for a in (logits, lse, grad_loss)]
    want_l, want_g = ref.distill(xs, ids, f64[0], f64[1], T, keep, f64[2])
    tol_l, tol_g = bounds(xs.astype(np.float64), ids, f64[0], f64[1], T, keep, f64[2], want_l,
                          want_g, dtype)
    some = np.isfinite(want_l)  # rows whose loss is infinite have a finite gradient
    for l, g in ((loss, grad), (loss2, grad2)):
        got_l, got_g = l.cpu().numpy().astype(np.float64), g.float().cpu().numpy()
        assert np.array_equal(got_l[~some], want_l[~some])
        assert (np.abs(got_l[some] - want_l[some]) <= tol_l[some]).all(), (got_l, want_l, tol_l)
        assert not got_g[:, V:].any() and np.isfinite(got_g).all()
        off = np.abs(got_g[some, :V] - want_g[some]) - tol_g[some]
        assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))
    return got_l, got_g[:, :V], xs


def batch(R, V, k, seed, T=1.0):
    rng = np.random.default_rng(seed)
    teacher = (4.0 * rng.standard_normal((R, V))).astype(np.float32)
    x = (0.8 * teacher + 2.0 * rng.standard_normal((R, V))).astype(np.float32)
    ids = np.argsort(-teacher, axis=1, kind="stable")[:, :k].astype(np.int32)
    if V < k:
        ids = np.concatenate([ids, np.full((R, k - V), -1, np.int32)], 1)
    logits = np.where(ids >= 0, np.take_along_axis(teacher, np.maximum(ids, 0), 1), -np.inf)
    z = teacher.astype(np.float64) / T
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    return x, ids, logits.astype(np.float32), lse.astype(np.float32), rng


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,k,T", [
    (1, 2, 1, 1.0), (3, 7, 3, 1.0), (2, 9, 9, 1.0), (2, 5, 8, 0.5), (4, 100, 20, 2.0),
    (5, 1025, 64, 1.0), (3, 5003, 128, 0.7), (6, 32000, 8, 1.0), (2, 50257, 50, 1.3),
    (1, 128256, 64, 1.0), (2, 300001, 17, 1.0), (2, 32768, 20, 1.0), (2, 32773, 20, 1.0),
    (1, 65536, 64, 1.0), (1, 65540, 64, 1.0), (1, 152064, 20, 0.7), (2, 163841, 20, 1.0)])
def test_loss_and_gradient(R, V, k, T, dtype, rest):
    x, ids, logits, lse, rng = batch(R, V, k, 7 * R + V + k, T)
    g = rng.random(R).astype(np.float32) * 3
    check(x, ids, logits, lse if rest else None, dtype=dtype, T=T, grad_loss=g)


# More rows than compute units take other workgroups than few rows of the same length.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,k", [(260, 5003, 8), (258, 34001, 20), (257, 70001, 64)])
def test_more_rows_than_compute_units(R, V, k, dtype):
    x, ids, logits, lse, rng = batch(R, V, k, R + V, 1.3)
    keep = (rng.random(R) < 0.9).astype(np.uint8)
    x[3] = -np.inf
    check(x, ids, logits, lse, dtype=dtype, T=1.3, grad_loss=rng.random(R).astype(np.float32),
          keep=keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_rows_and_strides(dtype):
    x, ids, logits, lse, rng = batch(9, 3001, 16, 3)
    keep = np.array([1, 0, 1, 1, 0, 0, 1, 1, 0], np.uint8)
    x[4], logits[5], ids[8] = np.nan, np.nan, 2 ** 31 - 1  # nothing of a left-out row is used
    l, g, _ = check(x, ids, logits, lse, dtype=dtype, keep=keep, stride=3048)
    assert not l[keep == 0].any() and not g[keep == 0].any() and (l[keep == 1] > 0).all()


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V", [600, 270001])
def test_lists_with_repeats_and_entries_that_are_none(V, rest):
    x, ids, logits, lse, rng = batch(6, V, 40, 11)
    ids[0, 5] = ids[0, 4]                    # one id twice
    ids[1, :] = ids[1, 0]                    # one id forty times
    ids[2, 1::2] = [-1, V, 2 ** 31 - 1, -2 ** 31] * 5
    logits[3, ::3] = -np.inf
    logits[4, 1:5] = [np.nan, -1e30, -3.4e38, 0.0]
    ids[5, 20:] = ids[5, :20]
    logits -= 1.0                            # so that repeats leave a rest
    for dtype in ("f32", "bf16"):
        check(x, ids, logits, lse if rest else None, dtype=dtype)


@pytest.mark.parametrize("rest", [True, False])
def test_empty_rows_are_left_out(rest):
    x, ids, logits, lse, rng = batch(5, 900, 12, 17)
    ids[0] = -1                              # the teacher lists nothing
    logits[1] = -np.inf
    lse[1] = -np.inf
    x[2] = -np.inf                           # the student sees nothing
    x[3] = float(torch.finfo(torch.float32).min)
    l, g, _ = check(x, ids, logits, lse if rest else None)
    assert not l[:4].any() and not g[:4].any() and l[4] > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_student_entries(dtype):
    x, ids, logits, lse, rng = batch(4, 3000, 24, 23)
    low = float(torch.finfo(DT[dtype]).min)
    for r in range(4):
        mask = rng.random(3000) < (0.2, 0.9, 0.5, 1.0)[r]
        mask[ids[r]] = False
        x[r] = np.where(mask, (-np.inf, low, np.nan, -2e30)[r], x[r])
    l, g, xs = check(x, ids, logits, lse, dtype=dtype)
    assert not g[~ref.visible(xs)].any() and np.isfinite(l).all()
    x[1, ids[1, 3]] = -np.inf                # a listed entry that the student masks
    l, g, _ = check(x, ids, logits, lse, dtype=dtype)
    assert l[1] == np.inf and np.isfinite(g).all()
    assert g[1, ids[1, 3]] < 0               # the formula's -p there


def test_a_student_sure_of_the_list():
    # rho is about e^-60, then far below the smallest float: formed as
    # 1 - (the list's share) it would be zero
    x, ids, logits, lse, rng = batch(3, 2000, 8, 29)
    x = (0.1 * x).astype(np.float32)
    for r, up in enumerate((60.0, 200.0, 3000.0)):
        x[r, ids[r]] += up
    l, g, _ = check(x, ids, logits, lse)
    assert np.isfinite(l).all() and l[2] > 100 * l[0] / 60


@pytest.mark.parametrize("rest", [True, False])
def test_gradient_against_differences(rest):
    x, ids, logits, lse, rng = batch(3, 400, 10, 31, T=1.5)
    x, z = x / 2, lse if rest else None
    _, g, _ = check(x, ids, logits, z, T=1.5)
    l64, z64 = logits.astype(np.float64), None if z is None else z.astype(np.float64)
    for seed in range(5):
        d = np.random.default_rng(seed).standard_normal(x.shape)
        h = 1e-4
        up, _ = ref.distill(x + h * d, ids, l64, z64, 1.5)
        down, _ = ref.distill(x - h * d, ids, l64, z64, 1.5)
        # central differences: h^2/6 of the third derivative (of order one
        # along a unit-variance direction), and float32 rounding of g
        assert np.allclose((up - down) / (2 * h), (g * d).sum(1), rtol=1e-5, atol=2e-6)


def test_leading_dimensions_and_no_rows():
    x, ids, logits, lse, _ = batch(6, 500, 5, 37)
    t = [torch.from_numpy(a).to(DEV) for a in (x, ids, logits, lse)]
    loss, _ = sv.distill_loss(*t)
    shaped = [a.reshape((2, 3) + a.shape[1:]) for a in t]
    loss3, state = sv.distill_loss(*shaped)
    grad3 = sv.distill_grad(*shaped[:3], state)
    assert loss3.shape == (2, 3) and grad3.shape == (2, 3, 500)
    assert torch.equal(loss3.reshape(-1), loss)
    none = [a[:0] for a in t]
    loss0, grad0 = sv.distill_step(*none)
    assert loss0.shape == (0,) and grad0.shape == (0, 500)


@pytest.mark.parametrize("T", [1.0, 1e-4])
def test_huge_logits(T):
    # |l| / T beyond 2^30: only the largest unlisted logits have a share of rho
    x, ids, logits, lse, rng = batch(3, 1000, 6, 41)
    top = [i for i in range(1000) if i not in set(ids[0])][:3]
    x[0, top[:2]] = 4e11
    x[1] = -6e11
    x[1, ids[1]] = -6e11
    x[2] *= 1e10
    l, g, _ = check(x, ids, logits, None, T=T)
    assert np.isfinite(g).all()


def test_more_rows_than_a_grid_of_row_parts():
    # 2.1e6 rows (17 GB): the rows repeat, so every one has its first copy's results
    R, n, V, S, k = 525 * 4000, 4000, 4100, 4104, 4
    g = torch.Generator(device=DEV).manual_seed(5)
    block = torch.randn(n, S, generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.randint(0, V, (n, k), generator=g, device=DEV, dtype=torch.int32)
    logits = torch.randn(n, k, generator=g, device=DEV)
    weight = torch.rand(n, generator=g, device=DEV)
    one_l, state = sv.distill_loss(block, ids, logits, vocab=V)
    one_g = sv.distill_grad(block, ids, logits, state, weight, vocab=V)
    step_l, step_g = sv.distill_step(block, ids, logits, None, weight, vocab=V)
    times = R // n
    student = block.repeat(times, 1)
    args = [t.repeat((times,) + (1,) * (t.dim() - 1)) for t in (ids, logits, weight)]
    loss, state = sv.distill_loss(student, *args[:2], vocab=V)
    assert torch.equal(loss.view(times, n), one_l.expand(times, n))
    grad = sv.distill_grad(student, *args[:2], state, args[2], vocab=V)
    for i in (0, 1, times // 2, times - 1):
        assert torch.equal(grad[i * n:(i + 1) * n].view(torch.int16), one_g.view(torch.int16))
    some = grad.view(times, -1)[:, ::997]
    assert torch.equal(some, some[:1].expand_as(some))
    loss, _ = sv.distill_step(student, *args[:2], None, args[2], vocab=V, out=grad)
    assert torch.equal(loss.view(times, n), step_l.expand(times, n))
    for i in (0, 1, times // 2, times - 1):
        assert torch.equal(grad[i * n:(i + 1) * n].view(torch.int16), step_g.view(torch.int16))
