"""Beam selection and reordering on the GPU against their 64-bit definitions:
choices and moved bytes exactly, scores within the bound of their arithmetic."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def sum_error(V):
    """A normaliser's float sums: exponents off by three half steps of |d|
    (log2(e), its division by T, the fused product), |d| at most log2 V + 1 in
    the mean; exp2 by one step, five additions within a chunk by half a step."""
    return (np.log(2) * 3 * (np.log2(max(V, 2)) + 1) + 7) * 2.0 ** -24


def select(x, scores, n, dtype="f32", T=1.0, ended=None, eos=-1, stride=None):
    """One call against the oracle; returns its host arrays."""
    B, W, V = x.shape
    per = 8 if dtype == "bf16" else 4
    S = stride or -(-V // per) * per
    T = float(np.float32(T))
    t = torch.full((B, W, S), float("nan"), dtype=DT[dtype])
    t[..., :V] = torch.from_numpy(x).to(DT[dtype])
    e = None if ended is None else torch.from_numpy(ended).to(DEV)
    r = sv.beam_select(t.to(DEV), torch.from_numpy(scores).to(DEV), n, temperature=T, vocab=V,
                       ended=e, eos=eos)
    torch.cuda.synchronize()
    r = {k: v.cpu().numpy() for k, v in r.items()}
    want = ref.beam_select(t[..., :V].float().numpy(), scores.astype(np.float64), n, T, ended, eos)
    assert np.array_equal(r["parents"], want[1])
    assert np.array_equal(r["tokens"], want[2])
    assert np.array_equal(r["ended"], want[3])
    there = np.isfinite(want[0])
    assert np.array_equal(r["scores"][~there], want[0][~there].astype(np.float32))
    # a normaliser's float sums and half a step of the result
    tol = sum_error(V) + np.abs(want[0][there]) * 2.0 ** -24
    assert (np.abs(r["scores"][there] - want[0][there]) <= tol).all()
    return r


def beams(B, W, V, seed, scale=4.0):
    rng = np.random.default_rng(seed)
    x = (scale * rng.standard_normal((B, W, V))).astype(np.float32)
    scores = -np.sort(5.0 + 3.0 * rng.random((B, W)), axis=1).astype(np.float32)
    return x, scores, rng


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,n", [
    (1, 1, 2, 1), (2, 3, 5, 4), (3, 2, 9, 30), (1, 4, 1000, 8), (5, 5, 4099, 10),
    (2, 32, 700, 16), (3, 8, 3001, 64), (40, 8, 1500, 16), (1, 4, 32000, 8), (64, 4, 2003, 4),
    (1, 16, 50257, 32), (2, 2, 128256, 4), (260, 1, 777, 5), (2, 8, 98304, 16),
    (1, 3, 150001, 10), (8, 8, 98310, 8)])
def test_selection(B, W, V, n, dtype):
    x, scores, _ = beams(B, W, V, B + 100 * W + V + n)
    select(x, scores, n, dtype)


@pytest.mark.parametrize("V,W,n,dtype", [(300001, 2, 8, "bf16"), (1 << 20, 32, 16, "f32"),
                                        (140001, 270, 1, "f32")])
def test_rows_of_several_segments(V, W, n, dtype):
    B = 1
    if W > 32:
        B, W = W, 1
    g = torch.Generator(device=DEV).manual_seed(V)
    per = 8 if dtype == "bf16" else 4
    S = -(-V // per) * per
    t = (4 * torch.randn(B, W, S, generator=g, device=DEV)).to(DT[dtype])
    scores = -8 - 2 * torch.rand(B, W, generator=g, device=DEV)
    r = sv.beam_select(t, scores, n, vocab=V)
    lp = torch.log_softmax(t[..., :V].double(), -1) + scores.double()[..., None]
    best = torch.topk(lp.reshape(B, W * V), n)
    assert torch.equal(r["parents"], (best.indices // V).int())
    assert torch.equal(r["tokens"], (best.indices % V).int())
    assert ((r["scores"] - best.values).abs() <= sum_error(V) + best.values.abs() * 2.0 ** -24).all()


@pytest.mark.parametrize("T", [1e-4, 0.7, 3.0, 1e4])
def test_temperatures_and_strides(T):
    x, scores, _ = beams(3, 4, 2001, 5)
    if T == 1e4:  # nearly flat rows: logits far apart, so that scores differ
        x *= 1e4
    for dtype in ("bf16", "f32"):
        select(x, scores, 8, dtype, T, stride=2048)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ended_beams_and_beams_that_take_no_part(dtype):
    x, scores, rng = beams(12, 4, 900, 9)
    ended = (rng.random((12, 4)) < 0.4).astype(np.uint8)
    ended[0], ended[1] = 1, 0
    scores[2, 1:] = -np.inf                    # a first step
    scores[3] = -np.inf                        # nothing left
    scores[4, 0] = np.nan
    x[:, :, 7] += 9.0                          # eos among the best
    x[2, 1:] = np.nan                          # logits that are not read
    x[5][ended[5] != 0] = np.nan
    r = select(x, scores, 9, dtype, ended=ended, eos=7)
    assert (r["parents"][3] == -1).all() and (r["ended"][0, :4] == 1).all()
    assert (r["tokens"] == 7).sum() > 12
    assert (r["parents"][2][:9] <= 0).all() or ended[2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_that_leave_little_or_nothing(dtype):
    x, scores, rng = beams(6, 3, 1200, 13)
    low = float(torch.finfo(DT[dtype]).min)
    x[0] = -np.inf
    x[1, 0], x[1, 1] = low, np.nan             # one beam left
    x[2, :, 4:] = -np.inf                      # 12 continuations in all
    x[3, 0, 1:] = -np.inf                      # one continuation: probability 1
    x[4] = np.where(rng.random((3, 1200)) < 0.9, -2e30, x[4])
    r = select(x, scores, 16, dtype)
    assert (r["parents"][0] == -1).all() and (r["parents"][1] == 2).all()
    assert (r["parents"][2][12:] == -1).all() and (r["parents"][2][:12] >= 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_scores(dtype):
    x = np.zeros((3, 4, 513), np.float32)      # all continuations equal
    scores = np.full((3, 4), -2.0, np.float32)
    x[1] = np.random.default_rng(1).integers(0, 3, (1, 513)).astype(np.float32)  # equal beams
    scores[2, 2] = -1.0
    r = select(x, scores, 20, dtype)
    assert (r["parents"][0] == 0).all() and r["tokens"][0].tolist() == list(range(20))
    assert (r["parents"][2] == 2).all()


@pytest.mark.parametrize("V,B", [(4000, 48), (40000, 48), (100000, 12)])
def test_near_ties_are_decided_by_the_exact_scores(V, B):
    """Beams whose rows hold the same logits in another order, but for one that
    moves the normaliser by 1e-9 to 1e-6: float sums would order them at
    random, the gaps in double are a million times a double sum's error."""
    W = 4
    rng = np.random.default_rng(V)
    x = np.empty((B, W, V), np.float32)
    for b in range(B):
        base = rng.standard_normal(V).astype(np.float32)
        total = np.exp(base.astype(np.float64)).sum()
        for w in range(W):
            row = base.copy()
            gap = 10.0 ** rng.uniform(-9, -6) * (w + 1)
            # one entry's weight grows by gap * total
            i = int(rng.integers(V))
            row[i] = np.log(np.exp(np.float64(row[i])) + gap * total)
            x[b, w] = row[rng.permutation(V)]
    top = x.max(axis=2, keepdims=True)
    x = np.where(x == top, np.float32(6.0), x)  # equal largest logits
    scores = np.full((B, W), -3.0, np.float32)
    r = select(x, scores, 6)
    assert len(np.unique(r["parents"][:, 0])) == W


@pytest.mark.parametrize("T", [1.0, 1e-4])
def test_huge_logits(T):
    # l / T beyond a double's whole numbers: differences are formed first
    x, scores, rng = beams(3, 4, 100001, 15)
    x[:, 1:] += 7e11
    x[0, 2] *= 1e20
    x[1, 3] -= 3e12
    for V in (900, 100001):
        select(x[..., :V], scores, 6, T=T)
        select(x[..., :V], scores, 6, "bf16", T=T)


def test_workspace_is_reused_and_calls_agree():
    x, scores, _ = beams(8, 4, 5003, 21)
    t = torch.zeros(8, 4, 5004)
    t[..., :5003] = torch.from_numpy(x)
    t, s = t.to(DEV), torch.from_numpy(scores).to(DEV)
    n = sv.load().spec_beam_workspace_bytes(8, 4, 5003, sv.DTYPE_F32, 8)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    a = sv.beam_select(t, s, 8, vocab=5003)
    for _ in range(2):
        b = sv.beam_select(t, s, 8, vocab=5003, workspace=ws)
        assert all(torch.equal(a[k], b[k]) for k in a)
    with pytest.raises(sv.SpecVerifyError):
        sv.beam_select(t, s, 8, vocab=5003, workspace=ws[:n - 256])


# ---------------------------------------------------------------------------
# Reordering
# ---------------------------------------------------------------------------
def reorder_check(parents, shape, dtype, lengths=None, n=None, position_dim=3, count=2):
    B, W = shape[:2]
    n = n or W
    g = torch.Generator().manual_seed(sum(shape))
    if dtype.is_floating_point:
        src = [torch.randn(shape, generator=g).to(dtype) for _ in range(count)]
    else:
        src = [torch.randint(0, 127, shape, generator=g).to(dtype) for _ in range(count)]
    dst = [torch.full((B, n) + tuple(shape[2:]), 5).to(dtype) for _ in range(count)]
    p = torch.tensor(parents, dtype=torch.int32)
    le = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)

    def want(s, d):
        s5, d5 = s, d
        if le is None:
            s5, d5 = s.reshape(B, W, 1, -1), d.reshape(B, n, 1, -1)
        else:
            lead = int(np.prod(shape[2:position_dim]))
            s5 = s.reshape((B, W, lead) + tuple(shape[position_dim:]))
            d5 = d.reshape((B, n, lead) + tuple(shape[position_dim:]))
        to = torch.float64 if dtype.is_floating_point else torch.int64
        out = ref.beam_reorder(p.numpy(), s5.to(to).numpy(), d5.to(to).numpy(), lengths)
        return torch.from_numpy(out).reshape(d.shape).to(dtype)
    gp, gl = p.to(DEV), None if le is None else le.to(DEV)
    gs, gd = [s.to(DEV) for s in src], [d.to(DEV) for d in dst]
    out = sv.beam_reorder(gp, gs, gd, lengths=gl, position_dim=position_dim)
    assert all(a is b for a, b in zip(out, gd))
    for s, d, a, b in zip(src, dst, gs, gd):
        assert torch.equal(b.cpu(), want(s, d))
        assert torch.equal(a.cpu(), s)
    if n == W:
        sv.beam_reorder(gp, gs, lengths=gl, position_dim=position_dim)
        for s, a in zip(src, gs):
            assert torch.equal(a.cpu(), want(s, s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int32, torch.uint8])
@pytest.mark.parametrize("W", [1, 2, 4, 7, 8, 9, 16, 17, 32])
def test_reorder(W, dtype):
    rng = np.random.default_rng(W)
    parents = rng.integers(0, W, (3, W))
    parents[1] = np.roll(np.arange(W), 1)      # a cycle
    if W > 1:
        parents[2, 0], parents[2, 1] = -1, W   # rows that stay
    reorder_check(parents, (3, W, 2, 9, 8), dtype, lengths=[0, 9, 5])
    reorder_check(parents, (3, W, 2, 9, 5), dtype, lengths=[100, -3, 1])
    reorder_check(parents, (3, W, 37), dtype)


def test_reorder_to_more_and_fewer_beams():
    reorder_check([[0] * 6, [0] * 6], (2, 1, 2, 40, 16), torch.bfloat16, lengths=[40, 7], n=6)
    reorder_check([[3, 1], [2, 2]], (2, 4, 33, 7), torch.float32, n=2)
    reorder_check(np.arange(64).reshape(1, 64) % 32, (1, 32, 3, 5, 4), torch.int32, n=64)


def test_reorder_other_position_dimensions_and_many_states():
    reorder_check([[1, 0]], (1, 2, 6, 3), torch.float32, lengths=[4], position_dim=2)
    reorder_check([[1, 1], [0, 0]], (2, 2, 2, 3, 7, 4), torch.bfloat16, lengths=[3, 7],
                  position_dim=4)
    reorder_check([[1, 0, 0]], (1, 3, 2, 50, 8), torch.bfloat16, lengths=[33], count=70)


def test_reorder_odd_addresses_and_empty_states():
    p = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    raw = torch.arange(2 * 333 + 1, device=DEV).to(torch.uint8)
    s = raw[1:].view(1, 2, 333)                # one byte past an allocation's start
    out = torch.zeros(1, 2, 333, dtype=torch.uint8, device=DEV)
    sv.beam_reorder(p, [s], [out])
    assert torch.equal(out, s.flip(1))
    e = torch.zeros(1, 2, 4, 0, 8, device=DEV)
    assert sv.beam_reorder(p, [e], lengths=torch.tensor([3], dtype=torch.int32, device=DEV))
    assert sv.beam_reorder(p, []) == []
    assert sv.beam_reorder(p[:0], [torch.zeros(0, 2, 5, device=DEV)])


def test_reorder_large_state_in_place():
    # beams of 1.2e9 bytes: offsets pass 2^32
    s = torch.empty(1, 4, 2, 600_000_016, dtype=torch.uint8, device=DEV)
    for w in range(4):
        s[0, w] = w + 1
    s[0, :, 1, -1] = torch.tensor([11, 12, 13, 14], dtype=torch.uint8, device=DEV)
    p = torch.tensor([[3, 0, 0, 2]], dtype=torch.int32, device=DEV)
    sv.beam_reorder(p, [s])
    for w, v in enumerate((4, 1, 1, 3)):
        assert s[0, w, 1, -1].item() == v + 10
        assert s[0, w, 0].min().item() == v and s[0, w, 1, :-1].max().item() == v


@pytest.mark.parametrize("V,T", [(5003, 0.7), (98317, 1.0), (200003, 1.6)])
def test_near_ties_of_rows_with_masked_logits(V, T):
    """As above, a third of each row masked in three ways: what the exact sums
    count for masked logits has to stay below any gap."""
    W = 3
    rng = np.random.default_rng(V + 1)
    base = rng.standard_normal(V).astype(np.float32)
    base[: V // 3] = np.resize(np.float32([-np.inf, np.nan, -2e30]), V // 3)
    base[-1] = 6.0
    total = np.exp(base[V // 3:].astype(np.float64) / T).sum()
    x = np.empty((1, W, V), np.float32)
    for w in range(W):
        row = base.copy()
        i = int(rng.integers(V // 3, V - 1))
        row[i] = T * np.log(np.exp(np.float64(row[i]) / T) + 1e-7 * (w + 1) * total)
        x[0, w] = row[rng.permutation(V)]
    for order in ([0, 1, 2], [2, 0, 1]):
        r = select(np.ascontiguousarray(x[:, order]), np.full((1, W), -3.0, np.float32), 5, T=T)
        # the lightest row's maximum comes first
        assert list(r["parents"][0, :W]) == list(np.argsort(order))


@pytest.mark.parametrize("with_lengths", [False, True])
@pytest.mark.parametrize("W", [3, 12, 32])
def test_reorder_states_of_different_units_in_one_call(W, with_lengths):
    # caches in 16-byte units, histories in 4-byte ones, flags in single bytes,
    # more than one launch of them, alternating
    rng = np.random.default_rng(W)
    parents = rng.integers(-1, W + 1, (2, W))
    lengths = [11, 4] if with_lengths else None
    g = torch.Generator().manual_seed(W)
    shapes = [((2, W, 2, 13, 8), torch.bfloat16), ((2, W, 1, 13, 1), torch.int32),
              ((2, W, 3, 13, 3), torch.uint8), ((2, W, 1, 13, 5), torch.bfloat16)]
    src = [torch.randint(0, 127, shape, generator=g).to(dt)
           for i in range(18) for shape, dt in shapes[i % 2:] + shapes[:i % 2]]
    dst = [torch.full_like(s, 5) for s in src]

    def want(s, d):
        to = torch.float64 if s.is_floating_point() else torch.int64
        at = s if with_lengths else s.reshape(2, W, 1, 1, -1)
        out = ref.beam_reorder(parents, at.to(to).numpy(),
                               d.to(to).reshape(at.shape).numpy(), lengths)
        return torch.from_numpy(out).reshape(s.shape).to(s.dtype)
    p = torch.tensor(parents, dtype=torch.int32, device=DEV)
    le = torch.tensor(lengths, dtype=torch.int32, device=DEV) if with_lengths else None
    gs, gd = [s.to(DEV) for s in src], [d.to(DEV) for d in dst]
    sv.beam_reorder(p, gs, gd, lengths=le)
    for s, d, a, b in zip(src, dst, gs, gd):
        assert torch.equal(b.cpu(), want(s, d)) and torch.equal(a.cpu(), s)
    # some in place, the others to buffers of their own
    outs = [s if i % 3 else torch.full_like(s, 5) for i, s in enumerate(gs)]
    sv.beam_reorder(p, gs, outs, lengths=le)
    for i, (s, b) in enumerate(zip(src, outs)):
        assert torch.equal(b.cpu(), want(s, s if i % 3 else torch.full_like(s, 5)))


@pytest.mark.parametrize("W", [2, 8, 9, 16])
def test_reorder_large_states_of_different_units_in_one_call(W):
    # enough work for a launch per unit; bytes are checked on the GPU
    g = torch.Generator(device=DEV).manual_seed(W)
    p = torch.randint(0, W, (3, W), generator=g, device=DEV, dtype=torch.int32)
    shapes = [((3, W, 2, 4001, 64), torch.bfloat16), ((3, W, 1, 4001, 1), torch.int32),
              ((3, W, 1, 4001, 3), torch.uint8), ((3, W, 4, 4001, 16), torch.float32)]
    src = [torch.randint(0, 127, shape, generator=g, device=DEV).to(dt) for shape, dt in shapes]
    lengths = torch.tensor([4001, 0, 2777], dtype=torch.int32, device=DEV)
    used = torch.arange(4001, device=DEV) < lengths[:, None]
    for count in (2, 3, 4):
        outs = [torch.full_like(s, 5) for s in src[:count]]
        sv.beam_reorder(p, src[:count], outs, lengths=lengths)
        place = [s.clone() for s in src[:count]]
        sv.beam_reorder(p, place, lengths=lengths)
        for s, o, q in zip(src, outs, place):
            moved = s[torch.arange(3, device=DEV)[:, None], p.long()]
            at = used[:, None, None, :, None]
            assert torch.equal(o, torch.where(at, moved, torch.full_like(s, 5)))
            assert torch.equal(q, torch.where(at, moved, s))


@pytest.mark.parametrize("shape", [(1, 2, 2, (1 << 30) + 8), (1, 2, (1 << 31) + 48),
                                   (1, 2, 3, 715827883)])
def test_reorder_beams_of_more_than_two_gib(shape):
    # without lengths a beam is one run of bytes, here more than a position holds
    # (2^31 + 16 and 2^31 + 48; 2^31 + 1, which has no factor of 16 or 4)
    s = torch.zeros(shape, dtype=torch.uint8, device=DEV)
    flat = s.view(2, -1)
    ends = [0, 1, 2 ** 30 + 7, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, flat.shape[1] - 1]
    for w in range(2):
        flat[w] = w + 1
        flat[w, ends] = torch.arange(7, dtype=torch.uint8, device=DEV) + 10 * (w + 1)
    p = torch.tensor([[1, 1]], dtype=torch.int32, device=DEV)
    out = torch.zeros_like(s)
    sv.beam_reorder(p, [s], [out])
    assert torch.equal(out.view(2, -1)[0], flat[1]) and torch.equal(out.view(2, -1)[1], flat[1])
    sv.beam_reorder(p, [s])
    assert torch.equal(flat[0], out.view(2, -1)[0]) and torch.equal(flat[1], out.view(2, -1)[1])


def hair_apart(j, ahead, parts):
    """Two rows of float32 logits and their beams' scores, the second beam's best
    continuation ahead of the first's by `ahead` (beyond a double's digits).
    Sixteen of the first row's terms lie halfway between two powers of
    2^(1/parts), the second row's on one; three small logits of the second set the distance."""
    with localcontext() as ctx:
        ctx.prec = 60

        def total(x):
            return sum(Decimal(float(v)).exp() for v in x)
        step = np.log(2.0) / parts
        k = -round(1.0 / step) - j
        a = [np.float32(0)] + [np.float32((k + 0.5) * step)] * 16
        b = [np.float32(0)] + [np.float32(k * step)] * 16
        want = (total(b) / total(a)).ln() + ahead
        score = np.nextafter(np.float32(want), np.float32(1))
        for _ in range(4):
            more = total(a) * (Decimal(float(score)) - ahead).exp() - total(b)
            if more < Decimal("1e-30"):
                break
            v = np.float32(more.ln())
            b.append(v if Decimal(float(v)).exp() <= more else np.nextafter(v, np.float32(-99)))
        gap = Decimal(float(score)) - (total(b) / total(a)).ln()
        assert abs(gap - ahead) < ahead / 1000
    return a, b, score


@pytest.mark.parametrize("parts", [32, 64])
def test_beams_a_hair_apart_are_decided_by_sums_good_to_a_double(parts):
    """1e-15 apart, nine half steps of a double near 1: the terms, their sum and
    its logarithm are rounded by one to four of them (each step of the double
    arithmetic emulated exactly); a term off by 2e-15 would tell."""
    n = 12
    x = np.full((n, 2, 128), -np.inf, np.float32)
    scores = np.zeros((n, 2), np.float32)
    for j in range(n):
        first, second, scores[j, 1] = hair_apart(j, Decimal("1e-15"), parts)
        for w, row in enumerate((first, second)):
            x[j, w, 4 * np.arange(len(row))] = row
    for flip in (False, True):
        order = [1, 0] if flip else [0, 1]
        r = sv.beam_select(torch.from_numpy(np.ascontiguousarray(x[:, order])).to(DEV),
                           torch.from_numpy(np.ascontiguousarray(scores[:, order])).to(DEV), 2)
        torch.cuda.synchronize()
        assert r["parents"][:, 0].tolist() == [0 if flip else 1] * n
        assert r["parents"][:, 1].tolist() == [1 if flip else 0] * n


# Rows that the plan cuts, unlike most above: the workspace holds a list and a
# normaliser per segment.
@pytest.mark.parametrize("B,W,V,n,dtype", [(1, 4, 1 << 20, 8, "f32"), (15, 4, 140001, 1, "f32"),
                                           (1, 2, 300001, 8, "bf16"), (2, 32, 100001, 4, "bf16"),
                                           (1, 1, 1 << 20, 64, "bf16"), (3, 5, 98309, 20, "bf16")])
def test_rows_that_are_cut_into_segments(B, W, V, n, dtype):
    code = sv.DTYPE_BF16 if dtype == "bf16" else sv.DTYPE_F32
    whole = sv.load().spec_beam_workspace_bytes(B, W, 2, code, n)
    assert sv.load().spec_beam_workspace_bytes(B, W, V, code, n) > 2 * whole - 512
    g = torch.Generator(device=DEV).manual_seed(V + W)
    per = 8 if dtype == "bf16" else 4
    S = -(-V // per) * per
    t = (4 * torch.randn(B, W, S, generator=g, device=DEV)).to(DT[dtype])
    t[:, W // 2, : V // 2] = float("-inf")           # segments with nothing visible
    scores = -8 - 2 * torch.rand(B, W, generator=g, device=DEV)
    r = sv.beam_select(t, scores, n, vocab=V)
    lp = torch.log_softmax(t[..., :V].double(), -1) + scores.double()[..., None]
    lp = lp.reshape(B, W * V)
    # equal logits of a row: the lowest token first
    best = torch.sort(lp, dim=-1, descending=True, stable=True)
    values, at = best.values[:, :n], best.indices[:, :n]
    assert torch.equal(r["parents"], (at // V).int())
    assert torch.equal(r["tokens"], (at % V).int())
    assert ((r["scores"] - values).abs() <= sum_error(V) + values.abs() * 2.0 ** -24).all()
