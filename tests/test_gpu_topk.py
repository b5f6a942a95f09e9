"""spec_row_topk on the GPU against its 64-bit definition: lists exactly, the
log-normaliser within the bound that its arithmetic gives."""
import math

import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def lse_tolerance(V, lse):
    """The float32 row pass: each term's exponent d = l log2(e)/T - n is off by
    three half steps of |d| (the constant log2(e), its division by T, the fused
    product), and the terms' mean |d| is at most log2 V + 1; exp2 by one step,
    the five additions within a chunk by half a step each (beyond it the sums
    are double), the result by half a step."""
    h = 2.0 ** -24
    return (math.log(2) * 3 * h * (math.log2(max(V, 2)) + 1) + 7 * h +
            abs(lse) * h)


def rows_of(x, stride, dtype):
    t = torch.full(x.shape[:-1] + (stride,), float("nan"), dtype=DT[dtype])
    t[..., :x.shape[-1]] = torch.from_numpy(x).to(DT[dtype])
    return t


def check(x, k, dtype, T=1.0, stride=None):
    V = x.shape[-1]
    per = 8 if dtype == "bf16" else 4
    S = stride or -(-V // per) * per
    t = rows_of(x, S, dtype)
    r = sv.row_topk(t.to(DEV), k, temperature=T, vocab=V)
    torch.cuda.synchronize()
    values, ids, lse = ref.row_topk(t[..., :V].float().numpy().reshape(-1, V), k,
                                    float(np.float32(T)))
    got = {n: v.cpu().numpy().reshape((-1,) + v.shape[x.ndim - 1:]) for n, v in r.items()}
    assert np.array_equal(got["ids"], ids)
    assert np.array_equal(got["values"], values.astype(np.float32))
    for a, b in zip(got["lse"], lse):
        assert a == b or abs(a - b) <= lse_tolerance(V, b), (a, b)
    alone = sv.row_topk(t.to(DEV), k, temperature=T, vocab=V, lse=False)
    assert set(alone) == {"values", "ids"} and torch.equal(alone["ids"], r["ids"])
    assert torch.equal(alone["values"], r["values"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,k", [
    (1, 2, 1), (2, 3, 5), (3, 7, 7), (2, 8, 3), (5, 9, 128), (4, 100, 20), (3, 1000, 128),
    (2, 1025, 64), (7, 4097, 33), (5, 32000, 8), (1, 50257, 50), (300, 5003, 16),
    (1, 128256, 128), (257, 32001, 1)])
def test_random_rows(rows, V, k, dtype):
    rng = np.random.default_rng(rows * 1000003 + V + k)
    check((4.0 * rng.standard_normal((rows, V))).astype(np.float32), k, dtype)


@pytest.mark.parametrize("rows,V,dtype", [(1, 300001, "bf16"), (260, 300001, "bf16"),
                                          (258, 140001, "f32"), (2, 1 << 20, "bf16")])
def test_long_rows(rows, V, dtype):
    g = torch.Generator().manual_seed(rows + V)
    x = 4.0 * torch.randn(rows, V, generator=g)
    per = 8 if dtype == "bf16" else 4
    t = torch.zeros(rows, -(-V // per) * per, dtype=DT[dtype])
    t[:, :V] = x.to(DT[dtype])
    r = sv.row_topk(t.to(DEV), 40, vocab=V)
    torch.cuda.synchronize()
    some = [0, rows // 2, rows - 1]
    values, ids, lse = ref.row_topk(t[some, :V].float().numpy(), 40)
    assert np.array_equal(r["ids"].cpu().numpy()[some], ids)
    assert np.array_equal(r["values"].cpu().numpy()[some], values.astype(np.float32))
    for a, b in zip(r["lse"].cpu().numpy()[some], lse):
        assert abs(a - b) <= lse_tolerance(V, b)


@pytest.mark.parametrize("T", [1e-4, 0.7, 2.0, 1e4])
def test_temperatures_and_padded_strides(T):
    rng = np.random.default_rng(5)
    x = (3.0 * rng.standard_normal((2, 3, 5003))).astype(np.float32)
    check(x, 12, "bf16", T, stride=5040)
    check(x, 12, "f32", T, stride=5040)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 260])
def test_equal_values_are_listed_by_lowest_id(rows, dtype):
    rng = np.random.default_rng(rows)
    V = 20011
    flat = np.full((rows, V), 1.5, np.float32)                       # one value
    levels = rng.integers(-2, 3, (rows, V)).astype(np.float32)       # five values
    zeros = np.where(rng.random((rows, V)) < 0.5, 0.0, -0.0).astype(np.float32)
    zeros[:, ::3] = -1.0
    for x in (flat, levels, zeros):
        for k in (1, 64, 128):
            check(x, k, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70001, 9000])
def test_rows_that_collect_too_many(V, dtype):
    rng = np.random.default_rng(V)
    x = (4.0 * rng.standard_normal((8, V))).astype(np.float32)
    x[0] = np.minimum(x[0], 6.0)                     # clamped: thousands at the maximum
    x[1] = -np.sort(-x[1])                           # decreasing
    x[2] = np.sort(x[2])                             # increasing
    x[3] = np.round(x[3])                            # a few dozen values
    x[4] = np.where(rng.random(V) < 0.3, 2.0, -1e9)  # one value and a far one
    x[4, 77] = 3.0
    x[5] = np.where(np.arange(V) >= V - 1500, 1.0, -np.inf)   # equal, at the end
    x[6] = 5.0 + rng.integers(0, 3, V) * 2.0 ** -5
    x[7] = np.float32(1.0) + rng.integers(0, 40, V).astype(np.float32) * np.float32(2.0 ** -23)
    for k in (1, 13, 128):
        check(x, k, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 256])
def test_masked_entries_are_never_listed(rows, dtype):
    rng = np.random.default_rng(rows + 1)
    V, low = 30011, float(torch.finfo(DT[dtype]).min)
    x = (4.0 * rng.standard_normal((rows, V))).astype(np.float32)
    x[0] = -np.inf                                   # nothing visible
    x[1] = low
    x[2] = np.where(rng.random(V) < 0.999, np.nan, x[2])   # about 30 visible
    for r in range(3, rows):
        mask = rng.random(V) < rng.random()
        x[r] = np.where(mask, (-np.inf, low, np.nan, -2e30)[r % 4], x[r])
        if r % 5 == 0:  # visible in one contiguous stretch only
            x[r, :10000] = -np.inf
            x[r, 12500:] = low
    for k in (5, 128):
        check(x, k, dtype)


def test_peaked_row_keeps_its_normaliser():
    x = np.zeros((2, 5000), np.float32)
    x[0, 4321] = 60.0
    x[1, 17], x[1, 18] = 1e29, 3e28
    check(x, 3, "f32")


def test_many_rows_beyond_32_bit_offsets():
    # 2.1e9 elements: row offsets pass 2^31 elements and 2^32 bytes
    rows, V = 8400, 256000
    t = torch.zeros(rows, V, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for r in (0, 4200, rows - 1):
        t[r] = torch.randn(V, generator=g, device=DEV).to(torch.bfloat16)
    r = sv.row_topk(t, 5)
    torch.cuda.synchronize()
    at = [0, 4200, rows - 1]
    values, ids, _ = ref.row_topk(t[at].float().cpu().numpy(), 5)
    assert np.array_equal(r["ids"][at].cpu().numpy(), ids)
    assert np.array_equal(r["values"][at].cpu().numpy(), values.astype(np.float32))
    assert r["ids"][1].tolist() == [0, 1, 2, 3, 4]


def test_huge_logits():
    # |l| / T beyond 2^30: only the largest logits count
    x = np.full((4, 3000), -5.0, np.float32)
    x[0, [5, 2999]] = 3e12
    x[1] = -np.linspace(2e29, 9e29, 3000)
    x[2, ::7] = 1.5e9
    x[3, 100:] = -7e11
    check(x, 9, "f32")
    check(x, 9, "f32", T=1e-4)
    check(x[:, :2990], 9, "bf16", T=3.0)


@pytest.mark.parametrize("up", [1, -1])
def test_normaliser_of_a_chunk_with_a_nan_entry(up):
    """One logit at 0 and fourteen whose terms are a hair more (or less) than half
    a step of 1: added to 1 one by one, each is rounded up to a step (or lost),
    fourteen half steps in all.  The sixteenth entry of their chunk is a NaN; the
    chunk's sum has to stay within the five additions that a term goes through
    in a chunk without one."""
    h, rows, V = 2.0 ** -24, 3, 4096
    # row 0: the 16 logits that a thread of a 4096-float row takes at once
    block = np.arange(V).reshape(4, 256, 4)          # [vector][thread][entry]
    x = np.full((rows, V), -np.inf, np.float32)
    small = np.float32(-24 * math.log(2) + up * 1e-3)
    at = [block[:, 0].ravel(), block[:, 131].ravel(), np.arange(16) * 200 + 7]
    for r in range(rows):
        x[r, at[r]] = small
        x[r, at[r][0]], x[r, at[r][9]] = 0.0, np.nan
    got = sv.row_topk(torch.from_numpy(x).to(DEV), 16)
    torch.cuda.synchronize()
    _, ids, lse = ref.row_topk(x, 16)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    # the exponents: 0, and fourteen of 24 whose terms weigh 2^-24 each
    tol = math.log(2) * 3 * h * 14 * 24 * 1.01 * h + 7 * h + abs(lse) * h
    off = np.abs(got["lse"].cpu().numpy() - lse)
    assert (off <= tol).all(), off / h
