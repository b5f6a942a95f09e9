"""Attention of chains and trees of new tokens over a paged cache, against the
64-bit definition.

Tolerances, from the arithmetic, per element.  With u = eps/2 of the type (half
a step), mass = sum of weight * |v|, size = the largest sum of |scale q k| and n
the visible keys:
  scores   products are exact or rounded once, added in 32 bits in any order, and
           scaled and shifted by the maximum: off by at most
           ds = (D + 8) 2^-23 size (the maximum's rounding is every key's alike)
  weights  2^x of the instruction within 2^-22: each weight is off by a factor
           within ds + 2^-22, numerator and denominator together twice that
  sums     n 2^-24 for the running sums and 2^-22 for each rescaling; a wave sees
           n / 128 + 1 blocks, but only a maximum that moves rescales: 16 allowed
  rounding of the weights (16-bit types) u, of the result u
lse: ds, and 2^-22 of its own value and of 1, and the sum's.
float16 weights below 2^-14 keep their absolute half step 2^-25 instead: n of
them add at most n 2^-25 max|v|."""
import itertools
import math

import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import cache_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def tolerances(dt, D, out, lse, mass, size, seen, high):
    u = torch.finfo(dt).eps / 2
    n = seen.double()
    ds = (D + 8) * 2.0 ** -23 * size
    rel = 2 * ds + 2.0 ** -21 + n * 2.0 ** -23 + 16 * 2.0 ** -22
    t = mass * rel[..., None] + out.abs() * 2.0 ** -23
    if dt != F32:
        t = t + u * mass + u * (out.abs() + t + u * mass)
    if dt == F16:
        t = t + (n[..., None] * 2.0 ** -25) * high[:, None] + 2.0 ** -25
    finite = torch.where(torch.isfinite(lse), lse.abs(), 0.0)
    return t, ds + rel + 2.0 ** -21 * (1 + finite)


def make(seed, dt, B, T, H, kv, D, page, low, high, tree=False, least=None, layout="heads",
         strided=False, spare=5, garbage=float("nan"), extra=1):
    """A paged batch; slots that hold no position, and rows that are not in use,
    are filled with garbage."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(low, high + 1, (B,), generator=g)
    nodes = None if least is None else torch.randint(least, T + 1, (B,), generator=g)
    held = [-(-(int(lengths[b]) + T) // page) for b in range(B)]
    width, pages = max(held) + extra, sum(held) + spare
    table = torch.full((B, width), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    pools = [torch.full((pages, kv, page, D), garbage, dtype=dt) for _ in range(2)]
    used = 0
    for b in range(B):
        table[b, :held[b]] = order[used:used + held[b]]
        used += held[b]
        n = T if nodes is None else int(nodes[b])
        for p in range(int(lengths[b]) + n):
            for x in pools:
                x[table[b, p // page].item(), :, p % page] = torch.randn(kv, D, generator=g).to(dt)
    q = (2.0 * torch.randn(B, T, H, D, generator=g)).to(dt)
    if nodes is not None:
        for b in range(B):
            q[b, int(nodes[b]):] = garbage
    parents = None
    if tree:
        at = torch.arange(T)
        parents = (torch.rand(B, T, generator=g) * at).long().clamp(max=(at - 1).clamp(min=0))
        parents[:, 0] = -1
        parents = parents.to(torch.int32)
    return dict(q=q, keys=pools[0], values=pools[1], table=table,
                lengths=lengths.to(torch.int32), parents=parents,
                num_nodes=None if nodes is None else nodes.to(torch.int32))


def on_gpu(c, layout="heads", strided=False):
    """The batch on the GPU: pools with heads before or behind slots or interleaved,
    queries alone or beside others."""
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    if layout == "slots":
        for k in ("keys", "values"):
            d[k] = d[k].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "both":
        two = torch.stack([d["keys"], d["values"]], dim=1)
        d["keys"], d["values"] = two[:, 0], two[:, 1]
    if strided:
        wide = torch.cat([d["q"], torch.full_like(d["q"], float("nan"))], dim=2)
        d["q"] = wide[:, :, :d["q"].shape[2]]
    return d


def call(d, **kw):
    return sv.tree_attention(d["q"], d["keys"], d["values"], d["table"], d["lengths"],
                             d["parents"], num_nodes=d["num_nodes"], **kw)


def check(c, got, scale=None):
    out, lse = (x.cpu().double() for x in got)
    want = ref.tree_attention(c["q"], c["keys"], c["values"], c["table"], c["lengths"],
                              c["parents"], c["num_nodes"], scale)
    t_out, t_lse = tolerances(c["q"].dtype, c["q"].shape[3], *want)
    empty = want[1] == float("-inf")
    assert torch.equal(lse == float("-inf"), empty)
    assert (out[empty] == 0).all()
    assert torch.isfinite(out).all()
    bad = (out - want[0]).abs() > t_out
    assert not bad.any(), ((out - want[0]).abs() / t_out.clamp(min=1e-300)).max()
    off = (lse - want[1]).abs()[~empty]
    assert (off <= t_lse[~empty]).all(), (off / t_lse[~empty]).max()


SHAPES = [
    # B, T, H, kv, D, page, low, high
    (1, 1, 1, 1, 64, 16, 0, 0),        # a single token over itself
    (1, 1, 8, 8, 128, 16, 1, 1),
    (2, 1, 4, 1, 128, 8, 31, 33),      # blocks of 32 keys, around their border
    (3, 5, 4, 2, 128, 16, 100, 140),   # 128-key tiles, around their border
    (2, 9, 8, 2, 64, 32, 250, 300),
    (3, 13, 6, 2, 80, 32, 0, 200),
    (2, 7, 5, 1, 96, 64, 0, 90),
    (1, 16, 16, 1, 128, 128, 500, 600),   # 256 rows to a key head
    (2, 33, 3, 3, 192, 16, 10, 70),
    (2, 4, 4, 2, 256, 16, 120, 130),
    (1, 3, 2, 1, 8, 8, 40, 60),
    (1, 128, 2, 1, 128, 256, 5, 300),
    (1, 65, 4, 2, 128, 1024, 1, 700),  # a page larger than the sequence
]


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("tree", [False, True])
def test_against_the_definition(dt, shape, tree):
    c = make(sum(shape), dt, *shape, tree=tree, least=0 if shape[0] > 1 else None)
    check(c, call(on_gpu(c), lse=True))


# rows of a key head: 16 to a tile, and every number of tiles that has a kernel
ROWS = [(4, 4), (9, 3), (9, 4), (12, 4), (15, 4), (9, 8), (12, 8), (13, 8), (17, 8), (40, 8)]


@pytest.mark.parametrize("dt,D", [(BF16, 128), (F16, 64), (F32, 128), (BF16, 256), (F16, 96),
                                  (F32, 72)])
@pytest.mark.parametrize("T,G", ROWS)
def test_several_tiles_to_a_workgroup(dt, D, T, G):
    """So many key heads that a workgroup walks along its keys."""
    kv = 64
    c = make(T * G, dt, 2, T, kv * G, kv, D, 16, 700, 1500, tree=T % 2 == 1, least=T - 2)
    c["keys"] = c["keys"] * 1.5
    check(c, call(on_gpu(c), lse=True))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("layout,strided", [("slots", False), ("both", True), ("heads", True)])
def test_layouts(dt, layout, strided):
    c = make(5, dt, 3, 6, 8, 4, 128, 16, 20, 200, tree=True, least=1)
    check(c, call(on_gpu(c, layout, strided), lse=True))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_long_and_short_sequences_share_the_work(dt):
    """One long cache among short ones: its tiles are cut over many workgroups,
    the others' several to a workgroup."""
    c = make(7, dt, 9, 3, 4, 2, 64, 16, 1, 60)
    long = make(8, dt, 1, 3, 4, 2, 64, 16, 9000, 9000)
    n = c["keys"].shape[0]
    w = long["table"].shape[1]
    both = {k: torch.cat([c[k], long[k]]) for k in ("q", "keys", "values", "lengths")}
    table = torch.full((10, w), -1, dtype=torch.int32)
    table[:9, :c["table"].shape[1]] = c["table"]
    table[9] = torch.where(long["table"][0] >= 0, long["table"][0] + n, -1)
    both.update(table=table, parents=None, num_nodes=None)
    order = [3, 9, 0, 1, 2, 4, 5, 6, 7, 8]
    for k in ("q", "table", "lengths"):
        both[k] = both[k][order].contiguous()
    check(both, call(on_gpu(both), lse=True))


@pytest.mark.parametrize("T,G", [(3, 2), (6, 4), (9, 4), (9, 8)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("most", [480, 900])
def test_cut_and_whole_sequences_agree(T, G, dt, most):
    """A wider table row has the same sequence cut over workgroups and joined."""
    c = make(T, dt, 3, T, 2 * G, 2, 128, 16, 0, most, tree=True, least=0)
    check(c, call(on_gpu(c), lse=True))
    c["table"] = torch.cat([c["table"], torch.full((3, 70), -1, dtype=torch.int32)], 1)
    check(c, call(on_gpu(c), lse=True))


def test_many_sequences():
    """More sequences than a workgroup has threads."""
    c = make(11, BF16, 700, 1, 2, 1, 64, 8, 0, 40, least=0)
    check(c, call(on_gpu(c), lse=True))


def test_chain_longer_than_a_tree_may_be():
    c = make(12, BF16, 2, 300, 2, 1, 64, 16, 3, 200, least=100)
    check(c, call(on_gpu(c), lse=True))


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_masked_infinities_and_nans(dt):
    """A node's key or value that a row does not see does not reach it; one that it
    sees does what the definition says: an infinite key is a score of either sign,
    so a weight of 0 (its row stays finite) or a NaN."""
    B, T, node = 1, 6, 2
    clean = make(13, dt, B, T, 4, 2, 128, 16, 45, 45, tree=True)
    clean["parents"] = torch.tensor([[-1, 0, 0, 1, 2, 3]], dtype=torch.int32)
    args = ("q", "keys", "values", "table", "lengths", "parents")
    good = ref.tree_attention(*(clean[k] for k in args))
    t_out, _ = tolerances(dt, 128, *good)
    see = torch.from_numpy(ref.ancestors([-1, 0, 0, 1, 2, 3], T))[:, node]
    p = 45 + node
    for pool, value in itertools.product(("keys", "values"), (float("inf"), float("nan"))):
        c = dict(clean)
        c[pool] = clean[pool].clone()
        c[pool][c["table"][0, p // 16].item(), :, p % 16, 3] = value
        want = ref.tree_attention(*(c[k] for k in args))
        assert not torch.isfinite(want[0][0, see]).all()
        out, lse = (x.cpu().double() for x in call(on_gpu(c), lse=True))
        assert torch.equal(torch.isfinite(out), torch.isfinite(want[0]))
        assert ((out - good[0]).abs() <= t_out)[0, ~see].all()
        assert torch.isfinite(lse[0, ~see]).all()


def test_missing_pages_are_not_there():
    """Entries of -1 and beyond the pool drop their positions, all of a row's too."""
    c = make(14, BF16, 4, 3, 4, 2, 128, 16, 100, 200)
    N = c["keys"].shape[0]
    c["table"][0, 1] = -1
    c["table"][0, 4] = N
    c["table"][1, 0] = -2 ** 31
    c["table"][2] = -1
    c["table"][3, 3] = 2 ** 31 - 1
    check(c, call(on_gpu(c), lse=True))
    # in the middle of a long walk
    c = make(15, BF16, 1, 3, 256, 128, 64, 16, 1500, 1500)
    c["table"][0, 20] = -1
    check(c, call(on_gpu(c), lse=True))


def test_lengths_beyond_the_table_and_below_zero():
    c = make(15, BF16, 4, 3, 4, 2, 64, 16, 50, 50, extra=0)
    room = c["table"].shape[1] * 16
    for pool in ("keys", "values"):
        c[pool] = torch.randn(c[pool].shape).to(BF16)
    c["lengths"] = torch.tensor([room + 5, room - 1, -3, 2 ** 31 - 1], dtype=torch.int32)
    c["num_nodes"] = torch.tensor([3, 9, 2, -4], dtype=torch.int32)
    check(c, call(on_gpu(c), lse=True))


def test_parents_that_do_not_precede_are_roots():
    c = make(16, BF16, 2, 8, 4, 2, 64, 16, 20, 60, tree=True)
    c["parents"][0] = torch.tensor([5, 1, -7, 2, 100, 4, 6, 3], dtype=torch.int32)
    check(c, call(on_gpu(c), lse=True))


def test_deep_tree():
    """A chain given as a tree of 128 nodes equals the chain, to the bit."""
    c = make(17, BF16, 2, 128, 2, 1, 64, 16, 20, 60)
    d = on_gpu(c)
    a = call(d, lse=True)
    d["parents"] = (torch.arange(128, dtype=torch.int32, device="cuda") - 1).expand(2, -1).contiguous()
    b = call(d, lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_huge_scores(dt):
    """Scores of thousands, rising along the cache: the running maximum moves."""
    c = make(18, dt, 2, 3, 2, 1, 64, 16, 400, 500)
    for b in range(2):
        for p in range(int(c["lengths"][b])):
            c["keys"][c["table"][b, p // 16].item(), :, p % 16] *= p / 40
    check(c, call(on_gpu(c), lse=True, scale=3.0), 3.0)


def test_scores_of_minus_infinity_count_as_nothing():
    c = make(19, F32, 1, 2, 1, 1, 64, 16, 10, 10)
    c["q"][:] = 1.0
    c["keys"][:] = 0.0
    c["keys"][..., 0] = float("-inf")
    out, lse = call(on_gpu(c), lse=True)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_lse_joins_two_caches():
    """Attention over two halves, joined by their lse, is attention over the whole."""
    c = make(20, F32, 1, 1, 4, 2, 64, 16, 159, 159)
    whole, lse = call(on_gpu(c), lse=True)
    d = on_gpu(c)
    d["lengths"] = torch.tensor([79], dtype=torch.int32, device="cuda")
    a, la = call(d, lse=True)
    d["table"] = d["table"][:, 5:].contiguous()
    b, lb = call(d, lse=True)
    top = torch.maximum(la, lb)
    wa, wb = (la - top).exp()[..., None], (lb - top).exp()[..., None]
    assert torch.allclose((a * wa + b * wb) / (wa + wb), whole, rtol=1e-5, atol=1e-6)
    assert torch.allclose(top + (wa + wb).log()[..., 0], lse, rtol=1e-6, atol=1e-6)


def test_offsets_beyond_32_bits():
    """Pages whose elements lie more than 2^32 bytes and 2^31 elements into the pool."""
    page, kv, D = 1024, 8, 128
    pages = 2200  # of 2 MiB: 4.6 GB, 2.3e9 elements
    c = make(21, BF16, 1, 2, 8, kv, D, page, 1500, 1500)
    d = on_gpu(c)
    far = torch.tensor([pages - 1, pages - 2], device="cuda")
    for k in ("keys", "values"):
        big = torch.empty(pages, kv, page, D, dtype=BF16, device="cuda")
        big[far] = d[k][d["table"][0, :2].long()]
        d[k] = big
    d["table"] = far.to(torch.int32)[None].contiguous()
    check(c, call(d, lse=True))


def test_slots_far_apart():
    """All pages' first slots, then their second ones: a slot's neighbour in its page lies
    half a gigabyte behind it, the furthest that 16-bit types may have."""
    page, kv, D, apart = 8, 2, 64, 1 << 28
    c = make(23, BF16, 2, 5, 4, kv, D, page, 30, 60, tree=True)
    d, want = on_gpu(c), c["keys"].shape
    for k in ("keys", "values"):
        room = torch.empty(apart * (page - 1) + want[0] * kv * D, dtype=BF16, device="cuda")
        far = room.as_strided(want, (kv * D, D, apart, 1))
        far.copy_(d[k])
        d[k] = far
    check(c, call(d, lse=True))


def test_repeats_to_the_bit_and_with_any_workspace():
    c = make(22, BF16, 5, 4, 8, 2, 128, 16, 1100, 1900, tree=True)
    d = on_gpu(c)
    a = call(d, lse=True)
    n = sv._tree_workspace_bytes(5, c["table"].shape[1], 16, 2, 128, sv.DTYPE_BF16, 4, 8)
    w = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(d["q"], float("nan"))
    b = call(d, lse=True, workspace=w, out=out)
    assert b[0] is out
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_in_graphs_that_share_a_workspace_and_on_streams():
    cs = [make(30 + i, BF16, 3, 4, 8, 2, 128, 16, 1100, 1700, tree=i == 1) for i in range(2)]
    ds = [on_gpu(c) for c in cs]
    want = [call(d, lse=True) for d in ds]
    n = max(sv._tree_workspace_bytes(3, c["table"].shape[1], 16, 2, 128, sv.DTYPE_BF16, 4, 8)
            for c in cs)
    w = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    torch.cuda.synchronize()
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(d, lse=True, workspace=w))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        call(ds[0])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            a_nan = b[0].fill_(float("nan"))
            assert a_nan.isnan().all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = call(ds[0], lse=True)
    s.synchronize()
    assert torch.equal(r[0], want[0][0]) and torch.equal(r[1], want[0][1])


def test_new_lengths_without_a_new_capture():
    """A captured call follows the lengths, tables and node counts it finds."""
    c = make(33, BF16, 3, 4, 8, 2, 128, 16, 200, 200, garbage=0.5)
    d = on_gpu(c)
    d["num_nodes"] = torch.full((3,), 4, dtype=torch.int32, device="cuda")
    call(d, lse=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(d, lse=True)
    for lengths, nodes in (([200, 3, 77], [4, 2, 0]), ([0, 128, 199], [1, 4, 3])):
        d["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))
        d["num_nodes"].copy_(torch.tensor(nodes, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c["lengths"], c["num_nodes"] = d["lengths"].cpu(), d["num_nodes"].cpu()
        check(c, got)


def test_no_sequences():
    c = make(1, BF16, 1, 2, 4, 2, 64, 16, 5, 5)
    d = on_gpu(c)
    for k in ("q", "table", "lengths"):
        d[k] = d[k][:0]
    out, lse = call(d, lse=True)
    assert out.shape == (0, 2, 4, 64) and lse.shape == (0, 2, 4)


def test_refusals():
    c = make(1, BF16, 2, 2, 4, 2, 64, 16, 5, 9, tree=True)
    d = on_gpu(c)

    def refused(error, **kw):
        e = dict(d)
        e.update({k: v for k, v in kw.items() if k in d})
        with pytest.raises(error):
            call(e, **{k: v for k, v in kw.items() if k not in d})
        torch.cuda.synchronize()
    refused(ValueError, q=d["q"].cpu())
    refused(ValueError, q=d["q"].float())
    refused(ValueError, q=d["q"][:1])
    refused(ValueError, q=d["q"][..., :32])
    refused(ValueError, q=d["q"].transpose(2, 3).contiguous().transpose(2, 3))
    refused(ValueError, values=d["values"][:, :, :, :32])
    refused(ValueError, values=d["values"].transpose(1, 2).contiguous().transpose(1, 2))
    refused(TypeError, keys=d["keys"].double(), values=d["values"].double())
    refused(ValueError, table=d["table"].long())
    refused(ValueError, lengths=d["lengths"][:1])
    refused(ValueError, parents=d["parents"][:, :1])
    refused(ValueError, num_nodes=torch.ones(3, dtype=torch.int32, device="cuda"))
    refused(ValueError, out=d["q"][:, :1].contiguous())
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
               dict(out=d["q"]), dict(q=d["q"][:, :, :3].contiguous())):
        refused(sv.SpecVerifyError, **kw)
    refused(sv.SpecVerifyError, table=torch.full((2, 100), -1, dtype=torch.int32, device="cuda"),
            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(2, 2, 4, 68, dtype=BF16, device="cuda")[..., 2:66]  # 4 bytes off
    refused(sv.SpecVerifyError, q=wide)
    c = make(1, BF16, 1, 129, 1, 1, 64, 16, 5, 9, tree=True)
    with pytest.raises(sv.SpecVerifyError):
        call(on_gpu(c))
