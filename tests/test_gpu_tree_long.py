"""Attention over caches so long that a sequence's rows are joined from more parts than
a wave has lanes, against the 64-bit definition, within test_gpu_tree.py's bounds."""
import pytest
import torch

import test_gpu_tree as tree

pytestmark = pytest.mark.gpu
BF16, F16, F32 = tree.BF16, tree.F16, tree.F32


def make(seed, dt, lengths, T, H, kv, D, page, rise=0.0):
    """A batch of chains; slots without a position hold NaN.  rise: how much larger
    keys are at a cache's end."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-(n + T) // page) for n in lengths]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lengths), max(held) + 1), -1, dtype=torch.int32)
    pools = [torch.randn(pages, kv, page, D, generator=g).to(dt) for _ in range(2)]
    used = 0
    for b, n in enumerate(lengths):
        mine = order[used:used + held[b]]
        used += held[b]
        table[b, :held[b]] = mine
        for pool in pools:
            pool[mine[-1].long(), :, (n + T - 1) % page + 1:] = float("nan")
        if rise:
            at = torch.linspace(1.0, rise, held[b])[:, None, None, None]
            pools[0][mine.long()] = (pools[0][mine.long()] * at).to(dt)
    return dict(q=torch.randn(len(lengths), T, H, D, generator=g).to(dt), keys=pools[0],
                values=pools[1], table=table,
                lengths=torch.tensor(lengths, dtype=torch.int32), parents=None, num_nodes=None)


def parts(c):
    """Workgroups that the longest sequence's tiles are dealt to, at the least."""
    B, T, H, _ = c["q"].shape
    kv = c["keys"].shape[1]
    tiles = [-(-(int(n) + T) // 128) for n in c["lengths"]]
    rows = 64 if T * H // kv <= 64 else 128
    slices = max(1, 256 // (-(-T * (H // kv) // rows) * kv))   # or twice as many
    return max(tiles) // -(-sum(tiles) // slices)


@pytest.mark.parametrize("dt,D", [(BF16, 64), (F16, 128), (F32, 64), (BF16, 256), (F32, 80)])
@pytest.mark.parametrize("rise", [0.0, 12.0])
def test_more_parts_than_lanes(dt, D, rise):
    c = make(D, dt, [70001], 2, 4, 1, D, 16, rise)
    assert parts(c) > 64
    tree.check(c, tree.call(tree.on_gpu(c), lse=True))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_several_rows_to_a_wave_of_the_join(dt):
    """One long cache among 2050 tokens of short ones."""
    g = torch.Generator().manual_seed(5)
    lengths = torch.randint(0, 60, (2051,), generator=g).tolist()
    lengths[1200] = 200000
    c = make(6, dt, lengths, 1, 4, 1, 64, 64)
    assert parts(c) > 64
    tree.check(c, tree.call(tree.on_gpu(c), lse=True))


@pytest.mark.parametrize("dt,D", [(BF16, 128), (F16, 64)])
def test_long_caches_of_many_rows(dt, D):
    c = make(7, dt, [131072, 40000, 100003], 9, 16, 1, D, 128)
    tree.check(c, tree.call(tree.on_gpu(c), lse=True))


def test_a_million_positions():
    c = make(8, BF16, [1 << 20], 1, 1, 1, 64, 1024)
    tree.check(c, tree.call(tree.on_gpu(c), lse=True))
