"""The pages' bookkeeping where a table lists a page more than once in a row, and pools
that lie in one tensor, against the plain definitions; results are equal."""
import numpy as np
import pytest
import torch

import draft_token_verification_vocab_amd as sv
from oracle import cache_ref as ref
from test_gpu_cache import check_reserve, i32, paged

pytestmark = pytest.mark.gpu


def repeated_tables(rng, rows, P, N, most):
    """Rows of which many entries list the same few pages, some of them in a row, all
    counted, some held elsewhere too."""
    few = rng.permutation(N)[:max(1, most)]
    table = np.where(rng.random((rows, P)) < 0.6, few[rng.integers(0, len(few), (rows, P))], -1)
    refs = np.bincount(table[table >= 0], minlength=N)
    refs[few[rng.random(len(few)) < 0.3]] += 1
    refs[(refs == 0) & (rng.random(N) < 0.2)] = 1
    return table, refs


@pytest.mark.parametrize("rows,P,most", [(1, 2, 1), (3, 5, 2), (40, 8, 9),   # an entry to a thread
                                         (3, 400, 5), (1, 3000, 40), (600, 7, 30), (1500, 3, 4)])
@pytest.mark.parametrize("enough", [True, False])
def test_reserve_of_rows_that_list_a_page_twice(rows, P, most, enough):
    """The first of all entries keeps the page, be it of a row or within one."""
    page, N = 8, 20000 if enough else 60
    for seed in range(6):
        rng = np.random.default_rng(seed * 100 + rows)
        table, refs = repeated_tables(rng, rows, P, N, min(most, 30))
        lengths = rng.integers(0, page * min(P, 2), rows)
        new = np.minimum(rng.integers(0, P * page, rows), P * page - lengths)
        if seed == 0:
            lengths[:], new[:] = 3, P * page - 3
        got = check_reserve(table, lengths, refs, page, new)
        assert not enough or got[3] == 0


def test_reserve_of_one_page_in_two_entries():
    page = 8
    table, refs = [[5, 5, -1]], [0, 0, 0, 0, 0, 2]
    got = check_reserve(table, [3], refs, page, [13])
    assert got[0].tolist() == [[5, 0, -1]] and got[1].tolist() == [1, 0, 0, 0, 0, 1]
    # and the same where the row is too wide for a thread to an entry
    wide = [5, 5] + 1500 * [-1]
    got = check_reserve([wide], [3], [0] * 5 + [2] + [0] * 2000, page, [13 + 1400 * page])
    assert got[0][0, :3].tolist() == [5, 0, 1] and got[1][5] == 1


@pytest.mark.parametrize("axis", [0, 1, 3])
def test_pools_between_each_others_elements(axis):
    """All layers' pools in one tensor: in turn, within each page, or within each slot.
    Appending, keeping and copying move what they should and nothing else."""
    g = torch.Generator().manual_seed(axis)
    layers, N, kv, page, D, B, T = 6, 12, 2, 8, 16, 3, 5
    pools = [torch.randn(N, kv, page, D, generator=g) for _ in range(layers)]
    stacked = torch.stack(pools, dim=axis).cuda()
    views = list(stacked.unbind(axis))
    table, lengths = paged(g, B, N, 4, page, 25)
    path, counts = i32([[0, 2, 3, -1, -1], [1, 4, -1, -1, -1], [0, 1, 2, 3, 4]]), i32([3, 2, 5])
    k, v = (torch.randn(B, T, kv, D, generator=g) for _ in range(2))
    pools[2], pools[3] = ref.cache_append(k, v, pools[2], pools[3], table, lengths)
    sv.cache_append(k.cuda(), v.cuda(), views[2], views[3], table.cuda(), lengths.cuda())
    pools, new = ref.cache_keep(pools, table, lengths, path, counts)
    got = sv.cache_keep(views, table.cuda(), lengths.cuda(), path.cuda(), counts.cuda())
    assert got.tolist() == new
    copies = i32([[0, 1, 5], [2, 3, 8], [4, 5, 0]])
    pools = ref.pages_copy(pools, copies)
    sv.pages_copy(views, copies.cuda())
    assert torch.equal(stacked.cpu(), torch.stack(pools, dim=axis))
    # one of them once more, and one that reaches into the next
    for more in (views[0], stacked.flatten()[16:].as_strided(views[0].shape, views[0].stride())):
        with pytest.raises((ValueError, sv.SpecVerifyError)):
            sv.cache_keep(views + [more], table.cuda(), lengths.cuda(), path.cuda(), counts.cuda())
