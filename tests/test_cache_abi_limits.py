"""Host-side limits of the paged-cache calls at their ends (no GPU needed): strides
that wrap, counts past 32 bits, and memory that is given twice."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest
import torch

import draft_token_verification_vocab_amd as sv
from test_cache_abi import FAR, L, P, cache, host_only, pools  # noqa: F401

CSRC = os.path.join(os.path.dirname(sv.lib_path()), "csrc")

WRAPS = [-2 ** 63, -2 ** 62, -2 ** 61, -2 ** 40, -16]


@pytest.mark.parametrize("stride", WRAPS)
@pytest.mark.parametrize("dtype", [sv.DTYPE_F32, sv.DTYPE_BF16, sv.DTYPE_F16])
def test_negative_strides_are_refused_whatever_they_wrap_to(L, stride, dtype):  # noqa: F811
    for name in ("page_stride", "head_stride", "slot_stride"):
        c = cache(dtype=dtype, table_width=65, **{name: stride})
        assert L.spec_tree_attention_workspace_bytes(ctypes.byref(c), 3, 8) == 0, name
        assert L.spec_cache_append(ctypes.byref(c), P(16), P(16), 1024, 512, 64, 0, None,
                                   None) == -1, name
    c = cache(dtype=dtype, batch=0)
    for k in range(3):
        s = [1024, 512, 64]
        s[k] = stride
        assert L.spec_tree_attention(ctypes.byref(c), P(16), *s, 3, 8, None, None, 1.0,
                                     P(4 * FAR), None, None, 0, None) == -1, k
        assert L.spec_cache_append(ctypes.byref(c), P(16), P(16), *s, 3, None, None) == -1, k
    for name in ("page_stride", "head_stride", "slot_stride"):
        p = pools(**{name: stride})
        assert L.spec_pages_copy(ctypes.byref(p), None, 0, None) == -1, name


# (16-byte units of a position in a pool, sequences, pools) and pools to a launch
KEEP_LAUNCHES = [
    ((64 * 32, 32768, 1), 1),              # 262144 workgroups, far below 2^24
    ((64 * 32, 32768, 64), 32),
    ((128, 4096, 64), 64), ((128, 4096, 1000), 64), ((128, 1, 3), 3),
    ((16384 * 2048, 1, 64), 32),           # 2^31 units: past a 32-bit count
    ((16384 * 2048, 1, 63), 63),
    ((65535 * 4096, 1, 64), 8), ((65535 * 4096, 15, 64), 1), ((65535 * 4096, 16, 64), 1),
    ((65535 * 4096, 17, 64), 0), ((1, 2 ** 24 - 1, 9), 9), ((1, 2 ** 24, 9), 0)]


def test_pools_are_shared_out_to_launches_that_fit(tmp_path):
    """The library's own arithmetic, compiled for the host."""
    source = tmp_path / "launches.cpp"
    source.write_text('#include <cstdio>\n#include "sv_launch.hpp"\nint main() {\n' + "".join(
        'std::printf("%%d\\n", sv::keep_pools_per_launch(%d, %d, %d));\n' % a
        for a, _ in KEEP_LAUNCHES) + "}\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(source), "-o",
                    str(tmp_path / "launches")], check=True)
    got = subprocess.run([str(tmp_path / "launches")], check=True, capture_output=True, text=True)
    assert [int(x) for x in got.stdout.split()] == [n for _, n in KEEP_LAUNCHES]
    for (column, batch, count), n in KEEP_LAUNCHES:
        if n:
            assert column * n < 2 ** 31 and -(-column * n // 256) * batch < 2 ** 24
        if n < min(count, 64):   # twice as many do not fit
            m = 2 * n or 1
            assert column * m >= 2 ** 31 or -(-column * m // 256) * batch >= 2 ** 24


@host_only
def test_keep_takes_what_a_launch_holds(L):  # noqa: F811
    """Refused for want of a GPU, not of a grid."""
    p = pools(bases=(FAR,), heads=64, slot_bytes=512, slot_stride=512, head_stride=512 * 16,
              page_stride=512 * 16 * 64)
    a = [P(n << 32) for n in range(1, 6)]
    assert L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 32768, 4, a[4],
                             None) not in (-1, -2)
    assert L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 1 << 22, 4, a[4],
                             None) == -2


def span(n, stride, unit):
    return {sum(i * s for i, s in zip(at, stride)) + k for at in itertools.product(*map(range, n))
            for k in range(unit)}


# page, head and slot strides in 16-byte units for 3 pages, 2 heads and 8 slots of 2 units
STRIDES = [(32, 16, 2), (40, 16, 2), (32, 2, 4), (16, 48, 2), (2, 6, 12), (16, 1, 2), (15, 16, 2),
           (32, 15, 2), (31, 16, 2), (0, 16, 2), (32, 0, 2), (1, 16, 2), (32, 2, 3), (34, 17, 2)]


@host_only
@pytest.mark.parametrize("strides", STRIDES, ids=str)
def test_pools_that_are_written_have_a_place_for_every_element(L, strides):  # noqa: F811
    """An element that two pages, heads or slots share would have two writers."""
    apart = len(span((3, 2, 8), strides, 2)) == 3 * 2 * 8 * 2
    page, head, slot = strides
    p = pools(page_size=8, num_pages=3, heads=2, slot_bytes=32, page_stride=16 * page,
              head_stride=16 * head, slot_stride=16 * slot)
    c = cache(page_size=8, num_pages=3, kv_heads=2, dim=16, page_stride=8 * page,
              head_stride=8 * head, slot_stride=8 * slot)
    a = [P(n << 32) for n in range(1, 6)]
    for status in (L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 2, 4, a[4], None),
                   L.spec_pages_copy(ctypes.byref(p), a[0], 3, None),
                   L.spec_cache_append(ctypes.byref(c), a[0], a[1], 1024, 512, 64, 3, None, None)):
        assert (status not in (-1, -2)) if apart else status == -1
    # axes of one element may have any stride
    one = pools(page_size=8, num_pages=1, heads=1, slot_bytes=32, page_stride=0, head_stride=16,
                slot_stride=32)
    assert L.spec_pages_copy(ctypes.byref(one), a[0], 3, None) not in (-1, -2)


LAYOUTS = [(32, 16, 2), (64, 16, 2), (64, 32, 4), (64, 2, 8), (512, 128, 16)]


@host_only
@pytest.mark.parametrize("strides", LAYOUTS, ids=str)
def test_pools_that_share_memory_are_refused(L, strides):  # noqa: F811
    """Pools of one layout, some of them between each other's elements, against their
    elements listed."""
    page, head, slot = strides
    rng = random.Random(page)
    mine = span((3, 2, 8), strides, 2)
    a = [P(n << 32) for n in range(1, 6)]
    layout = dict(page_size=8, num_pages=3, heads=2, slot_bytes=32, page_stride=16 * page,
                  head_stride=16 * head, slot_stride=16 * slot)
    seen = set()
    # apart by every distance that matters
    for d in list(range(0, max(mine) + 3)):
        meet = any(x + d in mine for x in mine)
        seen.add(meet)
        for bases in ((FAR, FAR + 16 * d), (FAR + 16 * d, FAR)):
            p = pools(bases=bases, **layout)
            got = L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 2, 4, a[4], None)
            assert got == -1 if meet else got not in (-1, -2), d
            copy = L.spec_pages_copy(ctypes.byref(p), a[0], 3, None)
            # a pool given twice is copied to twice, alike
            assert copy == -1 if meet and d else copy not in (-1, -2), d
            c = cache(keys=bases[0], values=bases[1], page_size=8, num_pages=3, kv_heads=2, dim=16,
                      page_stride=8 * page, head_stride=8 * head, slot_stride=8 * slot)
            got = L.spec_cache_append(ctypes.byref(c), a[0], a[1], 1024, 512, 64, 3, None, None)
            assert got == -1 if meet else got not in (-1, -2), d
    assert True in seen
    # several at once, in any order
    for _ in range(300):
        at = [rng.randrange(0, 3 * max(mine)) for _ in range(rng.randint(2, 6))]
        if rng.random() < 0.5:
            at = [slot // 2 * 2 * rng.randrange(0, 64) + rng.choice((0, 0, 2)) for _ in at]
        used = [x + b for b in at for x in mine]
        p = pools(bases=[FAR + 16 * b for b in at], **layout)
        got = L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 2, 4, a[4], None)
        if len(set(used)) < len(used):
            assert got == -1, at
        else:
            assert got not in (-1, -2), at


@host_only
@pytest.mark.parametrize("axis", ["apart", "pages", "slots"])
def test_many_pools_of_one_tensor(L, axis):  # noqa: F811
    """All layers' pools in one allocation: one behind the other, or within each page
    or slot; then one of them once more."""
    n, unit = 1500, 2 * 8 * 32
    layout = dict(page_size=8, num_pages=3, heads=2, slot_bytes=32, head_stride=8 * 32, slot_stride=32)
    if axis == "apart":
        layout.update(page_stride=unit)
        bases = [FAR + 3 * unit * i for i in range(n)]
    elif axis == "pages":
        layout.update(page_stride=unit * n)
        bases = [FAR + unit * i for i in range(n)]
    else:
        layout.update(slot_stride=64 * n, head_stride=32, page_stride=8 * 64 * n)
        bases = [FAR + 64 * i for i in range(n)]
    random.Random(1).shuffle(bases)
    a = [P(m << 32) for m in range(1, 6)]
    for k in (2, 130, n):
        for extra, bad in (((), False), ((bases[0],), True), ((bases[1] + 16,), True)):
            p = pools(bases=tuple(bases[:k]) + extra, **layout)
            got = L.spec_cache_keep(ctypes.byref(p), a[0], 5, a[1], a[2], a[3], 2, 4, a[4], None)
            assert (got == -1) if bad else got not in (-1, -2), (k, extra)


def places(sizes, start=1 << 40):
    """Addresses of buffers one behind the other, with no gap."""
    at = {}
    for name, size in sizes.items():
        at[name] = start
        start += -(-size // 256) * 256
    return at


def overlapping(call, sizes, written, allowed=()):
    """call(addresses) is refused where a buffer that is written to overlaps another, by
    its first byte or its last, and only there."""
    at = places(sizes)
    assert call(at) not in (-1, -2, -3)
    for w in written:
        for other in sizes:
            if other == w or (w, other) in allowed or (other, w) in allowed:
                continue
            for move in (at[other] + sizes[other] // 16 * 16 - (sizes[other] % 16 == 0) * 16,
                         at[other] - (sizes[w] - 1) // 16 * 16):
                assert call(dict(at, **{w: move})) == -1, (w, other)


@host_only
def test_attention_writes_over_nothing(L):  # noqa: F811
    B, T, H, width = 2, 3, 8, 65
    pool = (9 * 4096 + 3 * 1024 + 15 * 64 + 64) * 2
    need = L.spec_tree_attention_workspace_bytes(ctypes.byref(cache(table_width=width)), T, H)
    sizes = dict(keys=pool, values=pool, table=B * width * 4, lengths=B * 4, q=B * T * H * 64 * 2,
                 parents=B * T * 4, nodes=B * 4, out=B * T * H * 64 * 2, lse=B * T * H * 4,
                 workspace=need)

    def call(at):
        c = cache(keys=at["keys"], values=at["values"], table=at["table"], lengths=at["lengths"],
                  table_width=width)
        return L.spec_tree_attention(ctypes.byref(c), P(at["q"]), T * H * 64, H * 64, 64, T, H,
                                     P(at["parents"]), P(at["nodes"]), 1.0, P(at["out"]),
                                     P(at["lse"]), P(at["workspace"]), need, None)
    overlapping(call, sizes, ("out", "lse", "workspace"))


@host_only
def test_append_and_keep_and_copy_write_over_nothing(L):  # noqa: F811
    B, T, width = 2, 3, 5
    pool = (9 * 4096 + 3 * 1024 + 15 * 64 + 64) * 2
    rows = (1024 + 2 * 512 + 3 * 64 + 64) * 2
    sizes = dict(keys=pool, values=pool, table=B * width * 4, lengths=B * 4, nodes=B * 4, k=rows,
                 v=rows)

    def append(at):
        c = cache(**{k: at[k] for k in ("keys", "values", "table", "lengths")})
        return L.spec_cache_append(ctypes.byref(c), P(at["k"]), P(at["v"]), 1024, 512, 64, T,
                                   P(at["nodes"]), None)
    overlapping(append, sizes, ("keys", "values"), allowed=[("keys", "values")])

    pool = 9 * 4096 + 2048 + 15 * 128 + 128
    sizes = dict(a=pool, b=pool, table=B * width * 4, lengths=B * 4, path=B * T * 4, count=B * 4,
                 new=B * 4)

    def keep(at):
        p = pools(bases=(at["a"], at["b"]))
        return L.spec_cache_keep(ctypes.byref(p), P(at["table"]), width, P(at["lengths"]),
                                 P(at["path"]), P(at["count"]), B, T, P(at["new"]), None)
    overlapping(keep, sizes, ("a", "b", "new"), allowed=[("a", "b")])

    def copy(at):
        p = pools(bases=(at["a"], at["b"]))
        return L.spec_pages_copy(ctypes.byref(p), P(at["copies"]), 7, None)
    overlapping(copy, dict(a=pool, b=pool, copies=84), ("a", "b"), allowed=[("a", "b")])


@host_only
def test_accept_writes_over_nothing_but_in_place(L):  # noqa: F811
    B, T = 3, 8
    row = B * T * 4
    sizes = dict(parents=row, tokens=row, chosen=row, nodes=B * 4, path=row, count=B * 4, emitted=row)

    def call(at):
        names = ("parents", "tokens", "chosen", "nodes")
        return L.spec_tree_accept(*[P(at[n]) for n in names], B, T, P(at["path"]), P(at["count"]),
                                  P(at["emitted"]), None)
    overlapping(call, sizes, ("path", "count", "emitted"), allowed=[("count", "nodes")])
    # a row is read as a whole before it is written
    at = places(sizes)
    for new in ("path", "emitted"):
        for old in ("parents", "tokens", "chosen"):
            assert call(dict(at, **{new: at[old]})) not in (-1, -2)
    assert call(dict(at, count=at["nodes"])) not in (-1, -2)
    assert call(dict(at, path=at["emitted"])) == -1


@host_only
def test_page_calls_write_over_nothing(L):  # noqa: F811
    R, width, N = 3, 5, 40
    sizes = dict(table=R * width * 4, refs=N * 4, lengths=R * 4)

    def release(at):
        return L.spec_pages_release(P(at["table"]), P(at["lengths"]), R, width, 16, N, P(at["refs"]),
                                    None)
    overlapping(release, sizes, ("table", "refs"))
    need = L.spec_pages_reserve_workspace_bytes(R, N)
    sizes.update(new=R * 4, copies=R * 12, missing=4, workspace=need)

    def reserve(at):
        return L.spec_pages_reserve(P(at["table"]), P(at["lengths"]), P(at["new"]), R, width, 16, N,
                                    P(at["refs"]), P(at["copies"]), P(at["missing"]),
                                    P(at["workspace"]), need, None)
    overlapping(reserve, sizes, ("table", "refs", "copies", "missing", "workspace"))
    # inputs may be one and the same
    at = places(sizes)
    assert reserve(dict(at, new=at["lengths"])) not in (-1, -2, -3)


@host_only
def test_an_empty_workspace_is_nowhere(L):  # noqa: F811
    """A table of few positions needs none, whatever it points to."""
    c = cache(keys=1 << 40, values=1 << 41)
    for at in (None, P((1 << 42) + 16), P((1 << 40) + 16), P(FAR + 16)):
        assert L.spec_tree_attention(ctypes.byref(c), P(1 << 42), 3 * 8 * 64, 8 * 64, 64, 3, 8, None,
                                     None, 1.0, P(FAR), None, at, 0, None) not in (-1, -2, -3)


@host_only
def test_scales_whose_powers_of_two_overflow_are_refused(L):  # noqa: F811
    """The kernels take scale / ln 2, which has to be finite as well."""
    c = cache(keys=1 << 40, values=1 << 41)
    for scale, fine in ((2.3e38, True), (2.4e38, False), (3.4e38, False), (1e-45, True)):
        got = L.spec_tree_attention(ctypes.byref(c), P(1 << 42), 3 * 8 * 64, 8 * 64, 64, 3, 8, None,
                                    None, scale, P(FAR), None, None, 0, None)
        assert (got not in (-1, -2, -3)) if fine else got == -1


def test_workspace_sizes_of_types_without_a_kernel():
    keys = torch.empty(4, 2, 16, 64, dtype=torch.float64)
    q = torch.empty(3, 5, 8, 64, dtype=torch.float64)
    with pytest.raises(TypeError, match="float64"):
        sv.tree_workspace_bytes(q, keys, torch.empty(3, 65, dtype=torch.int32))


def test_tiles_are_counted_in_32_bits_with_room_for_rounding(L):  # noqa: F811
    """Tiles of 128 positions are dealt out in runs rounded up, over at most 512
    workgroups: their count stays that far from 2^31."""
    def need(tiles, batch):
        c = cache(kv_heads=1, page_size=128, table_width=tiles, batch=batch)
        return L.spec_tree_attention_workspace_bytes(ctypes.byref(c), 1, 1)
    for tiles in (129, 1000, 1 << 23):
        fits = (2 ** 31 - 1 - 512) // tiles
        assert need(tiles, fits) > 0, tiles
        if fits < (2 ** 31 - 1) // tiles:
            assert need(tiles, fits + 1) == 0, tiles
