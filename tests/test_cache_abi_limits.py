"""Host-side limits of the paged-cache calls at their ends (no GPU needed): strides
that wrap, counts past 32 bits, and memory that is given twice."""
import ctypes
import itertools
import os
import subprocess

import pytest

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
