"""Host-side limits of the paged-cache calls at their ends (no GPU needed): strides
that wrap, and pools whose elements are shared."""
import ctypes

import pytest

import draft_token_verification_vocab_amd as sv
from test_cache_abi import FAR, L, P, cache, host_only, pools  # noqa: F401

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
