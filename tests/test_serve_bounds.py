"""The bounds that include/fa.h gives for the cache calls, and the helpers' checks of what is no tensor (CPU only).

Refusals alone: a call that passes the checks would go on to a GPU."""

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from tests.test_norm_rope_args import APPEND, FWD_PAGED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load_library()


@pytest.mark.parametrize("kw", [
    dict(max_pages=(1 << 26) + 1), dict(page_size=65536, max_pages=(1 << 14) + 1), dict(kp_stride_p=1 << 38),
    dict(kp_stride_h=1 << 38), dict(kp_stride_r=1 << 38), dict(vp_stride_p=1 << 38), dict(vp_stride_h=1 << 38),
    dict(vp_stride_r=1 << 38), dict(vp_stride_r=56), dict(kp_stride_r=65),
])
def test_bounds_of_the_cache(kw):
    assert fa.fa_paged_append(**(APPEND | kw)) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_fwd_paged(**(FWD_PAGED | kw)) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(Hq=2049), dict(Hk=2049), dict(T=1 << 23, Hq=2048),
                                dict(T=(1 << 31) - 1, Hq=5, Hk=2)])   # T (Hq + 2 Hk) = 2^34 + 2^25, 9 (2^31 - 1)
def test_bounds_of_the_append(kw):
    assert fa.fa_paged_append(**(APPEND | kw)) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q_stride_t=1 << 31), dict(q_stride_h=1 << 31), dict(q_stride_t=56),
                                dict(q_stride_h=0), dict(T=1 << 30), dict(Hq=1 << 15, Hk=1 << 8)])
def test_bounds_of_the_attention(kw):
    assert fa.fa_fwd_paged(**(FWD_PAGED | kw)) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [[1.0, 2.0], np.zeros((2, 3, 64)), 7, torch.zeros(2, 3, 64, dtype=torch.bfloat16)])
def test_what_is_no_cuda_tensor_is_a_value_error(bad):
    for check in (fa._rows, fa._flat):
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            check(bad, "x", (2, 3, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        fa._rows(None, "x", (2, 3, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        fa._room(bad, 0)
    for call in (lambda: fa.qk_norm_rope(bad, bad), lambda: fa.paged_forward(bad, bad, bad, bad, bad, bad)):
        with pytest.raises(ValueError):
            call()
