"""Failure detection of the serving kernels without faulting the GPU (needs a GB300).

As in tests/test_gpu_failure_detection.py: a test-only build of the library
(-DFA_TEST_HOOKS) withholds an arrival, so that a bounded wait (1 s) runs out.
Nothing here traps, asserts on the device or spins without a limit.
"""

import ctypes

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from tests.gpu_util import require_gpu
from tests.test_gpu_failure_detection import HOOKS_LIB
from workloads import make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    require_gpu()
    lib = ctypes.CDLL(build.build(extra_flags=["-DFA_TEST_HOOKS"], out=HOOKS_LIB))
    product = fa.load_library()
    for name in ("fa_fwd", "fa_qk_norm_rope", "fa_fwd_paged", "fa_fwd_paged_workspace_size", "fa_get_device_status"):
        getattr(lib, name).argtypes = getattr(product, name).argtypes
        getattr(lib, name).restype = getattr(product, name).restype
    for name in ("fa_test_withhold_arrival",):
        getattr(lib, name).argtypes = [ctypes.c_int]
    return lib


@pytest.mark.parametrize("order", ["timeout first", "index first"])
def test_an_index_error_does_not_hide_a_timeout(hooks, order):
    B, H, N, d = 1, 2, 256, 64
    q, k, v, _ = (t.cuda() for t in make_inputs(B, H, N, d, seed=5))
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    table, pos = fa.rope_table(8, 64), torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream().cuda_stream

    def give_up():
        assert hooks.fa_test_withhold_arrival(1) == 0
        try:
            assert hooks.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                                0.125, 1, s) == fa.FA_OK
            torch.cuda.synchronize()
        finally:
            assert hooks.fa_test_withhold_arrival(0) == 0

    def miss():
        assert hooks.fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), o.data_ptr(), v.data_ptr(), B, H, H, N, d,
                                     *q.stride()[:3], *k.stride()[:3], 0, None, None, 0, 1e-6, table.data_ptr(), 8, 64,
                                     0, pos.data_ptr(), s) == fa.FA_OK

    assert hooks.fa_get_device_status(s) == fa.FA_OK
    miss()
    assert hooks.fa_get_device_status(s) == fa.FA_ERR_DEVICE_INDEX
    for step in (give_up, miss) if order == "timeout first" else (miss, give_up):
        step()
    assert hooks.fa_get_device_status(s) == fa.FA_ERR_DEVICE_TIMEOUT
    assert hooks.fa_get_device_status(s) == fa.FA_OK
