"""Failure detection of the serving kernels without faulting the GPU (needs a GB300).

As in tests/test_gpu_failure_detection.py: a test-only build of the library
(-DFA_TEST_HOOKS) withholds an arrival, so that a bounded wait (1 s) runs out.
Nothing here traps, asserts on the device or spins without a limit.
"""

import ctypes
import time

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from tests.gpu_util import require_gpu
from tests.test_gpu_failure_detection import HOOKS_LIB
from tests.test_gpu_paged import batch, check, reference
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
    for name in ("fa_test_withhold_arrival", "fa_test_paged"):
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


def paged_call(hooks, q_lens, kv_lens, Hq, Hk, d, hint):
    """A call of the test library: its arguments as a function, its outputs, what they should be."""
    q, pages, table, cu, lens = batch((q_lens, kv_lens, Hq, Hk, d, 32, False, True))
    ref = reference(q, pages, table, cu, lens, 0.11, True)
    table, cu, lens = table.cuda(), cu.cuda(), lens.cuda()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    room = torch.empty(hooks.fa_fwd_paged_workspace_size(d), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        o.fill_(3.0), lse.fill_(4.0), room.fill_(1)   # (of the workspace's headers, each number says "a unit to merge")
        st = hooks.fa_fwd_paged(q.data_ptr(), *(p.data_ptr() for p in pages), o.data_ptr(), lse.data_ptr(),
                                table.data_ptr(), cu.data_ptr(), lens.data_ptr(), q.shape[0], len(q_lens), Hq, Hk, d,
                                pages[0].shape[0], 32, table.shape[1], *q.stride()[:2], *pages[0].stride()[:3],
                                *pages[1].stride()[:3], 0.11, 1, hint, room.data_ptr(), room.numel(), stream)
        assert st == fa.FA_OK
        return hooks.fa_get_device_status(stream)     # synchronises, reads and clears

    return call, o, lse, ref


FORMS = [
    ([1], [9000], 4, 2, 128, 1),              # four copies, in the kernels of short chunks
    ([3] * 40, [300] * 40, 8, 8, 64, 3),      # (units that are not cut among them)
    ([1, 2], [5000, 70], 4, 2, 64, 0),        # four copies, in the others
    ([20, 9], [4000, 300], 4, 1, 128, 0),     # one query tile
    ([200, 300], [4000, 900], 2, 1, 64, 0),   # two
    ([300, 1, 40], [2500, 900, 41], 4, 2, 128, 0),
]


@pytest.mark.parametrize("form", FORMS, ids=["split", "short", "copies", "one_tile", "two_tiles", "mix"])
def test_paged_attention_gives_up_and_the_next_call_is_clean(hooks, form):
    """An arrival withheld in every CTA with work: the roles' waits run out, the merge launch behind them ends."""
    call, o, lse, ref = paged_call(hooks, *form)
    assert call() == fa.FA_OK
    check(o, lse, ref)
    assert hooks.fa_test_paged(1) == 0
    try:
        t0 = time.time()
        st = call()
        took = time.time() - t0
    finally:
        assert hooks.fa_test_paged(0) == 0
    assert st == fa.FA_ERR_DEVICE_TIMEOUT, fa.fa_status_string(st)
    assert took < 30.0
    assert call() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("form", FORMS, ids=["split", "short", "copies", "one_tile", "two_tiles", "mix"])
def test_paged_attention_that_does_not_start_merges_nothing(hooks, form):
    """CTAs that leave at once: no row is written, whatever the workspace holds."""
    call, o, lse, ref = paged_call(hooks, *form)
    assert hooks.fa_test_paged(2) == 0
    try:
        assert call() == fa.FA_ERR_INTERNAL
    finally:
        assert hooks.fa_test_paged(0) == 0
    assert bool((o == 3).all()) and bool((lse == 4).all())
    assert call() == fa.FA_OK
    check(o, lse, ref)
