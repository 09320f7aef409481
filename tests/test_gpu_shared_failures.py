"""Failure detection of the attention over shared keys without faulting the GPU (needs a GB300).

As in tests/test_gpu_serve_failures.py: a test-only build withholds an arrival, so that bounded waits (1 s) run out;
the launches behind end, say so, and the next call is clean."""

import ctypes
import time

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from tests.gpu_util import require_gpu
from tests.test_gpu_failure_detection import HOOKS_LIB
from tests.test_gpu_paged import check, reference
from tests.test_gpu_paged_shared import SHAPES, batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    require_gpu()
    lib = ctypes.CDLL(build.build(extra_flags=["-DFA_TEST_HOOKS"], out=HOOKS_LIB))
    product = fa.load_library()
    for name in ("fa_fwd_paged_shared", "fa_fwd_paged_shared_workspace_size", "fa_get_device_status"):
        getattr(lib, name).argtypes = getattr(product, name).argtypes
        getattr(lib, name).restype = getattr(product, name).restype
    for name in ("fa_test_paged", "fa_test_rows"):
        getattr(lib, name).argtypes = [ctypes.c_int]
    return lib


def shared_call(hooks, shape, d):
    groups, Hq, Hk = shape
    q, pages, table, cu, lens, starts, prefix = x = batch(groups, Hq, Hk, d, 32, False)
    ref = reference(*x[:5], 0.11, True)
    t, c, n, g, pre = (v.cuda() for v in (table, cu, lens, starts, prefix))
    T, S, NG = q.shape[0], len(lens), len(prefix)
    o = torch.full_like(q, 3.0)
    lse = torch.full((T, Hq), 4.0, device="cuda")
    room = torch.full((hooks.fa_fwd_paged_shared_workspace_size(T, S, NG, Hq, d),), 255, dtype=torch.uint8,
                      device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        st = hooks.fa_fwd_paged_shared(q.data_ptr(), pages[0].data_ptr(), pages[1].data_ptr(), o.data_ptr(),
                                       lse.data_ptr(), t.data_ptr(), c.data_ptr(), n.data_ptr(), g.data_ptr(),
                                       pre.data_ptr(), T, S, NG, Hq, Hk, d, pages[0].shape[0], 32, t.shape[1],
                                       *q.stride()[:2], *pages[0].stride()[:3], *pages[1].stride()[:3], 0.11, 1, 0,
                                       room.data_ptr(), room.numel(), stream)
        assert st == fa.FA_OK
        return hooks.fa_get_device_status(stream)     # synchronises, reads and clears

    return call, o, lse, ref


MANY = ([(700, [(1, 400 + i) for i in range(200)])], 32, 8)     # more units than CTAs, of several stages
WIDE = ([(700, [(1, 400 + i) for i in range(60)])], 64, 4)      # 16 rows: joined by all warps
FORMS = [("fa_test_paged", SHAPES["long, two tiles"], 64), ("fa_test_paged", SHAPES["one tile"], 128),
         ("fa_test_paged", SHAPES["chunks"], 64), ("fa_test_rows", MANY, 128), ("fa_test_rows", WIDE, 64)]
IDS = ["two tiles", "one tile", "chunks", "rows", "wide rows"]


@pytest.mark.parametrize("hook,shape,d", FORMS, ids=IDS)
def test_gives_up_and_the_next_call_is_clean(hooks, hook, shape, d):
    call, o, lse, ref = shared_call(hooks, shape, d)
    assert call() == fa.FA_OK
    check(o, lse, ref)
    assert getattr(hooks, hook)(1) == 0
    try:
        t0 = time.time()
        st = call()
        took = time.time() - t0
    finally:
        assert getattr(hooks, hook)(0) == 0
    assert st == fa.FA_ERR_DEVICE_TIMEOUT, fa.fa_status_string(st)
    assert took < 30.0
    assert call() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("hook,shape,d", FORMS, ids=IDS)
def test_ctas_that_do_not_start_merge_nothing(hooks, hook, shape, d):
    """Rows that wait for parts of CTAs that left at once stay as they were, whatever the workspace holds."""
    call, o, lse, ref = shared_call(hooks, shape, d)
    assert getattr(hooks, hook)(2) == 0
    try:
        assert call() == fa.FA_ERR_INTERNAL
    finally:
        assert getattr(hooks, hook)(0) == 0
    assert bool((o == 3).all()) and bool((lse == 4).all())
    assert call() == fa.FA_OK
    check(o, lse, ref)
