"""What the calls on a paged cache's tables refuse, and the plain form of them by hand (CPU only)."""

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from oracle import serve
from tests.test_norm_rope_args import INVALID, UNSUPPORTED, A

STATE = dict(S=2, R=4, num_pages=8, page_size=16, max_pages=4, stream=None)
EXTEND = dict(requests=A, new_lens=A, request_lens=A, request_table=A, pool=A, cu_seqlens=A, kv_lens=A, page_table=A,
              positions=A, slots=A, T=5, **STATE)
RELEASE = dict(requests=A, keep_lens=A, kept_pages=A, request_lens=A, request_table=A, pool=A, **STATE)
BOTH = [
    (dict(S=-1), INVALID), (dict(R=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=(1 << 30) + 1), INVALID),
    (dict(max_pages=0), INVALID), (dict(page_size=8), INVALID), (dict(page_size=48), INVALID),
    (dict(page_size=1 << 17), INVALID), (dict(max_pages=1 << 27), INVALID), (dict(S=4097), UNSUPPORTED),
    (dict(R=16385), UNSUPPORTED), (dict(requests=None), INVALID), (dict(request_lens=None), INVALID),
    (dict(request_table=A + 2), INVALID), (dict(pool=None), INVALID), (dict(requests=A + 1), INVALID),
    (dict(S=0, requests=None, pool=None), fa.FA_OK),
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load_library()


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(T=-1), INVALID), (dict(new_lens=None), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(kv_lens=A + 2), INVALID), (dict(page_table=None), INVALID), (dict(positions=A + 2), INVALID),
    (dict(slots=A + 4), INVALID),
])
def test_extend_refusals(kw, code):
    assert fa.fa_paged_extend(**(EXTEND | kw)) == code


@pytest.mark.parametrize("kw,code", BOTH + [(dict(keep_lens=A + 2), INVALID), (dict(kept_pages=A + 1), INVALID)])
def test_release_refusals(kw, code):
    assert fa.fa_paged_release(**(RELEASE | kw)) == code


def test_pool():
    assert fa.paged_pool(3, device="cpu").tolist() == [3, 0, 2, 1, 0]
    with pytest.raises(ValueError):
        fa.paged_pool(0, device="cpu")


def test_helpers_reject_cpu_tensors():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_extend(i, i, i, i[None], i, 16, 4)
    with pytest.raises(ValueError):
        fa.paged_release(i, i, i[None], i, 16)


def test_the_plain_form_by_hand():
    """Pages of 16: request 2 grows from 15 to 18 keys, request 0 starts with 33, request 1 finds one page too few."""
    t = serve.Tables([0, 0, 15], np.full((3, 4), -1), [4, 3, 2, 1, 0], 6, 16)
    t.table[2, 0] = 5
    cu, kv, table, pos, slots = t.extend([2, -1, 0, 1], [3, 7, 33, 17], 60, np.full((4, 4), 9))
    assert cu.tolist() == [0, 3, 3, 36, 53] and kv.tolist() == [18, 0, 33, 0] and t.bad
    assert table.tolist() == [[5, 0, 9, 9], [9] * 4, [1, 2, 3, 9], [9] * 4] and t.free == [4]
    assert pos[:5].tolist() == [15, 16, 17, 0, 1] and pos[36:].tolist() == [-1] * 17 + [0] * 7
    assert slots[:4].tolist() == [5 * 16 + 15, 0, 1, 16] and slots[35] == 3 * 16 and set(slots[36:]) == {-1}
    assert t.lens == [33, 0, 18]
    t.release([0, 2], [17, 0], [0, 0, 1])             # request 2 does not own its first page
    assert t.free == [4, 0, 3] and t.lens == [17, 0, 0]
