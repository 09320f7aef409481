"""Shared keys and the cache's tables at the edges of what their calls allow (needs a GB300).

Tolerances are those of tests/test_gpu_paged.py (its ``check``); tables are whole numbers and equal the plain form's.
"""

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from tests.gpu_util import require_gpu
from tests.test_gpu_norm_rope import status
from tests.test_gpu_paged import check, reference
from tests.test_gpu_paged_shared import batch, call
from tests.test_gpu_paged_tables import State

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("groups", [0, 1])
@pytest.mark.parametrize("what", ["keys", "rows"])
@pytest.mark.parametrize("S,at", [(3, 2), (300, 299), (600, 511), (600, 512), (600, 599), (1300, 1024)])
def test_lengths_of_every_sequence_are_checked(S, at, what, groups):
    """More sequences than the plan's block has threads, with groups and without: a length out of range is said
    wherever it stands, and the other sequences are right."""
    q, pages, table, cu, lens, _, _ = batch([(0, [(1, 1 + i % 40) for i in range(S)])], 2, 1, 64, 16, False)
    if what == "keys":
        lens[at] = -1                             # no keys, then: a row of zeros
    else:
        cu[at + 1:] += 3                          # three rows more, the last ones behind the batch
        q = torch.cat([q, q[:3]])
        cu[-1] += 7                               # (cut to the batch's rows)
    x = (q, pages, table, cu, lens, torch.tensor([S] * (groups + 1), dtype=torch.int32),
         torch.zeros(groups, dtype=torch.int32))
    o, lse = call(x, scale=0.2)
    assert status() == fa.FA_ERR_DEVICE_INDEX and status() == fa.FA_OK
    good = lens.clamp_min(0), cu.clamp_max(q.shape[0])
    check(o, lse, reference(q, pages, table, good[1], good[0], 0.2, True))


@pytest.mark.parametrize("page", [-1, 9, 2 ** 31 - 1])
def test_a_page_outside_of_the_pool_has_no_slots(page):
    """In a request's row, or come back to the pool from there: tokens in it have the slot -1, and every call that
    meets it says so."""
    s = State([40], 4, 16, 9)
    s.table[0, 2] = s.plain.table[0, 2] = page    # the page that the next tokens go to
    _, _, _, _, slots = s.extend([0], [12])
    assert (slots < 0).tolist() == [True] * 8 + [False] * 4
    s.table[0, 1] = s.plain.table[0, 1] = page    # one that no new token goes to
    s.extend([0], [3])
    s.release([0])
    s = State([40, 0, 0], 4, 16, 9)
    s.table[0, 1] = s.plain.table[0, 1] = page
    s.release([0])
    got = s.extend([2, 1], [16, 40])              # takes all that came back
    assert (got[4] >= 0).sum() == 16 + 40 - 16
    s.extend([-1, 1], [0, 0])
    s.release([1, 2], [33, 16])
    s.extend([0], [5])


def test_pages_outside_of_the_pool_among_many():
    """More sequences than a block looks at: whichever block meets the page says so."""
    s = State([300] * 700, 40, 16, 700 * 19 + 700 * 2 + 5)
    s.table[650, 3] = s.plain.table[650, 3] = -4
    s.extend(list(range(700)), [1 + i % 9 for i in range(700)])
    s.extend([650], [1])
    s.extend([r for r in range(700) if r != 650], [20] * 699)
