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
