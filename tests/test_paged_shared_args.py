"""What the attention of a batch that shares keys refuses (CPU only: validation fails before any device work)."""

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build
from tests.test_norm_rope_args import FWD_PAGED, INVALID, POOL, UNSUPPORTED, WORKSPACE, A

SHARED = dict(list(FWD_PAGED.items())[:8], groups=A, prefix_lens=A, T=5, S=2, num_groups=2,
              **dict(list(FWD_PAGED.items())[10:]))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load_library()


@pytest.mark.parametrize("kw,code", POOL + [
    (dict(d=96), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hq=5), INVALID),
    (dict(Hq=258), UNSUPPORTED), (dict(T=1 << 30), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(causal=2), INVALID), (dict(max_q=-1), INVALID), (dict(q=A + 8), INVALID), (dict(o=None), INVALID),
    (dict(lse=A + 2), INVALID), (dict(q_stride_h=68), INVALID), (dict(num_groups=-1), INVALID),
    (dict(num_groups=4097), UNSUPPORTED), (dict(groups=None), INVALID), (dict(prefix_lens=None), INVALID),
    (dict(groups=A + 2), INVALID), (dict(prefix_lens=A + 1), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace=A + 64), WORKSPACE), (dict(num_groups=0, groups=None, prefix_lens=None, workspace=None), WORKSPACE),
    (dict(T=0), fa.FA_OK), (dict(S=0, q=None, o=None, workspace=None, groups=None), fa.FA_OK),
])
def test_refusals(kw, code):
    assert fa.fa_fwd_paged_shared(**(SHARED | kw)) == code


@pytest.mark.parametrize("args", [(0, 2, 1, 4, 64), (5, 0, 1, 4, 64), (5, 2, -1, 4, 64), (5, 2, 4097, 4, 64),
                                  (5, 2, 1, 0, 64), (5, 2, 1, 1 << 15, 64), (5, 2, 1, 4, 96), (1 << 30, 2, 1, 4, 64)])
def test_workspace_size_of_invalid_sizes_is_zero(args):
    assert fa.fa_fwd_paged_shared_workspace_size(*args) == 0


def test_helper_rejects_cpu_tensors():
    x, i = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_forward_shared(x, x[None], x[None], i[None], i, i[:1], i, i[:1])
